// Head norm and position rotation of projected rows, written out in the
// [B, H, N, d] layout that every attention call of the library reads.
//
//   y = x * rsqrt(mean(x^2) + eps) * w          (query and key heads, given w)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = pos * inv_freq[i]
//
// over the first `rot` elements; a, b are elements i and i + rot / 2, or
// 2i and 2i + 1.  The angle is taken in 64 bits as a number of turns, of which
// only the fraction goes on in 32 bits: at position 10^6 a 32-bit product is
// off by 2^-4 of a radian, the fraction of a 64-bit one by 2^-30.  Everything
// else is in 32 bits with one rounding at the end.
#include <algorithm>

#include "minf_device.cuh"
#include "serve_internal.h"

namespace minf {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;  // tokens per block
constexpr int kUnroll = 4;     // rows a lane group has in flight

// A row takes D / 8 lanes of eight elements (one 16-byte load each).  A block
// takes `tb` tokens and `hb` heads: its tokens' cosines and sines are formed
// once, in shared memory, for all of their heads.
template <int D>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p, int tb, int hb) {
  constexpr int L = D / 8;
  constexpr int kRows = kThreads / L;
  __shared__ float2 cs[kMaxTokens][D / 2];
  const int lane = threadIdx.x % L, grp = threadIdx.x / L;
  const int heads = p.Hq + 2 * p.Hkv;
  const int h0 = blockIdx.y * hb, nh = min(hb, heads - h0);
  const long long tokens = (long long)p.B * p.N;
  const long long t0 = (long long)blockIdx.x * tb;
  const int nt = (int)min((long long)tb, tokens - t0);
  const int half = p.inv_freq ? p.rot / 2 : 0;
  if (h0 < p.Hq + p.Hkv) {
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
      const int t = i / half, f = i % half;
      const long long tok = t0 + t;
      const int pos = p.pos ? __ldg(p.pos + tok) : (int)(tok % p.N);
      constexpr double kInvTwoPi = 0.15915494309189533577;
      const double turns = (double)pos * (__ldg(p.inv_freq + f) * kInvTwoPi);
      float s, c;
      sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
      cs[t][f] = make_float2(c, s);
    }
  }
  __syncthreads();
  const int items = nt * nh;
  for (int i0 = grp; i0 < items; i0 += kRows * kUnroll) {
    uint4 raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kRows;
      if (i < items) {
        const int t = i / nh, h = h0 + i % nh;
        const long long tok = t0 + t;
        const __nv_bfloat16* src = p.x + (tok / p.N) * p.sb + (tok % p.N) * p.sn + (long long)h * D;
        raw[u] = __ldg(reinterpret_cast<const uint4*>(src) + lane);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kRows;
      // the whole warp goes through the shuffles below
      const bool live = i < items;
      const int t = live ? i / nh : 0, h = live ? h0 + i % nh : h0;
      if (!live) raw[u] = make_uint4(0, 0, 0, 0);
      const bool is_q = h < p.Hq, is_k = !is_q && h < p.Hq + p.Hkv;
      float x[8];
      const __nv_bfloat162* r2 = reinterpret_cast<const __nv_bfloat162*>(&raw[u]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = __bfloat1622float2(r2[e]);
        x[2 * e] = f.x;
        x[2 * e + 1] = f.y;
      }
      const __nv_bfloat16* w = is_q ? p.qw : is_k ? p.kw : nullptr;
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      if (w) {
        const float inv = rsqrtf(ss * (1.f / D) + p.eps);
        const uint4 wr = __ldg(reinterpret_cast<const uint4*>(w) + lane);
        const __nv_bfloat162* w2 = reinterpret_cast<const __nv_bfloat162*>(&wr);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = __bfloat1622float2(w2[e]);
          x[2 * e] = x[2 * e] * inv * f.x;
          x[2 * e + 1] = x[2 * e + 1] * inv * f.y;
        }
      }
      if (half) {
        const bool turn = (is_q || is_k) && lane * 8 < p.rot;
        if (p.interleaved) {
          if (turn) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 c = cs[t][lane * 4 + e];
              const float a = x[2 * e], b = x[2 * e + 1];
              x[2 * e] = a * c.x - b * c.y;
              x[2 * e + 1] = b * c.x + a * c.y;
            }
          }
        } else {
          // element i's partner i +- rot / 2 is the same element of another lane
          const int hl = p.rot / 16;
          const bool first = lane < hl;
          const int src = ((threadIdx.x & 31) - lane) + (turn ? (first ? lane + hl : lane - hl) : lane);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float other = __shfl_sync(0xFFFFFFFFu, x[e], src);
            if (turn) {
              const float2 c = cs[t][(first ? lane : lane - hl) * 8 + e];
              x[e] = first ? x[e] * c.x - other * c.y : x[e] * c.x + other * c.y;
            }
          }
        }
      }
      if (!live) continue;
      const long long tok = t0 + t;
      const long long b = tok / p.N, n = tok % p.N;
      __nv_bfloat16* dst;
      if (is_q)
        dst = p.q + ((b * p.Hq + h) * p.N + n) * D;
      else if (is_k)
        dst = p.k + ((b * p.Hkv + h - p.Hq) * p.N + n) * D;
      else if (p.v)
        dst = p.v + ((b * p.Hkv + h - p.Hq - p.Hkv) * p.N + n) * D;
      else
        continue;
      if (is_q || is_k) {
        uint32_t* o = reinterpret_cast<uint32_t*>(&raw[u]);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
      }
      reinterpret_cast<uint4*>(dst)[lane] = raw[u];
    }
  }
}

template <int D>
cudaError_t launch(const RopeParams& p, cudaStream_t stream) {
  const long long tokens = (long long)p.B * p.N;
  if (tokens == 0) return cudaSuccess;
  const int heads = p.Hq + (p.v ? 2 : 1) * p.Hkv;
  const int tb = (int)std::min<long long>(kMaxTokens, std::max<long long>(1, tokens / 592));
  const int rows = kThreads / (D / 8);
  // few tokens: one row per lane group, so that the heads spread over the SMs
  const int hb = tokens < 592 ? std::min(rows, heads) : heads;
  const long long nx = (tokens + tb - 1) / tb;
  const int ny = (heads + hb - 1) / hb;
  if (nx > 0x7fffffff || ny > 65535) return cudaErrorInvalidConfiguration;
  rope_kernel<D><<<dim3((unsigned)nx, ny), kThreads, 0, stream>>>(p, tb, hb);
  return cudaGetLastError();
}

}  // namespace

cudaError_t rope_launch(int d, const RopeParams& p, cudaStream_t stream) {
  if (d == 128) return launch<128>(p, stream);
  if (d == 64) return launch<64>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace minf
