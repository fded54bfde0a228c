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
constexpr int kUnroll = 4;  // rows a lane group has in flight

// A row takes D / 8 lanes of eight elements (one 16-byte load each).  A lane
// group takes `hb` consecutive heads of one token: its lanes form the cosines
// and sines of their own eight elements once and keep them in registers for all
// of those heads.  Bound by memory: each row is read and written once.
template <int D>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p, int hb, int chunks) {
  constexpr int L = D / 8;
  constexpr int kRows = kThreads / L;
  const int lane = threadIdx.x % L;
  const long long item = (long long)blockIdx.x * kRows + threadIdx.x / L;
  // groups without work follow the last one through the shuffles, and store nothing
  const bool live = item < (long long)p.B * p.N * chunks;
  const int at = (int)(live ? item : (long long)p.B * p.N * chunks - 1);
  const int tok = at / chunks, h0 = (at % chunks) * hb;
  const int b = tok / p.N, n = tok % p.N;
  const int turned = p.Hq + p.Hkv;
  const int h1 = min(h0 + hb, turned + (p.v ? p.Hkv : 0));
  const __nv_bfloat16* src = p.x + b * p.sb + n * p.sn + lane * 8;

  // y = x * c + partner * s, the partner being element i +- rot / 2 (the same
  // element of another lane) or 2i + 1 of 2i and the reverse
  const int hl = p.rot / 16;
  const bool turn = lane * 8 < p.rot, low = lane < hl;
  const int from = ((threadIdx.x & 31) - lane) + (!turn || p.interleaved ? lane : low ? lane + hl : lane - hl);
  float c[8], s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    c[e] = 1.f;
    s[e] = 0.f;
  }
  if (turn && h0 < turned) {
    const double pos = (double)(p.pos ? __ldg(p.pos + tok) : n) * 0.15915494309189533577;  // 1 / (2 pi)
    const int i0 = p.interleaved ? lane * 4 : (low ? lane : lane - hl) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (p.interleaved && (e & 1)) continue;
      const double turns = pos * __ldg(p.inv_freq + i0 + (p.interleaved ? e / 2 : e));
      sincospif(2.f * (float)(turns - rint(turns)), &s[e], &c[e]);
      if (p.interleaved) {
        c[e + 1] = c[e];
        s[e + 1] = s[e];
        s[e] = -s[e];
      } else if (low) {
        s[e] = -s[e];
      }
    }
  }
  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  if (p.qw) wq = __ldg(reinterpret_cast<const uint4*>(p.qw) + lane);
  if (p.kw) wk = __ldg(reinterpret_cast<const uint4*>(p.kw) + lane);

  for (int h = h0; h < h0 + hb; h += kUnroll) {  // the same trip count in every group of a warp
    uint4 raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      raw[u] = make_uint4(0, 0, 0, 0);
      if (h + u < h1) raw[u] = __ldg(reinterpret_cast<const uint4*>(src + (long long)(h + u) * D));
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int hh = h + u;
      const bool is_q = hh < p.Hq, is_k = !is_q && hh < turned;
      float x[8];
      const __nv_bfloat162* r2 = reinterpret_cast<const __nv_bfloat162*>(&raw[u]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = __bfloat1622float2(r2[e]);
        x[2 * e] = f.x;
        x[2 * e + 1] = f.y;
      }
      if (p.qw || p.kw) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        if (is_q ? p.qw != nullptr : p.kw != nullptr) {
          const float inv = rsqrtf(ss * (1.f / D) + p.eps);
          const uint4 wr = is_q ? wq : wk;
          const __nv_bfloat162* w2 = reinterpret_cast<const __nv_bfloat162*>(&wr);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = __bfloat1622float2(w2[e]);
            x[2 * e] = x[2 * e] * inv * f.x;
            x[2 * e + 1] = x[2 * e + 1] * inv * f.y;
          }
        }
      }
      if (p.rot) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float other = p.interleaved ? x[e ^ 1] : __shfl_sync(0xFFFFFFFFu, x[e], from);
          y[e] = turn ? x[e] * c[e] + other * s[e] : x[e];  // an infinite partner stays out of unturned elements
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = y[e];
      }
      if (!live || hh >= h1) continue;
      __nv_bfloat16* dst;
      if (is_q) dst = p.q + (((long long)b * p.Hq + hh) * p.N + n) * D;
      else if (is_k) dst = p.k + (((long long)b * p.Hkv + hh - p.Hq) * p.N + n) * D;
      else dst = p.v + (((long long)b * p.Hkv + hh - turned) * p.N + n) * D;
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
  // as many heads of a token per lane group (they share its angles) as leave
  // about 16 thousand groups, a few for every place on the GPU
  const int hb = (int)std::min<long long>(heads, std::max<long long>(1, tokens * heads / 16384));
  const int chunks = (heads + hb - 1) / hb;
  const int rows = kThreads / (D / 8);
  rope_kernel<D><<<(unsigned)((tokens * chunks + rows - 1) / rows), kThreads, 0, stream>>>(p, hb, chunks);
  return cudaGetLastError();
}

}  // namespace

cudaError_t rope_launch(int d, const RopeParams& p, cudaStream_t stream) {
  if (d == 128) return launch<128>(p, stream);
  if (d == 64) return launch<64>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace minf
