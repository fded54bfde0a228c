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

#include "serve_device.cuh"
#include "serve_internal.h"

namespace minf {

namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 4;  // rows a lane group has in flight

__device__ __forceinline__ float2 halves(uint32_t two) {  // of a bf16 pair
  return make_float2(__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u));
}

// A row takes D / 8 lanes of eight elements (one 16-byte load each).  A lane
// group takes `hb` consecutive heads of one token: its lanes form the cosines
// and sines of their own eight elements once, for all of those heads.
//
// Bound by memory (each row is read and written once: 131,072 tokens of 48 heads
// of 128 take 521 us in a row of calls, 0.94 of the measured copy rate; through
// read-only loads 549, and with those fewer or more rows in flight, more threads or
// streaming accesses up to 670) as long as few instructions go with a row: with the
// weights multiplied into the cosines and sines of the query and then the key heads,
//   y = inv * (x * (c w) + partner * (s w')),  inv = rsqrt(mean(x^2) + eps),
// and the partner arrives by exchanging the rows as read, two elements a word.
template <int D>
__global__ void __launch_bounds__(kThreads, 8) rope_kernel(const RopeParams p, int hb, int chunks) {
  constexpr int L = D / 8;
  constexpr int kRows = kThreads / L;
  __shared__ float2 angles[8][kThreads];  // (cos, sin) of each thread's elements, read by it alone
  const int lane = threadIdx.x % L;
  const long long item = (long long)blockIdx.x * kRows + threadIdx.x / L;
  launch_dependents();
  wait_prerequisite();
  if (item >= (long long)p.B * p.N * chunks) return;
  const unsigned group = (L == 16 ? 0xffffu : 0xffu) << ((threadIdx.x & 31) - lane);  // the group's lanes of the warp
  const int tok = (int)(item / chunks), h0 = (int)(item % chunks) * hb;
  const int b = tok / p.N, n = tok % p.N;
  const int turned = p.Hq + p.Hkv;
  const int h1 = min(h0 + hb, turned + (p.v ? p.Hkv : 0));
  const __nv_bfloat16* src = p.x + b * p.sb + n * p.sn + lane * 8;

  // the partner is element i +- rot / 2 (the same element of another lane), or
  // 2i + 1 of 2i and the reverse
  const int hl = p.rot / 16;
  const bool turn = lane * 8 < p.rot, low = lane < hl;
  const int from = !turn || p.interleaved ? lane : low ? lane + hl : lane - hl;  // of the group
  if (h0 < turned) {
    const double pos = (double)(p.pos ? load(p.pos + tok) : n) * 0.15915494309189533577;  // 1 / (2 pi)
    const int i0 = p.interleaved ? lane * 4 : (low ? lane : lane - hl) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float sn = 0.f, cs = 1.f;
      if (turn && !(p.interleaved && (e & 1))) {
        const double turns = pos * load(p.inv_freq + i0 + (p.interleaved ? e / 2 : e));
        sincospif(2.f * (float)(turns - rint(turns)), &sn, &cs);
        if (p.interleaved || low) sn = -sn;
      } else if (turn) {
        const float2 pair = angles[e - 1 + (e == 0)][threadIdx.x];
        cs = pair.x;
        sn = -pair.y;
      }
      angles[e][threadIdx.x] = make_float2(cs, sn);
    }
  }

  for (int kind = 0; kind < 3; ++kind) {  // query, key, value heads
    const int first = kind == 0 ? 0 : kind == 1 ? p.Hq : turned, heads = kind == 0 ? p.Hq : p.Hkv;
    const int ha = max(h0, first), hz = min(h1, first + heads);
    if (ha >= hz) continue;
    __nv_bfloat16* base = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
    __nv_bfloat16* dst = base + (((long long)b * heads - first) * p.N + n) * D + lane * 8;  // + head * N * D
    const __nv_bfloat16* w = kind == 0 ? p.qw : p.kw;
    float c[8], s[8];
    if (kind < 2) {
      uint4 wr = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u), wo = wr;  // ones
      if (w) {
        wr = load(reinterpret_cast<const uint4*>(w) + lane);
        wo = load(reinterpret_cast<const uint4*>(w) + from);
      }
      const uint32_t* w2 = reinterpret_cast<const uint32_t*>(&wr);
      const uint32_t* o2 = reinterpret_cast<const uint32_t*>(&wo);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 a = angles[e][threadIdx.x], own = halves(w2[e / 2]), other = halves(o2[e / 2]);
        c[e] = a.x * (e & 1 ? own.y : own.x);
        s[e] = a.y * ((e & 1) != (p.interleaved != 0) ? other.y : other.x);
      }
    }
    for (int h = ha; h < hz; h += kUnroll) {
      uint4 raw[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (h + u < hz) raw[u] = load(reinterpret_cast<const uint4*>(src + (long long)(h + u) * D));
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (h + u >= hz) break;
        uint4 out = raw[u];
        if (kind < 2) {
          uint32_t* x2 = reinterpret_cast<uint32_t*>(&out);
          float inv = 1.f;
          if (w) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = halves(x2[e]);
              ss = fmaf(f.x, f.x, fmaf(f.y, f.y, ss));
            }
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
            inv = rsqrtf(ss * (1.f / D) + p.eps);
          }
          uint32_t other[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            other[e] = p.interleaved ? __byte_perm(x2[e], 0, 0x1032) : __shfl_sync(group, x2[e], from, L);
            if (!turn) other[e] = 0;  // and not an infinite element times no sine
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = halves(x2[e]), o = halves(other[e]);
            const float y0 = fmaf(f.x, c[2 * e], o.x * s[2 * e]), y1 = fmaf(f.y, c[2 * e + 1], o.y * s[2 * e + 1]);
            x2[e] = pack_bf16x2(y0 * inv, y1 * inv);
          }
        }
        *reinterpret_cast<uint4*>(dst + (long long)(h + u) * p.N * D) = out;
      }
    }
  }
}

template <int D>
cudaError_t launch(const RopeParams& p, cudaStream_t stream) {
  const long long tokens = (long long)p.B * p.N;
  if (tokens == 0) return cudaSuccess;
  const int heads = p.Hq + (p.v ? 2 : 1) * p.Hkv;
  // as many heads of a token per lane group (they share its angles) as leave
  // about 16 thousand groups, a few for every place on the GPU (all of a prompt's
  // heads together; 24 apart cost it 770 us, 6 apart 1060)
  const int hb = (int)std::min<long long>(heads, std::max<long long>(1, tokens * heads / 16384));
  const int chunks = (heads + hb - 1) / hb;
  const int rows = kThreads / (D / 8);
  return launch_early(rope_kernel<D>, dim3((unsigned)((tokens * chunks + rows - 1) / rows)), kThreads, 0, stream, p, hb,
                      chunks);
}

}  // namespace

cudaError_t rope_launch(int d, const RopeParams& p, cudaStream_t stream) {
  if (d == 128) return launch<128>(p, stream);
  if (d == 64) return launch<64>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace minf
