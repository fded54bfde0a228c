// Attention of a few new tokens per sequence (one generated token, or a tree of
// drafted ones) over the paged key-value cache that already holds their keys
// and values behind the context's.
//
// Row t of a sequence sees every key of the context, and the drafted key u when
// bit u of its mask word is set.  Simple form: one block per row and split of
// the keys, one warp per key at a time with the head spread over its lanes,
// online softmax in 32 bits; a second kernel joins the splits in order.
#include <cuda_fp8.h>

#include <algorithm>

#include "minf_device.cuh"
#include "serve_internal.h"

namespace minf {

namespace {

constexpr int kMaxSplits = 64;

int splits_for(long long rows) { return (int)std::max<long long>(1, std::min<long long>(kMaxSplits, 2368 / rows)); }

struct Seq {
  int ctx, nd, len;
  bool ok;
};

// A sequence's lengths; a bad one counts as empty, and is reported by the caller.
__device__ __forceinline__ Seq seq_of(const TreeParams& p, int b) {
  Seq s;
  s.ctx = __ldg(p.ctx + b);
  s.nd = p.ndraft ? __ldg(p.ndraft + b) : p.T;
  s.ok = s.ctx >= 0 && s.nd >= 0 && s.nd <= p.T &&
         (long long)s.ctx + s.nd <= ((long long)p.c.max_pages << p.c.log_page);
  s.len = s.ok ? s.ctx + s.nd : 0;
  return s;
}

template <int D, bool F8>
__global__ void __launch_bounds__(128) tree_rows_kernel(const TreeParams p, int nsplit) {
  constexpr int E = D / 32;  // elements per lane
  const int row = blockIdx.y, split = blockIdx.x;
  const int t = row % p.T, hq = row / p.T % p.Hq, b = row / p.T / p.Hq;
  const int h = hq / p.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Seq s = seq_of(p, b);
  if (!s.ok && threadIdx.x == 0) report(p.status, MINF_ERR_DEVICE_BOUNDS, 110);
  float* part = p.part + ((long long)row * nsplit + split) * (D + 2);
  const unsigned long long mask = t < s.nd ? (p.mask ? p.mask[(long long)b * p.T + t] : (2ull << t) - 1) : 0ull;
  float q[E], acc[E];
  const __nv_bfloat16* qr = p.q + (long long)row * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(qr[e]) * p.scale_log2;
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int per = (s.len + nsplit - 1) / nsplit;
  const int j1 = t < s.nd ? min(s.len, (split + 1) * per) : 0;
  for (int j = split * per + warp; j < j1; j += 4) {
    if (j >= s.ctx && !(mask >> (j - s.ctx) & 1)) continue;
    const int id = __ldg(p.c.pages + (long long)b * p.c.max_pages + (j >> p.c.log_page));
    if (id < 0 || id >= p.c.n_pages) {
      if (lane == 0) report(p.status, MINF_ERR_DEVICE_BOUNDS, 111);
      continue;
    }
    const long long at = (((long long)id * p.c.Hkv + h) << p.c.log_page) + (j & ((1 << p.c.log_page) - 1));
    float k[E], v[E];
    if constexpr (F8) {
      const uint32_t ke = p.c.ke[at], ve = p.c.ve[at];
      const float ks = ke == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(ke << 23);
      const float vs = ve == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(ve << 23);
      const __nv_fp8_e4m3* kr = static_cast<const __nv_fp8_e4m3*>(p.c.k) + at * D + lane * E;
      const __nv_fp8_e4m3* vr = static_cast<const __nv_fp8_e4m3*>(p.c.v) + at * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        k[e] = (float)kr[e] * ks;
        v[e] = (float)vr[e] * vs;
      }
    } else {
      const __nv_bfloat16* kr = static_cast<const __nv_bfloat16*>(p.c.k) + at * D + lane * E;
      const __nv_bfloat16* vr = static_cast<const __nv_bfloat16*>(p.c.v) + at * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        k[e] = __bfloat162float(kr[e]);
        v[e] = __bfloat162float(vr[e]);
      }
    }
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) x = fmaf(q[e], k[e], x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    if (x == -INFINITY) continue;
    const float m2 = x == x ? fmaxf(m, x) : x, f = exp2f(m - m2), w = exp2f(x - m2);
    m = m2;
    l = l * f + w;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(w, v[e], acc[e] * f);
  }
  __shared__ float sm[4][D + 2];
#pragma unroll
  for (int e = 0; e < E; ++e) sm[warp][lane * E + e] = acc[e];
  if (lane == 0) {
    sm[warp][D] = m;
    sm[warp][D + 1] = l;
  }
  __syncthreads();
  float M = -INFINITY;
  for (int w = 0; w < 4; ++w) M = fmaxf(M, sm[w][D]);
  for (int i = threadIdx.x; i < D + 2; i += 128) {
    float a = 0.f;
    for (int w = 0; w < 4; ++w)
      if (sm[w][D] != -INFINITY) a += sm[w][i] * exp2f(sm[w][D] - M);
    part[i] = i == D ? M : a;
  }
}

template <int D>
__global__ void __launch_bounds__(D) tree_join_kernel(const TreeParams p, int nsplit) {
  const int row = blockIdx.x, t = row % p.T, b = row / p.T / p.Hq;
  if (t >= seq_of(p, b).nd || !seq_of(p, b).ok) return;  // rows behind the last token stay as they were
  const float* part = p.part + (long long)row * nsplit * (D + 2);
  float M = -INFINITY, l = 0.f, a = 0.f;
  for (int i = 0; i < nsplit; ++i) M = fmaxf(M, part[i * (D + 2) + D]);
  for (int i = 0; i < nsplit; ++i) {
    const float mi = part[i * (D + 2) + D];
    if (mi == -INFINITY) continue;
    const float f = exp2f(mi - M);
    l += part[i * (D + 2) + D + 1] * f;
    a += part[i * (D + 2) + threadIdx.x] * f;
  }
  p.o[(long long)row * D + threadIdx.x] = __float2bfloat16(M == -INFINITY ? 0.f : a / l);
  if (threadIdx.x == 0 && p.lse) p.lse[row] = M == -INFINITY ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
}

template <int D>
cudaError_t launch(const TreeParams& p, cudaStream_t stream) {
  const int rows = p.B * p.Hq * p.T, nsplit = splits_for(rows);
  if (rows > 65535) return cudaErrorInvalidConfiguration;
  if (p.c.ke) tree_rows_kernel<D, true><<<dim3(nsplit, rows), 128, 0, stream>>>(p, nsplit);
  else tree_rows_kernel<D, false><<<dim3(nsplit, rows), 128, 0, stream>>>(p, nsplit);
  tree_join_kernel<D><<<rows, D, 0, stream>>>(p, nsplit);
  return cudaGetLastError();
}

}  // namespace

size_t tree_part_floats(int B, int Hq, int, int T, int d) {
  const long long rows = (long long)B * Hq * T;
  return (size_t)rows * splits_for(rows) * (d + 2);
}

cudaError_t tree_attn_launch(int d, const TreeParams& p, cudaStream_t stream) {
  if (d == 128) return launch<128>(p, stream);
  if (d == 64) return launch<64>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace minf
