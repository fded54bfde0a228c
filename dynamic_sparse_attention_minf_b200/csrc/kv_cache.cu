// The paged key-value cache: writing rows into it, as they are or in 8 bits,
// and reading them back into the dense layout of the pre-fill calls.
//
// An 8-bit row holds e4m3 values times one power of two, 2^e with the smallest
// e >= -80 for which max |x| <= 448 * 2^e (e = 0 for a row of zeros).  A power
// of two keeps the division and the product exact, so the only rounding is
// e4m3's own (at most 2^-4 of the value above 2^-6 * 2^e), what is read back
// is exact in bf16, and attention can take the scale into an exponent.  The
// scale costs one byte a row, e + 127; 255 marks a row that held a NaN or an
// infinity, which reads back as NaN.
#include <cuda_fp8.h>

#include <type_traits>

#include "serve_device.cuh"
#include "serve_internal.h"

namespace minf {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // rows (of K and of V) that a lane group has in flight

// Row index in the pools of position `at` of sequence b, or -1 with the error
// reported: the position is outside the table or its page outside the pool.
__device__ __forceinline__ long long pool_row(const KvView& c, int b, int h, long long at, DevStatus* st, int where) {
  const long long pi = at >> c.log_page;
  if (at < 0 || pi >= c.max_pages) {
    report(st, MINF_ERR_DEVICE_BOUNDS, where);
    return -1;
  }
  const int id = load(c.pages + (long long)b * c.max_pages + pi);
  if (id < 0 || id >= c.n_pages) {
    report(st, MINF_ERR_DEVICE_BOUNDS, where + 1);
    return -1;
  }
  return (((long long)id * c.Hkv + h) << c.log_page) + (at & ((1 << c.log_page) - 1));
}

// Eight bf16 of one lane to eight e4m3 bytes of the row's scale; every lane of
// the row's L gets the row's stored exponent.
template <int L>
__device__ __forceinline__ uint2 quantise8(const uint4& raw, uint32_t& exp_byte) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  // max |x| as ordered bf16 bits, two elements a word
  uint32_t two = __vimax3_u16x2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu, __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) two = __vmaxu2(two, __shfl_xor_sync(0xFFFFFFFFu, two, o));
  const uint32_t top = max(two & 0xffffu, two >> 16);
  const int ex = (int)(top >> 7);                       // biased exponent
  const int up = (top & 0x7fu) > 0x60u;                 // mantissa above 1.75 (448 = 1.75 * 2^8)
  const int e = top == 0 ? 0 : max(ex - 135 + up, -80);
  const bool bad = ex == 255;
  exp_byte = bad ? 255u : (uint32_t)(e + 127);
  const float s = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e
  uint32_t out[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t v = 0;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t x = w[2 * i + q];
      const float2 f = make_float2(__uint_as_float(x << 16) * s, __uint_as_float(x & 0xffff0000u) * s);
      v |= (uint32_t)__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3) << (16 * q);
    }
    out[i] = bad ? 0x7f7f7f7fu : v;
  }
  return make_uint2(out[0], out[1]);
}

__device__ __forceinline__ uint4 dequantise8(const uint2& q, uint32_t exp_byte) {
  const float s = exp_byte == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(exp_byte << 23);
  uint32_t out[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t two = (e < 2 ? q.x : q.y) >> (16 * (e & 1));
    const __half2 h(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xffffu), __NV_E4M3));
    const float2 f = __half22float2(h);
    out[e] = pack_bf16x2(f.x * s, f.y * s);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// One row of K and one of V per group of D / 8 lanes, kUnroll of them in
// flight; a block takes kRows * kUnroll tokens of one head.  Bound by memory:
// a 131,072-token prompt of 8 heads of 128 in 8 bits moves 807 MB in 136 us in a
// row of calls, 0.90 of the measured copy rate; back (kv_read_kernel) in 131 us,
// 0.94; in 16 bits 1,074 MB in 166 and 165 us, 0.98 and 0.99.  (Two rows in flight:
// 139 us, eight: 159 us.)
template <int D, bool F8>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvWriteParams p, int chunks) {
  constexpr int L = D / 8;
  constexpr int kRows = kThreads / L;
  const int lane = threadIdx.x % L, grp = threadIdx.x / L;
  const int bh = blockIdx.x / chunks, h = bh % p.c.Hkv, b = bh / p.c.Hkv;
  const int n0 = (blockIdx.x % chunks) * (kRows * kUnroll) + grp;
  launch_dependents();
  wait_prerequisite();
  int count = p.count ? load(p.count + b) : p.N;
  if (count < 0 || count > p.N) {
    if (threadIdx.x == 0) report(p.status, MINF_ERR_DEVICE_BOUNDS, 100);
    count = 0;
  }
  const int start = load(p.start + b);
  const __nv_bfloat16* kb = p.k + b * p.ksb + h * p.ksh + lane * 8;
  const __nv_bfloat16* vb = p.v + b * p.vsb + h * p.vsh + lane * 8;
  // lane u of a group finds out where its row u comes from and goes to
  int my_src = -1;
  long long my_dst = -1;
  if (lane < kUnroll) {
    const int n = n0 + lane * kRows;
    if (n < count) {
      my_src = p.rows ? load(p.rows + (long long)b * p.N + n) : n;
      if (my_src < 0 || my_src >= p.M) {
        report(p.status, MINF_ERR_DEVICE_BOUNDS, 101);
        my_src = -1;
      } else {
        my_dst = pool_row(p.c, b, h, start < 0 ? -1ll : (long long)start + n, p.status, 102);
      }
    }
  }
  uint4 rk[kUnroll], rv[kUnroll];
  long long dst[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int src = __shfl_sync(0xFFFFFFFFu, my_src, u, L);
    dst[u] = __shfl_sync(0xFFFFFFFFu, my_dst, u, L);
    rk[u] = rv[u] = make_uint4(0, 0, 0, 0);
    if (src >= 0) {
      // read once, and first to leave L2 (137 us for the 131,072-token prompt, 144 without)
      rk[u] = __ldcs(reinterpret_cast<const uint4*>(kb + src * p.ksn));
      rv[u] = __ldcs(reinterpret_cast<const uint4*>(vb + src * p.vsn));
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if constexpr (F8) {
      uint32_t ek, ev;  // every lane of the warp takes part in the row maxima
      const uint2 qk = quantise8<L>(rk[u], ek), qv = quantise8<L>(rv[u], ev);
      if (dst[u] < 0) continue;
      reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.c.k) + dst[u] * D)[lane] = qk;
      reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.c.v) + dst[u] * D)[lane] = qv;
      if (lane == 0) {
        p.c.ke[dst[u]] = (uint8_t)ek;
        p.c.ve[dst[u]] = (uint8_t)ev;
      }
    } else {
      if (dst[u] < 0) continue;
      reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.c.k) + dst[u] * D)[lane] = rk[u];
      reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.c.v) + dst[u] * D)[lane] = rv[u];
    }
  }
}

template <int D, bool F8>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvReadParams p, int chunks) {
  constexpr int L = D / 8;
  constexpr int kRows = kThreads / L;
  const int lane = threadIdx.x % L, grp = threadIdx.x / L;
  const int bh = blockIdx.x / chunks, h = bh % p.c.Hkv, b = bh / p.c.Hkv;
  const int n0 = (blockIdx.x % chunks) * (kRows * kUnroll) + grp;
  launch_dependents();
  wait_prerequisite();
  using Raw = typename std::conditional<F8, uint2, uint4>::type;
  const int len = min(load(p.lens + b), p.N);
  // lane u of a group finds its row u, and reads that row's exponents
  long long my_row = -1;
  uint32_t my_exp = 127 | 127 << 8;
  if (lane < kUnroll && n0 + lane * kRows < len) {
    my_row = pool_row(p.c, b, h, n0 + lane * kRows, p.status, 104);
    if (F8 && my_row >= 0) my_exp = load(p.c.ke + my_row) | (uint32_t)load(p.c.ve + my_row) << 8;
  }
  Raw rk[kUnroll], rv[kUnroll];
  uint32_t ek[kUnroll], ev[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long row = __shfl_sync(0xFFFFFFFFu, my_row, u, L);
    rk[u] = rv[u] = Raw{};
    if (row >= 0) {
      constexpr int kEl = F8 ? 1 : 2;
      rk[u] = load(reinterpret_cast<const Raw*>(static_cast<const uint8_t*>(p.c.k) + row * D * kEl) + lane);
      rv[u] = load(reinterpret_cast<const Raw*>(static_cast<const uint8_t*>(p.c.v) + row * D * kEl) + lane);
    }
  }
  if constexpr (F8) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t e = __shfl_sync(0xFFFFFFFFu, my_exp, u, L);
      ek[u] = e & 0xffu;
      ev[u] = e >> 8;
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int n = n0 + u * kRows;
    if (n >= p.N) continue;
    uint4 ok, ov;
    if constexpr (F8) {
      ok = dequantise8(rk[u], ek[u]);
      ov = dequantise8(rv[u], ev[u]);
    } else {
      ok = rk[u];
      ov = rv[u];
    }
    const long long row = (long long)bh * p.N + n;
    reinterpret_cast<uint4*>(p.k + row * D)[lane] = ok;
    reinterpret_cast<uint4*>(p.v + row * D)[lane] = ov;
  }
}

// chunks of a head's N rows
template <int D>
int chunks_of(int N) {
  const int per = kThreads / (D / 8) * kUnroll;
  return (N + per - 1) / per;
}

template <int D, bool F8>
cudaError_t launch_write(const KvWriteParams& p, cudaStream_t stream) {
  const int chunks = chunks_of<D>(p.N);
  return launch_early(kv_write_kernel<D, F8>, dim3((unsigned)(p.B * p.c.Hkv * chunks)), kThreads, 0, stream, p, chunks);
}
template <int D, bool F8>
cudaError_t launch_read(const KvReadParams& p, cudaStream_t stream) {
  const int chunks = chunks_of<D>(p.N);
  return launch_early(kv_read_kernel<D, F8>, dim3((unsigned)(p.B * p.c.Hkv * chunks)), kThreads, 0, stream, p, chunks);
}

}  // namespace

cudaError_t kv_write_launch(int d, const KvWriteParams& p, cudaStream_t stream) {
  if (p.N == 0) return cudaSuccess;
  if (d == 128) return p.c.ke ? launch_write<128, true>(p, stream) : launch_write<128, false>(p, stream);
  if (d == 64) return p.c.ke ? launch_write<64, true>(p, stream) : launch_write<64, false>(p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t kv_read_launch(int d, const KvReadParams& p, cudaStream_t stream) {
  if (p.N == 0) return cudaSuccess;
  if (d == 128) return p.c.ke ? launch_read<128, true>(p, stream) : launch_read<128, false>(p, stream);
  if (d == 64) return p.c.ke ? launch_read<64, true>(p, stream) : launch_read<64, false>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace minf
