// Device primitives of the serving kernels beyond minf_device.cuh: 8-bit
// tensor-core products, further operand layouts and TMEM access widths, a
// wait that ends at once after an abort, and dependent launches.  Written
// against the PTX ISA (tcgen05 / cp.async.bulk / griddepcontrol chapters).
#pragma once

#include "minf_device.cuh"

namespace minf {

// mbar_wait for roles that go on after a failure (their outputs are invalid and
// the status says so): once *abort is set, a wait that is not over ends at once.
__device__ __forceinline__ void mbar_wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort, DevStatus* st,
                                                   int where) {
  if (mbar_test(bar, parity) || *abort) return;
  const unsigned long long t0 = globaltimer();
  for (uint32_t it = 1; !mbar_test(bar, parity); ++it) {
    if (*abort) return;
    if ((it & 63) == 0 && globaltimer() - t0 > kWaitLimitNs) {
      *abort = 1;
      report(st, MINF_ERR_DEVICE_TIMEOUT, where);
      return;
    }
  }
}

// Whether the phase with the given parity is over; never suspends the thread.
__device__ __forceinline__ bool mbar_poll(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_lane() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Asynchronous copy of four bytes (4-byte aligned), global to shared.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// D(tmem) (+)= A(smem) * B(smem), kind::f8f6f4 (8-bit inputs, fp32 accumulate).
__device__ __forceinline__ void umma_ss_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// D(tmem) (+)= A(tmem) * B(smem), kind::f8f6f4 (A: four elements of a row in each 32-bit column).
__device__ __forceinline__ void umma_ts_f8(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::f8f6f4 with fp32 D; A and B are e4m3 or e5m2.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, int a_e5m2, int b_e5m2, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)a_e5m2 << 7) | ((uint32_t)b_e5m2 << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Shared-memory matrix descriptor; layout 0: no swizzle, 2: 128-byte, 4: 64-byte.
// Unswizzled K-major: 16-byte columns `lbo` apart, 8-row groups `sbo` apart.
// Unswizzled MN-major: 16-byte MN groups `sbo` apart, 8-row K groups `lbo` apart.
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t layout) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
         (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1u << 46 | (uint64_t)layout << 61;
}

// 32 lanes x 4, 8 or 16 consecutive 32-bit TMEM columns; valid after tmem_wait_ld().
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }
// Waits for the thread's TMEM loads, and ties the values of `r` to that wait.
template <int N>
__device__ __forceinline__ void tmem_landed(uint32_t (&r)[N]) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Largest value over the warp's lanes; NaN counts as -infinity.  The float's bits
// are made ordered as a signed integer, for the integer warp reduction.
__device__ __forceinline__ float warp_max(float x) {
  int k = __float_as_int(x == x ? x : -INFINITY);
  k ^= (k >> 31) & 0x7fffffff;
  k = __reduce_max_sync(0xFFFFFFFFu, k);
  return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
}

// Lets the dependent launch begin; waits until the launch depended on is over
// and its writes are visible.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_prerequisite() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// An ordinary load, for whatever an earlier launch may have written.  The read-only
// path (ld.global.nc) is for memory that nobody writes during the kernel's life, and
// a kernel that is launched early lives while its predecessor still writes; what the
// wait makes visible is promised to ordinary loads.
template <class T>
__device__ __forceinline__ T load(const T* p) {
  return *p;
}

// Launches a kernel that may begin before the one before it in the stream is over,
// and waits for that (wait_prerequisite) before it touches global memory.  A
// kernel lets the next begin (launch_dependents) when all of its own blocks are
// resident, so none that waits can keep out one that is waited for.
template <class... Params, class... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                         Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

}  // namespace minf
