// Attention of new tokens over the cache with more than 64 rows (tokens times
// query heads) of a KV head: groups of 128 rows fill the tensor instruction, so
// the products run the plain way round, S = Q K^T and O += P V with the rows as
// lanes.  A softmax thread owns one row and half of a tile's keys: its maximum
// and its sum are its own, and the weights stay in TMEM, over their scores, as
// the second product's operand.  (Keys as lanes, as tree_attn.cu has them, take
// 128 registers of a thread for 128 rows' sums, and their weights shared memory.)
//
// Bound, for 16-bit caches, by the softmax's chain and the tensor pipe (1024
// cycles a tile) rather than by memory: 256 rows of each of 8 KV heads over 131,064
// positions take 142 to 147 us at full clocks (208 transposed; 168 to 180 in long
// rows of calls, under the power cap), 225 us in 8 bits (357 transposed).  8-bit keys,
// values, queries and weights are multiplied as tree_attn.cu describes; the keys' and
// values' powers of two are read per tile from shared memory, a row's own factor from
// its thread.  All exponentials are the hardware's: running part of them as
// polynomials on the FMA pipe, as the pre-fill kernel does, has not been measured.
#include <cuda_fp8.h>

#include <type_traits>

#include "tree_attn.cuh"

namespace minf {

namespace {

template <int D, bool F8>
struct Wide {
  static constexpr int kSoft = 256;                 // two warpgroups: keys 0-63 and 64-127 of every tile
  static constexpr int kThreads = kSoft + 96;       // and the issuer, the K and the V producer
  static constexpr int kRowB = D * (F8 ? 1 : 2);
  static constexpr int kPitch = kRowB < 128 ? kRowB : 128;
  static constexpr int kRegions = kRowB / kPitch;
  static constexpr int kRegion = 128 * kPitch;
  static constexpr int kTileB = 128 * kRowB;
  static constexpr int kQParts = F8 ? 2 : 1, kPParts = F8 ? 3 : 1;
  static constexpr int kQPart = 128 * kRowB;
  static constexpr int kExpB = F8 ? 256 : 0;
  static constexpr int kKeyB = F8 ? 2 * 3 * 512 : 0;  // of two tiles' keys: 2^key exponents, value exponents, 2^-those
  static constexpr int kTiles = (232448 - kQParts * kQPart - kKeyB - 8 * kExpB - 3 * 1024) / kTileB;
  static constexpr int kKStages = (kTiles + 1) / 2 < 8 ? (kTiles + 1) / 2 : 8;
  static constexpr int kVStages = kTiles / 2 < 8 ? kTiles / 2 : 8;
  static constexpr int kOffV = 0;
  static constexpr int kOffK = kOffV + kVStages * kTileB;
  static constexpr int kOffQ = kOffK + kKStages * kTileB;
  static constexpr int kOffExp = kOffQ + kQParts * kQPart;
  static constexpr int kOffKey = kOffExp + kKStages * kExpB;
  static constexpr int kOffFac = kOffKey + kKeyB;   // [128] row factors
  static constexpr int kOffML = kOffFac + 512;      // [2][128] (maximum, sum)
  static constexpr int kOffBars = kOffML + 2048;
  // k_full, k_empty, v_full, v_empty, s_full[2], p_full[2], pv_done[2], q_full, mma_done
  static constexpr int kNumBars = 2 * kKStages + 2 * kVStages + 8;
  static constexpr int kOffMisc = kOffBars + kNumBars * 8;
  static constexpr int kSmem = kOffMisc + 64;
  static constexpr uint32_t kSwizzle = kPitch == 128 ? 2u : 4u;
  static constexpr uint32_t kGroup8 = 8 * kPitch;
  static constexpr int kOffO = 256;                 // TMEM: S of two tiles (128 columns each), then O of two halves
  static constexpr uint32_t kIdescS = F8 ? idesc_f8(128, 128, 0, 0, 0, 0) : idesc_bf16(128, 128, 0, 0);
  static constexpr uint32_t kIdescO = F8 ? idesc_f8(128, D, 1, 0, 0, 1) : idesc_bf16(128, D, 0, 1);
  // the weights' reference lies kOff below the maximum seen; kTop above it, it moves.
  // The three 8-bit parts share one accumulator and its lowest step, 2^-16: weights
  // are held to half of that, 2^-27 of the row's largest (kOff 4, 2^-21, is no faster)
  static constexpr float kOff = F8 ? 10.f : 0.f, kTop = F8 ? 15.f : 8.f;
  static_assert(kVStages >= 2 && kKStages >= 2 && kSmem <= 232448, "shared memory");
};

template <int D, bool F8>
__global__ void __launch_bounds__(Wide<D, F8>::kThreads, 1)
    tree_wide_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const TreeParams p) {
  using C = Wide<D, F8>;
  constexpr int NR = 128;
  constexpr int kIssuer = 8, kLoadK = 9, kLoadV = 10;  // warps
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part_lane = blockIdx.x / p.groups, rg = blockIdx.x % p.groups;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kOffBars);
  uint64_t* k_empty = k_full + C::kKStages;
  uint64_t* v_full = k_empty + C::kKStages;
  uint64_t* v_empty = v_full + C::kVStages;
  uint64_t* s_full = v_empty + C::kVStages;
  uint64_t* p_full = s_full + 2;
  uint64_t* pv_done = p_full + 2;
  uint64_t* q_full = pv_done + 2;
  uint64_t* mma_done = q_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  Walk* start = reinterpret_cast<Walk*>(smem + C::kOffML);  // until the roles have copied it

  if ((smem_u32(smem) & 1023u) != 0u) {
    if (threadIdx.x == 0) report(p.status, MINF_ERR_DEVICE_BOUNDS, 112);
    return;
  }
  if (warp == kIssuer) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  } else if (warp == kLoadK) {
    if (lane == 0) {
      for (int s = 0; s < C::kKStages; ++s) {
        mbar_init(&k_full[s], 1);
        mbar_init(&k_empty[s], F8 ? 5 : 1);  // 8-bit: also the four warps that read the tile's exponents
      }
      for (int s = 0; s < C::kVStages; ++s) {
        mbar_init(&v_full[s], 1);
        mbar_init(&v_empty[s], 1);
      }
      for (int w = 0; w < 2; ++w) {
        mbar_init(&s_full[w], 1);
        mbar_init(&p_full[w], C::kSoft);
        mbar_init(&pv_done[w], 1);
      }
      mbar_init(q_full, C::kSoft);
      mbar_init(mma_done, 1);
      *abort = 0;
      fence_mbar_init();
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
    }
  }
  if (warp == 0) {
    const Walk w = block_share(p, part_lane);
    if (lane == 0) *start = w;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  launch_dependents();
  const uint32_t tmem = *tmem_slot;
  Walk w = *start;
  __syncthreads();

  if (warp == kLoadK || warp == kLoadV) {
    // ----------------------------------------------------------- producers
    const bool is_k = warp == kLoadK;
    load_tiles<C, F8, NR>(p, is_k ? tmK : tmV, is_k, smem, is_k ? k_full : v_full, is_k ? k_empty : v_empty, rg, w, abort);
  } else if (warp == kIssuer) {
    // --------------------------------------------------------- MMA issuer
    // S(t) goes out before P V(t - 1): the next tile's scores are formed while the
    // softmax works on this one's.  S(t) takes the buffer of P(t - 2), which the
    // products before it in the pipe have read.
    const uint64_t q0 = sdesc(smem_u32(smem + C::kOffQ), NR * 16, 128, 0);
    const uint64_t k0 = sdesc(smem_u32(smem + C::kOffK), 16, C::kGroup8, C::kSwizzle);
    const uint64_t v0 = sdesc(smem_u32(smem + C::kOffV), C::kRegion, C::kGroup8, C::kSwizzle);
    int it = 0, segs = 0;
    auto issue_pv = [&](int i, bool first) {
      const int b = i & 1, st = i % C::kVStages;
      mbar_wait_or_abort(&p_full[b], (i >> 1) & 1, abort, p.status, 117);
      mbar_wait_or_abort(&v_full[st], (i / C::kVStages) & 1, abort, p.status, 118);
      if (__any_sync(0xFFFFFFFFu, *abort)) return;
      tc_fence_after();
      const uint64_t v = v0 + (uint32_t)(st * (C::kTileB / 16));
      if (elect_lane()) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a = tmem + b * 128 + h * 64, d = tmem + C::kOffO + h * D;
#pragma unroll
          for (int part = 0; part < C::kPParts; ++part)
#pragma unroll
            for (int kk = 0; kk < (F8 ? 2 : 4); ++kk) {
              constexpr int kKeys = F8 ? 32 : 16;
              const uint64_t vb = v + (uint32_t)((h * 64 + kk * kKeys) * C::kPitch / 16);
              const uint32_t acc = part > 0 || kk > 0 || !first;
              if constexpr (F8) umma_ts_f8(d, a + part * 16 + kk * 8, vb, C::kIdescO, acc);
              else umma_ts(d, a + kk * 8, vb, C::kIdescO, acc);
            }
        }
        umma_commit(&v_empty[st]);
        umma_commit(&pv_done[b]);
      }
      __syncwarp();
    };
    while (!__any_sync(0xFFFFFFFFu, *abort) && w.next(p)) {
      if (rg * NR >= w.nd * p.group) continue;
      mbar_wait_or_abort(q_full, segs & 1, abort, p.status, 119);
      ++segs;
      const int n = w.t1 - w.t0;
      for (int i = 0; i < n; ++i, ++it) {
        const int st = it % C::kKStages;
        mbar_wait_or_abort(&k_full[st], (it / C::kKStages) & 1, abort, p.status, 120);
        if (__any_sync(0xFFFFFFFFu, *abort)) break;
        const uint64_t k = k0 + (uint32_t)(st * (C::kTileB / 16));
        const uint32_t d = tmem + (it & 1) * 128;
        if (elect_lane()) {
#pragma unroll
          for (int part = 0; part < C::kQParts; ++part)
#pragma unroll
            for (int kk = 0; kk < C::kRowB / 32; ++kk) {
              const uint64_t a = q0 + (uint32_t)((part * C::kQPart + kk * 2 * NR * 16) / 16);
              const uint64_t b = k + (uint32_t)(((kk * 32 / C::kPitch) * C::kRegion + (kk * 32) % C::kPitch) / 16);
              const uint32_t acc = part > 0 || kk > 0;
              if constexpr (F8) umma_ss_f8(d, a, b, C::kIdescS, acc);
              else umma_ss(d, a, b, C::kIdescS, acc);
            }
          umma_commit(&s_full[it & 1]);
          umma_commit(&k_empty[st]);
        }
        __syncwarp();
        if (i > 0) issue_pv(it - 1, i == 1);
      }
      if (!__any_sync(0xFFFFFFFFu, *abort)) issue_pv(it - 1, n == 1);
    }
    if (elect_lane()) umma_commit(mma_done);
    __syncwarp();
    if (lane == 0) {
      int dummy = 0;
      mbar_wait(mma_done, 0, &dummy, p.status, 121);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- softmax
    // A failed wait is not followed up here: the status word and *abort are set,
    // every later wait ends at once, and the barriers below keep their counts.
    const int wg = warp >> 2, tid = threadIdx.x & 127;  // half of the keys; row (TMEM lane)
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    float* fac = reinterpret_cast<float*>(smem + C::kOffFac);
    float2* ml = reinterpret_cast<float2*>(smem + C::kOffML);
    const int bar_wg = 1 + wg, bar_all = 3;
    int it = 0;
    while (w.next(p)) {
      const int rows = min(NR, w.nd * p.group - rg * NR);
      if (rows <= 0) continue;
      const int len = w.ctx + w.nd, n = w.t1 - w.t0;
      const long long qb = ((long long)w.b * p.Hq + w.h * p.group) * p.T;  // first query row of the KV head
      // ---- this thread's row, and the segment's queries as the A operand
      const int t = (unsigned)(rg * NR + tid) / (unsigned)p.group;
      const long long row = qb + (rg * NR + tid - t * p.group) * p.T + t;
      unsigned long long word = 0;
      if (tid < rows) {
        word = p.mask ? p.mask[(long long)w.b * p.T + t] : (2ull << t) - 1;
        if (w.nd < 64) word &= (1ull << w.nd) - 1;
      }
      if constexpr (!F8) {
        constexpr int kPieces = D / 16;  // 16-byte pieces of the row, the warpgroups taking alternate ones
        uint4 x[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          x[i] = tid < rows ? load(reinterpret_cast<const uint4*>(p.q + row * D) + 2 * i + wg) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          *reinterpret_cast<uint4*>(smem + C::kOffQ + (2 * i + wg) * NR * 16 + tid * 16) = x[i];
      } else {
        constexpr int E = D / 32;  // elements of a lane; a warp takes 16 rows, four at a time
#pragma unroll 1
        for (int r0 = warp * 16; r0 < warp * 16 + 16; r0 += 4) {
          uint32_t raw[4][E / 2];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = r0 + i, tr = (unsigned)(rg * NR + r) / (unsigned)p.group;
            const long long at = qb + (rg * NR + r - tr * p.group) * p.T + tr;
#pragma unroll
            for (int e = 0; e < E / 2; ++e)
              raw[i][e] = r < rows ? load(reinterpret_cast<const uint32_t*>(p.q + at * D) + lane * (E / 2) + e) : 0u;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = r0 + i;
            float x[E], top = 0.f;
            bool bad = false;
#pragma unroll
            for (int e = 0; e < E; ++e) {
              x[e] = __uint_as_float(e & 1 ? raw[i][e / 2] & 0xffff0000u : raw[i][e / 2] << 16);
              bad = bad || !(fabsf(x[e]) <= 3.4e38f);
              top = fmaxf(top, fabsf(x[e]));
            }
            top = warp_max(top);
            bad = __any_sync(0xFFFFFFFFu, bad);
            // 2^up brings the largest to [128, 256)
            const int up = top == 0.f ? 0 : min(100, 134 - (int)(__float_as_uint(top) >> 23));
            const float s = __uint_as_float((uint32_t)(127 + up) << 23);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
              const float2 a = make_float2(x[e] * s, x[e + 1] * s);
              const uint32_t hi = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
              const float2 back =
                  __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi, __NV_E4M3)));
              const uint32_t lo =
                  __nv_cvt_float2_to_fp8x2(make_float2(a.x - back.x, a.y - back.y), __NV_SATFINITE, __NV_E4M3);
              const int byte = lane * E + e;
              uint8_t* q = smem + C::kOffQ + (byte / 16) * NR * 16 + r * 16 + byte % 16;
              *reinterpret_cast<uint16_t*>(q) = (uint16_t)hi;
              *reinterpret_cast<uint16_t*>(q + C::kQPart) = (uint16_t)lo;
            }
            if (lane == 0) fac[r] = bad ? NAN : p.scale_log2 * __uint_as_float((uint32_t)(127 - up) << 23);
          }
        }
      }
      fence_proxy_async();
      mbar_arrive(q_full);
      named_bar_sync(bar_all, C::kSoft);
      const float mul = F8 ? fac[tid] : p.scale_log2;
      const uint64_t mul2 = f32x2_pack(mul, mul);

      float m = -INFINITY, l = 0.f;  // reference and sum of the row's half
#pragma unroll 1
      for (int i = 0; i < n; ++i, ++it) {
        const int b = it & 1, kst = it % C::kKStages;
        const int j0 = (w.t0 + i) * 128 + wg * 64;  // first key of the half
        const uint32_t s_col = lanes + b * 128 + wg * 64;
        // the half's keys: 2^key exponent, value exponent, its inverse power (four keys a read)
        float* key_pow = reinterpret_cast<float*>(smem + C::kOffKey) + b * 384 + wg * 64;
        float *val_exp = key_pow + 128, *val_inv = key_pow + 256;
        bool ask = false, zeros = false;  // whether this key's (a key's) row may be of zeros
        if constexpr (F8) {
          if (tid < 64) {
            mbar_wait_or_abort(&k_full[kst], (it / C::kKStages) & 1, abort, p.status, 122);
            const uint8_t* e = smem + C::kOffExp + kst * C::kExpB + wg * 64 + tid;
            const uint32_t ke = e[0], ve = max((uint32_t)e[128], kLeastExp);
            __syncwarp();
            if (lane == 0) mbar_arrive(&k_empty[kst]);
            const bool in = j0 + tid < len;
            key_pow[tid] = !in ? 0.f : ke == 255u ? NAN : __uint_as_float(ke << 23);
            val_exp[tid] = !in ? 0.f : ve == 255u ? NAN : (float)((int)ve - 127);
            val_inv[tid] = !in ? 1.f : ve == 255u ? NAN : __uint_as_float((254u - ve) << 23);
            ask = in && ve == kZeroExp;
          }
          zeros = !bar_and(bar_wg, 128, !ask);
        }
        mbar_wait_or_abort(&s_full[b], (it >> 1) & 1, abort, p.status, 123);
        tc_fence_after();
        if (zeros) {
          // A row of zeros adds nothing to O, so it must not raise the reference, as the
          // power 2^0 that it is stored with would.  (This tile's scores were issued
          // behind the product of the tile before the last, so its values' stage is at
          // most one round behind and the wait is for the right one.)
          if (ask) {
            const int st = it % C::kVStages;
            mbar_wait_or_abort(&v_full[st], (it / C::kVStages) & 1, abort, p.status, 126);
            if (zero_row<C::kPitch>(smem + C::kOffV + st * C::kTileB + (wg * 64 + tid) * C::kPitch)) {
              val_exp[tid] = (float)((int)kLeastExp - 127);
              val_inv[tid] = __uint_as_float((254u - kLeastExp) << 23);
            }
          }
          named_bar_sync(bar_wg, 128);
        }
        uint32_t s[2][32];
        tmem_ld(s_col, s[0]);
        tmem_ld(s_col + 32, s[1]);
        tmem_landed(s[0]);
        tmem_landed(s[1]);
        // 8-bit: scores in powers of two with the values' exponents, in place
        if constexpr (F8) {
#pragma unroll
          for (int c = 0; c < 64; c += 4) {
            const float4 k = *reinterpret_cast<const float4*>(key_pow + c), v = *reinterpret_cast<const float4*>(val_exp + c);
            uint32_t* x = &s[c / 32][c % 32];
            float y[4];
            f32x2_unpack(f32x2_fma(f32x2_mul(f32x2_pack(__uint_as_float(x[0]), __uint_as_float(x[1])), f32x2_pack(k.x, k.y)),
                                   mul2, f32x2_pack(v.x, v.y)),
                         y[0], y[1]);
            f32x2_unpack(f32x2_fma(f32x2_mul(f32x2_pack(__uint_as_float(x[2]), __uint_as_float(x[3])), f32x2_pack(k.z, k.w)),
                                   mul2, f32x2_pack(v.z, v.w)),
                         y[2], y[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = __float_as_uint(y[e]);
          }
        }
        const int base = j0 - w.ctx;  // drafted index of the half's first key
        if (base + 63 >= 0) {
          // bit c: the row sees the half's key c (bits behind the sequence's end are zero)
          const unsigned long long vis = base >= 64    ? 0ull
                                         : base >= 0   ? word >> base
                                         : base > -64  ? word << -base | ((1ull << -base) - 1)
                                                       : ~0ull;
          const uint32_t v2[2] = {(uint32_t)vis, (uint32_t)(vis >> 32)};
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (!(v2[c / 32] >> (c % 32) & 1)) s[c / 32][c % 32] = 0xff800000u;  // -infinity
        }
        float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 64; ++c) top4[c & 3] = fmaxf(top4[c & 3], __uint_as_float(s[c / 32][c % 32]));
        float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
        // in powers of two (16-bit scores are still unscaled; the scale is positive)
        if constexpr (!F8) top *= mul;
        if (__any_sync(0xFFFFFFFFu, top > m + C::kTop || m == -INFINITY)) {
          const float now = fmaxf(fmaxf(m, top - C::kOff), kFloor);
          if (i > 0) {
            // O and l follow; the O before this tile's product is complete
            const float f = fast_exp2(m - now);
            mbar_wait_or_abort(&pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1, abort, p.status, 124);
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              uint32_t o[32];
              tmem_ld(lanes + C::kOffO + wg * D + c0, o);
              tmem_landed(o);
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
              tmem_st32(lanes + C::kOffO + wg * D + c0, o);
            }
            tmem_wait_st();
            l *= f;
          }
          m = now;
        }
        const uint64_t nm2 = f32x2_pack(-m, -m);
        uint64_t sum[2] = {0ull, 0ull};
        auto weights2 = [&](uint32_t s0, uint32_t s1, float& p0, float& p1) {
          const uint64_t x = f32x2_pack(__uint_as_float(s0), __uint_as_float(s1));
          float t0, t1;
          if constexpr (F8) f32x2_unpack(f32x2_add(x, nm2), t0, t1);
          else f32x2_unpack(f32x2_fma(x, mul2, nm2), t0, t1);
          p0 = fast_exp2(t0);
          p1 = fast_exp2(t1);
        };
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (!F8) {
            uint32_t out[16];
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              float p0, p1;
              weights2(s[h][c], s[h][c + 1], p0, p1);
              sum[c / 2 & 1] = f32x2_add(sum[c / 2 & 1], f32x2_pack(p0, p1));
              out[c / 2] = pack_bf16x2(p0, p1);
            }
            tmem_st16(s_col + h * 16, out);
          } else {
            uint32_t out[3][8];
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              uint32_t x[2];
              const float4 iv = *reinterpret_cast<const float4*>(val_inv + h * 32 + c);
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                float p0, p1;
                weights2(s[h][c + 2 * g], s[h][c + 2 * g + 1], p0, p1);
                sum[g] = f32x2_fma(f32x2_pack(p0, p1), g == 0 ? f32x2_pack(iv.x, iv.y) : f32x2_pack(iv.z, iv.w), sum[g]);
                const __half2 two = __floats2half2_rn(p0, p1);
                x[g] = *reinterpret_cast<const uint32_t*>(&two);
              }
              // e5m2 is the upper byte of a half: each part is the remainder rounded
              // there (half a step up, in magnitude), and leaves an exact remainder.
              // A NaN weight may be lost here, not in l.
#pragma unroll
              for (int q = 0; q < 3; ++q) {
                const uint32_t a = x[0] + 0x00800080u, bb = x[1] + 0x00800080u;
                out[q][c / 4] = __byte_perm(a, bb, 0x7531);
                const uint32_t ta = a & 0xff00ff00u, tb = bb & 0xff00ff00u;
                const __half2 ra = __hsub2(*reinterpret_cast<const __half2*>(&x[0]), *reinterpret_cast<const __half2*>(&ta));
                const __half2 rb = __hsub2(*reinterpret_cast<const __half2*>(&x[1]), *reinterpret_cast<const __half2*>(&tb));
                x[0] = *reinterpret_cast<const uint32_t*>(&ra);
                x[1] = *reinterpret_cast<const uint32_t*>(&rb);
              }
            }
#pragma unroll
            for (int q = 0; q < 3; ++q) tmem_st(s_col + q * 16 + h * 8, out[q]);
          }
        }
        float a0, a1, a2, a3;
        f32x2_unpack(sum[0], a0, a1);
        f32x2_unpack(sum[1], a2, a3);
        l += (a0 + a1) + (a2 + a3);
        if (j0 + 64 > len) {
          // what lies behind the sequence's end may be anything: zero weight needs a
          // finite value (two threads a row of the half)
          const int st = it % C::kVStages, r = wg * 64 + (tid >> 1);
          if ((w.t0 + i) * 128 + r >= len) {
            mbar_wait_or_abort(&v_full[st], (it / C::kVStages) & 1, abort, p.status, 126);
            uint8_t* v = smem + C::kOffV + st * C::kTileB + r * C::kPitch + (tid & 1) * (C::kPitch / 2);
#pragma unroll
            for (int x = 0; x < C::kRegions; ++x)
#pragma unroll
              for (int o = 0; o < C::kPitch / 2; o += 16)
                *reinterpret_cast<uint4*>(v + x * C::kRegion + o) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async();
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[b]);
      }

      // ---- the segment's end: the two halves of every row joined
      mbar_wait_or_abort(&pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1, abort, p.status, 127);
      tc_fence_after();
      ml[wg * NR + tid] = make_float2(m, l);
      named_bar_sync(bar_all, C::kSoft);
      const float2 e0 = ml[tid], e1 = ml[NR + tid];
      const float M = fmaxf(e0.x, e1.x);
      float f0 = fast_exp2(e0.x - M), f1 = fast_exp2(e1.x - M);
      const float L = e0.y * f0 + e1.y * f1;
      const bool whole = w.t0 == 0 && w.t1 == w.nt;  // all of the sequence's tiles
      // a partial segment's sums go to the block's first or second place
      float* part = p.part + ((2ll * blockIdx.x + (w.t0 == 0 ? 1 : 0)) * NR + tid) * (D + 2);
      if (whole) {
        const float by = L == 0.f ? 0.f : 1.f / L;  // a row that saw nothing: 0, -infinity
        f0 *= by;
        f1 *= by;
      }
      if (wg == 0 && tid < rows) {
        if (!whole) *reinterpret_cast<float2*>(part + D) = make_float2(M, L);
        else if (p.lse) p.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
      }
      // the warpgroups take half of the row's elements each
#pragma unroll 1
      for (int c0 = wg * (D / 2); c0 < (wg + 1) * (D / 2); c0 += 32) {
        uint32_t a[32], b[32];
        tmem_ld(lanes + C::kOffO + c0, a);
        tmem_ld(lanes + C::kOffO + D + c0, b);
        tmem_landed(a);
        tmem_landed(b);
        if (tid < rows) {
          if (whole) {
#pragma unroll
            for (int c = 0; c < 32; c += 8) {
              uint32_t o[4];
#pragma unroll
              for (int e = 0; e < 8; e += 2)
                o[e / 2] = pack_bf16x2(__uint_as_float(a[c + e]) * f0 + __uint_as_float(b[c + e]) * f1,
                                       __uint_as_float(a[c + e + 1]) * f0 + __uint_as_float(b[c + e + 1]) * f1);
              *reinterpret_cast<uint4*>(p.o + row * D + c0 + c) = make_uint4(o[0], o[1], o[2], o[3]);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 32; c += 2)
              *reinterpret_cast<float2*>(part + c0 + c) =
                  make_float2(__uint_as_float(a[c]) * f0 + __uint_as_float(b[c]) * f1,
                              __uint_as_float(a[c + 1]) * f0 + __uint_as_float(b[c + 1]) * f1);
          }
        }
      }
      tc_fence_before();
      named_bar_sync(bar_all, C::kSoft);  // Q and the exchange are the next segment's
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool F8>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p, cudaStream_t stream) {
  using C = Wide<D, F8>;
  cudaError_t e = cudaFuncSetAttribute(tree_wide_kernel<D, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  // not ahead of its predecessor's end, as tree_attn.cu's are: long calls in a row
  // took 172 us instead of 168
  tree_wide_kernel<D, F8><<<p.lanes * p.groups, C::kThreads, C::kSmem, stream>>>(tk, tv, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t tree_wide_launch(int d, const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p,
                             cudaStream_t stream) {
  if (d == 128) return p.c.ke ? launch<128, true>(tk, tv, p, stream) : launch<128, false>(tk, tv, p, stream);
  return p.c.ke ? launch<64, true>(tk, tv, p, stream) : launch<64, false>(tk, tv, p, stream);
}

}  // namespace minf
