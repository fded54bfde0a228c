// Attention of a few new tokens per sequence (one generated token, or a tree of
// drafted ones) over the paged key-value cache that already holds their keys
// and values behind the context's.
//
//   s = scale q.k,  O = sum_j 2^(s_j log2 e - m) v_j / l,  l = sum_j 2^(...)
//
// over the keys j that a row sees: the whole context, and the drafted key u when
// bit u of the row's mask word is set.
//
// What bounds it is reading the cache once: a KV head's T * (Hq / Hkv) rows share
// each key, so there are few operations per byte, and everything here serves to
// keep loads in flight.  8 KV heads of 128, calls in a row at full clocks: one token
// over 262,144 positions takes 99 us in 8 bits (5.5 TB/s of the measured 6.55) and
// 171 us in 16 (6.3 TB/s), 64 rows over 131,072 in 16 bits 94 us and in 8 bits 108;
// the smallest calls 9 to 11 us, one-off steps.
//  * The products run transposed on the tensor cores, S^T = K Q^T and O^T =
//    V^T P: the 128 keys of a tile (then the d elements of a value) are the 128
//    rows of the instruction, and the query rows are its N = 16 .. 64 columns,
//    so that one row costs 16 columns, not 128.  K and V tiles are used as TMA
//    lays them down, in either element type.
//  * A softmax thread owns a key: it sees the key's scores with every row, so a
//    per-key scale is a thread's scalar, sums over keys stay in its registers
//    until the end, and no maximum crosses lanes while the reference m holds.
//    m is any value near the row's maximum: it is taken from the first tile and
//    moves (with a rescaling of O^T and l) only when a score is 16 above it, in
//    powers of two.  The weights are formed before that is known, and once more
//    in the rare tile where it happens.
//  * 8-bit keys and values enter the 8-bit product as they are.  The query row is
//    brought to [128, 256) by a power of two and split into two e4m3 parts, which
//    hold bf16's 8 bits (fewer of elements below 2^-9 of the row's largest); the
//    weight (times the value's power of two) into three e5m2 parts, 9 bits, down to
//    2^-29 of the row's largest: each part is kept 2^4 larger than the one before,
//    or their common lowest step would end that at 2^-21.
//  * The work is cut evenly over the blocks, one per SM.  Few sequences (at most
//    one per block, counted with their KV heads) are each cut into pieces, so that
//    no block pays for two sequences' beginning and end.  Many form one list of
//    tiles, cut into equal runs, so that a ragged batch loads every block alike.
//    What covers part of a sequence leaves its sums in the workspace, and a second
//    kernel, launched ahead of time, joins them in order.
// More than 64 rows of a KV head are tree_wide.cu's.
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "tree_attn.cuh"

namespace minf {

namespace {

// --------------------------------------------------------------------- layout
template <int D, bool F8, int NR>
struct Cfg {
  // softmax warpgroups, on alternate tiles: four where TMEM and registers allow
  // (one tile's chain of waits is longer than its loads), two otherwise
  static constexpr int kWG = NR == 16 || (NR == 32 && !F8) ? 4 : 2;
  static constexpr int kSoft = 128 * kWG;
  static constexpr int kThreads = kSoft + 96;         // and the issuer, the K and the V producer
  static constexpr int kRowB = D * (F8 ? 1 : 2);       // bytes of a cached row
  static constexpr int kPitch = kRowB < 128 ? kRowB : 128;  // row pitch within a swizzled region
  static constexpr int kRegions = kRowB / kPitch;
  static constexpr int kRegion = 128 * kPitch;
  static constexpr int kTileB = 128 * kRowB;
  static constexpr int kQParts = F8 ? 2 : 1, kPParts = F8 ? 3 : 1;
  static constexpr int kQPart = NR * kRowB;
  static constexpr int kPPart = NR * 128 * (F8 ? 1 : 2);
  static constexpr int kQB = kQParts * kQPart;
  static constexpr int kPB = kPParts * kPPart;         // of one warpgroup
  static constexpr int kMiscMax = kWG * NR * 4 + NR * 4 + (F8 ? NR * 4 : 0) + NR * 8 + 512;
  static constexpr int kExpB = F8 ? 256 : 0;           // a tile's key and value exponents
  static constexpr int kTiles = (232448 - kQB - kWG * kPB - kMiscMax - 8 * kExpB) / kTileB;
  static constexpr int kKStages = (kTiles + 1) / 2 < 8 ? (kTiles + 1) / 2 : 8;
  static constexpr int kVStages = kTiles / 2 < 8 ? kTiles / 2 : 8;
  static constexpr int kOffV = 0;                      // the rings first: a 64-element V tile is read
  static constexpr int kOffK = kOffV + kVStages * kTileB;  // past its end by the unused 64 output rows
  static constexpr int kOffQ = kOffK + kKStages * kTileB;
  static constexpr int kOffP = kOffQ + kQB;
  static constexpr int kOffExp = kOffP + kWG * kPB;
  static constexpr int kOffRef = kOffExp + kKStages * kExpB;  // [kWG][NR] references
  static constexpr int kOffRow = kOffRef + kWG * NR * 4;      // [NR] row of the KV head's [group, T] queries
  static constexpr int kOffFac = kOffRow + NR * 4;            // [NR] row factors (8-bit)
  static constexpr int kOffWords = kOffFac + (F8 ? NR * 4 : 0);  // [NR] mask words
  static constexpr int kOffBars = kOffWords + NR * 8;
  // k_full, k_empty, v_full, v_empty, s_full, p_full, pv_done [kWG], q_full, mma_done
  static constexpr int kNumBars = 2 * kKStages + 2 * kVStages + 3 * kWG + 2;
  static constexpr int kOffMisc = kOffBars + kNumBars * 8;    // TMEM slot, abort, the run
  static constexpr int kSmem = kOffMisc + 48;
  static constexpr uint32_t kSwizzle = kPitch == 128 ? 2u : 4u;
  static constexpr uint32_t kGroup8 = 8 * kPitch;             // eight rows of a region
  // The 8-bit parts of a query (of a weight) lie side by side as more columns of
  // one product while TMEM has room for them, and are added when read; they
  // accumulate in turn otherwise.  A product of few columns costs its issue
  // (about 100 cycles), not its columns.
  static constexpr int kQStack = F8 && NR <= 32 ? 2 : 1, kPStack = F8 && NR <= 64 ? 3 : 1;
  static constexpr int kSCols = kQStack * NR, kOCols = kPStack * NR;  // of a warpgroup
  static constexpr int kOffO = kWG * kSCols;                          // first column of O
  static constexpr int kTmem = kWG * (kSCols + kOCols) <= 128 ? 128 : kWG * (kSCols + kOCols) <= 256 ? 256 : 512;
  static constexpr uint32_t kIdescS = F8 ? idesc_f8(128, kSCols, 0, 0, 0, 0) : idesc_bf16(128, NR, 0, 0);
  static constexpr uint32_t kIdescO = F8 ? idesc_f8(128, kOCols, 0, 1, 1, 1) : idesc_bf16(128, NR, 1, 1);
  static constexpr int kCh = NR == 64 ? 32 : 16;              // columns a thread takes at once
  // the weights' references lie kOff below the maximum seen, so that 8-bit parts
  // use the top of their range; a score kTop above the reference moves it (kOff 8
  // moves it more often: 64 rows over 128K 8-bit positions 114 us, 107 with 4)
  static constexpr float kOff = F8 ? 4.f : 0.f, kTop = F8 ? 15.f : 16.f;
  static constexpr float kPartScale = F8 ? 0.0625f : 1.f;  // of each 8-bit part beside the one before
  static_assert(kVStages >= 2 && kKStages >= 2, "rings");
  // a softmax warpgroup that reads exponents is less than a round of the ring ahead
  static_assert(!F8 || kKStages >= kWG, "rounds that a wait can tell apart");
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(24 * NR <= kPB && 4 * kWG * NR <= kQB, "scratch in the idle P and Q buffers");
  static_assert(NR * D * 2 <= kWG * kPB && kWG * (kSCols + kOCols) <= kTmem, "the queries as they are in the idle P buffers");
};

// Sums each of N values (16 or 32) over the warp's lanes; lane i ends with the
// total of value i (of value i / 2 when N is 16).
template <int N>
__device__ __forceinline__ float lane_totals(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  int n = N;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < N / 2; ++i)
        if (i < n) {
          const float mine = up ? v[i + n] : v[i], other = up ? v[i] : v[i + n];
          v[i] = mine + __shfl_xor_sync(0xFFFFFFFFu, other, o);
        }
    } else {
      v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
    }
  }
  return v[0];
}

// What a sum was before x joined it; nothing when the two overflowed.
__device__ __forceinline__ float without(float sum, float x) { return sum == INFINITY ? 0.f : sum - x; }

template <int D, bool F8, int NR>
__global__ void __launch_bounds__(Cfg<D, F8, NR>::kThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const TreeParams p) {
  using C = Cfg<D, F8, NR>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part_lane = blockIdx.x / p.groups, rg = blockIdx.x % p.groups;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kOffBars);
  uint64_t* k_empty = k_full + C::kKStages;
  uint64_t* v_full = k_empty + C::kKStages;
  uint64_t* v_empty = v_full + C::kVStages;
  uint64_t* s_full = v_empty + C::kVStages;
  uint64_t* p_full = s_full + C::kWG;
  uint64_t* pv_done = p_full + C::kWG;
  uint64_t* q_full = pv_done + C::kWG;
  constexpr int kIssuer = 4 * C::kWG, kLoadK = kIssuer + 1, kLoadV = kIssuer + 2;  // warps
  uint64_t* mma_done = q_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  Walk* start = reinterpret_cast<Walk*>(smem + C::kOffP);  // until the roles have copied it

  if ((smem_u32(smem) & 1023u) != 0u) {
    if (threadIdx.x == 0) report(p.status, MINF_ERR_DEVICE_BOUNDS, 112);
    return;
  }
  if (warp == kIssuer) {
    tmem_alloc(tmem_slot, C::kTmem);
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
      for (int w = 0; w < C::kWG; ++w) {
        mbar_init(&s_full[w], 1);
        mbar_init(&p_full[w], 128);
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
  wait_prerequisite();  // nothing of global memory is read before this
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
  __syncthreads();  // the run's place is the P buffer

  if (warp == kLoadK || warp == kLoadV) {
    // ----------------------------------------------------------- producers
    const bool is_k = warp == kLoadK;
    load_tiles<C, F8, NR>(p, is_k ? tmK : tmV, is_k, smem, is_k ? k_full : v_full, is_k ? k_empty : v_empty, rg, w, abort);
  } else if (warp == kIssuer) {
    // --------------------------------------------------------- MMA issuer
    // operand descriptors: a base per buffer, plus constants (the start-address
    // field holds address / 16 and never carries out)
    const uint64_t q0 = sdesc(smem_u32(smem + C::kOffQ), C::kSCols * 16, 128, 0);
    const uint64_t p0 = sdesc(smem_u32(smem + C::kOffP), 128, 2048, 0);
    const uint64_t k0 = sdesc(smem_u32(smem + C::kOffK), 16, C::kGroup8, C::kSwizzle);
    const uint64_t v0 = sdesc(smem_u32(smem + C::kOffV), C::kRegion, C::kGroup8, C::kSwizzle);
    auto ready = [&](uint64_t* bar, int parity) { return (bool)__all_sync(0xFFFFFFFFu, mbar_poll(bar, parity)); };
    int it0 = 0, segs = 0;
    while (!__any_sync(0xFFFFFFFFu, *abort) && w.next(p)) {
      if (rg * NR >= w.nd * p.group) continue;
      mbar_wait_or_abort(q_full, segs & 1, abort, p.status, 119);
      ++segs;
      // Of the segment's n tiles, s have their scores issued, pd their weights
      // formed and pv their values' product issued.  Whatever is ready goes next,
      // scores first, so that no warpgroup waits behind another's product.
      const int n = w.t1 - w.t0;
      int s = 0, pd = 0, pv = 0, idle = 0;
      unsigned long long since = 0;
      while (pv < n) {
        bool moved = false;
        if (pd < s && ready(&p_full[(it0 + pd) % C::kWG], (it0 + pd) / C::kWG & 1)) {
          ++pd;
          tc_fence_after();
          moved = true;
        }
        const int is = it0 + s, ks = is % C::kKStages, iv = it0 + pv, vs = iv % C::kVStages;
        if (s < n && s - pd < C::kWG && ready(&k_full[ks], is / C::kKStages & 1)) {
          // the scores' buffer is that of tile s - kWG, whose weights are formed
          const int wg = is % C::kWG;
          const uint64_t k = k0 + (uint32_t)(ks * (C::kTileB / 16));
          if (elect_lane()) {
#pragma unroll
            for (int part = 0; part < C::kQParts / C::kQStack; ++part)
#pragma unroll
              for (int kk = 0; kk < C::kRowB / 32; ++kk) {
                const uint64_t a = k + (uint32_t)(((kk * 32 / C::kPitch) * C::kRegion + (kk * 32) % C::kPitch) / 16);
                const uint64_t b = q0 + (uint32_t)((part * C::kQPart + kk * 2 * C::kSCols * 16) / 16);
                const uint32_t acc = part > 0 || kk > 0;
                if constexpr (F8) umma_ss_f8(tmem + wg * C::kSCols, a, b, C::kIdescS, acc);
                else umma_ss(tmem + wg * C::kSCols, a, b, C::kIdescS, acc);
              }
            umma_commit(&s_full[wg]);
            umma_commit(&k_empty[ks]);
          }
          __syncwarp();
          ++s;
          moved = true;
        } else if (pv < pd && ready(&v_full[vs], iv / C::kVStages & 1)) {
          // O^T of the tile's warpgroup (+)= V^T P
          const int wg = iv % C::kWG;
          const uint64_t v = v0 + (uint32_t)(vs * (C::kTileB / 16)), pb = p0 + (uint32_t)(wg * (C::kPB / 16));
          const uint32_t d = tmem + C::kOffO + wg * C::kOCols;
          if (elect_lane()) {
#pragma unroll
            for (int part = 0; part < C::kPParts / C::kPStack; ++part)
#pragma unroll
              for (int kk = 0; kk < (F8 ? 4 : 8); ++kk) {
                constexpr int kKeys = F8 ? 32 : 16;
                const uint64_t a = v + (uint32_t)(kk * kKeys * C::kPitch / 16);
                const uint64_t b = pb + (uint32_t)((part * C::kPPart + kk * kKeys * 16) / 16);
                const uint32_t acc = part > 0 || kk > 0 || pv >= C::kWG;
                if constexpr (F8) umma_ss_f8(d, a, b, C::kIdescO, acc);
                else umma_ss(d, a, b, C::kIdescO, acc);
              }
            umma_commit(&v_empty[vs]);
            umma_commit(&pv_done[wg]);
          }
          __syncwarp();
          ++pv;
          moved = true;
        }
        if (moved) {
          idle = 0;
        } else if ((++idle & 63) == 0) {  // bounded, as every wait
          if (idle == 64) since = globaltimer();
          if (!*abort && globaltimer() - since > kWaitLimitNs) {
            *abort = 1;
            report(p.status, MINF_ERR_DEVICE_TIMEOUT, 117);
          }
          if (__any_sync(0xFFFFFFFFu, *abort)) break;
        }
      }
      it0 += n;
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
    const int wg = warp >> 2, tid = threadIdx.x & 127;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_col = lanes + wg * C::kSCols, o_col = lanes + C::kOffO + wg * C::kOCols;
    // the references, negated: [kWG][NR]
    float* nref_all = reinterpret_cast<float*>(smem + C::kOffRef);
    float* nref = nref_all + wg * NR;
    float* fac = reinterpret_cast<float*>(smem + C::kOffFac);
    int* row_at = reinterpret_cast<int*>(smem + C::kOffRow);
    unsigned long long* words = reinterpret_cast<unsigned long long*>(smem + C::kOffWords);
    const uint32_t* words32 = reinterpret_cast<const uint32_t*>(words);
    uint8_t* pbuf = smem + C::kOffP + wg * C::kPB;
    float* wmax = reinterpret_cast<float*>(pbuf);             // [4][NR] while P is idle
    float* shrink = wmax + 4 * NR;                            // [NR]
    float* nwas = shrink + NR;                                // [NR]
    float* lsum = reinterpret_cast<float*>(pbuf);             // [4][NR] after the segment's last tile
    float* weight = reinterpret_cast<float*>(smem + C::kOffQ);  // [kWG][NR] while Q is idle
    const int bar_wg = 1 + wg, bar_all = 1 + C::kWG;
    int it = 0, uses = 0;  // tiles of the block so far, and those of this warpgroup
    while (w.next(p)) {
      const int rows = min(NR, w.nd * p.group - rg * NR);
      if (rows <= 0) continue;
      const int len = w.ctx + w.nd, n = w.t1 - w.t0;
      const long long qb = ((long long)w.b * p.Hq + w.h * p.group) * p.T;  // first query row of the KV head
      // ---- the segment's queries, as the B operand; their mask words
      {
        // 16-byte pieces, each thread's all of one row: bf16 queries go where the
        // product reads them, 8-bit ones are staged in the P buffer (rows of D) and
        // split below
        constexpr int kStep = C::kSoft / NR, kPieces = (D / 8 + kStep - 1) / kStep;
        const int r = threadIdx.x % NR, c0 = threadIdx.x / NR;
        const int t = (unsigned)(rg * NR + r) / (unsigned)p.group, at = (rg * NR + r - t * p.group) * p.T + t;
        uint4 x[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int c = c0 + i * kStep;
          x[i] = make_uint4(0, 0, 0, 0);
          if (c < D / 8 && r < rows) x[i] = load(reinterpret_cast<const uint4*>(p.q + (qb + at) * D) + c);
        }
        if (c0 == 0) {
          unsigned long long m = 0;
          if (r < rows) {
            m = p.mask ? p.mask[(long long)w.b * p.T + t] : (2ull << t) - 1;
            if (w.nd < 64) m &= (1ull << w.nd) - 1;
          }
          row_at[r] = at;
          words[r] = m;
#pragma unroll
          for (int v = 0; v < C::kWG; ++v) nref_all[v * NR + r] = INFINITY;
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int c = c0 + i * kStep;
          if (c < D / 8)
            *reinterpret_cast<uint4*>(smem + (F8 ? C::kOffP + r * D * 2 + c * 16 : C::kOffQ + c * NR * 16 + r * 16)) = x[i];
        }
      }
      if constexpr (F8) {
        named_bar_sync(bar_all, C::kSoft);
        constexpr int E = D / 32;
#pragma unroll 1
        for (int r = warp; r < NR; r += 4 * C::kWG) {
          float x[E];
          float top = 0.f;
          bool bad = false;
          const __nv_bfloat162* q2 = reinterpret_cast<const __nv_bfloat162*>(smem + C::kOffP + r * D * 2) + lane * (E / 2);
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const float2 f = __bfloat1622float2(q2[e / 2]);
            x[e] = f.x;
            x[e + 1] = f.y;
            bad = bad || !(fabsf(f.x) <= 3.4e38f) || !(fabsf(f.y) <= 3.4e38f);
            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
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
            const float2 back = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi, __NV_E4M3)));
            const uint32_t lo =
                __nv_cvt_float2_to_fp8x2(make_float2(a.x - back.x, a.y - back.y), __NV_SATFINITE, __NV_E4M3);
            const int byte = lane * E + e;
            uint8_t* q = smem + C::kOffQ + (byte / 16) * C::kSCols * 16 + r * 16 + byte % 16;
            *reinterpret_cast<uint16_t*>(q) = (uint16_t)hi;
            *reinterpret_cast<uint16_t*>(q + (C::kQStack > 1 ? NR * 16 : C::kQPart)) = (uint16_t)lo;
          }
          if (lane == 0) fac[r] = bad ? NAN : p.scale_log2 * __uint_as_float((uint32_t)(127 - up) << 23);
        }
      }
      fence_proxy_async();
      mbar_arrive(q_full);
      named_bar_sync(bar_all, C::kSoft);

      uint64_t l[NR / 2];  // this key lane's sums of two rows each
#pragma unroll
      for (int r = 0; r < NR / 2; ++r) l[r] = 0ull;
      bool first = true;
#pragma unroll 1
      for (int i = 0; i < n; ++i, ++it) {
        if (it % C::kWG != wg) continue;
        const int j0 = (w.t0 + i) * 128, j = j0 + tid, u = j - w.ctx;
        const bool in = j < len;
        const int kst = it % C::kKStages;
        // the thread's row of the tile's values, once they have landed
        auto value_row = [&] {
          // A wait tells only odd rounds of the ring from even ones, so the stage's
          // former tile has to be known to have landed: by its product when there are
          // fewer stages than warpgroups (this tile's load waits for that as well), by
          // that of this warpgroup's tile before, which is no earlier, otherwise.
          const int st = it % C::kVStages, was = it - (C::kVStages < C::kWG ? C::kVStages : C::kWG);
          if (was >= 0) mbar_wait_or_abort(&pv_done[was % C::kWG], (was / C::kWG) & 1, abort, p.status, 126);
          mbar_wait_or_abort(&v_full[st], (it / C::kVStages) & 1, abort, p.status, 126);
          return smem + C::kOffV + st * C::kTileB + tid * C::kPitch;
        };
        float km = 0.f, lv = 0.f, inv = 1.f;  // 2^key exponent, value exponent, its inverse power
        bool zeros = false;  // whether a row of the warp's keys may be of zeros
        if constexpr (F8) {
          mbar_wait_or_abort(&k_full[kst], (it / C::kKStages) & 1, abort, p.status, 122);
          const uint8_t* e = smem + C::kOffExp + kst * C::kExpB + tid;
          const uint32_t ke = e[0], ve = max((uint32_t)e[128], kLeastExp);
          __syncwarp();
          if (lane == 0) mbar_arrive(&k_empty[kst]);
          if (in) {
            km = ke == 255u ? NAN : __uint_as_float(ke << 23);
            lv = ve == 255u ? NAN : (float)((int)ve - 127);
            inv = ve == 255u ? NAN : __uint_as_float((254u - ve) << 23);
          }
          zeros = __any_sync(0xFFFFFFFFu, in && ve == kZeroExp);
        }
        mbar_wait_or_abort(&s_full[wg], uses & 1, abort, p.status, 123);
        tc_fence_after();
        if (zeros) {
          // A row of zeros adds nothing to O, so it must not raise the reference, as
          // the power 2^0 that it is stored with would
          if (in && lv == (float)((int)kZeroExp - 127) && zero_row<C::kPitch>(value_row())) {
            lv = (float)((int)kLeastExp - 127);
            inv = __uint_as_float((254u - kLeastExp) << 23);
          }
          __syncwarp();
        }
        // scores of rows c0 .. of the thread's key: asked for, and taken
        auto ask = [&](int c0, auto& s, auto& lo) {
          tmem_ld(s_col + c0, s);
          if constexpr (C::kQStack > 1) tmem_ld(s_col + NR + c0, lo);
        };
        auto take = [&](auto& s, auto& lo) {
          tmem_landed(s);
          if constexpr (C::kQStack > 1) {
            tmem_landed(lo);
#pragma unroll
            for (int c = 0; c < (int)(sizeof(s) / 4); ++c)
              s[c] = __float_as_uint(__uint_as_float(s[c]) + __uint_as_float(lo[c]));
          }
        };
        // From the tile's scores s to the exponents of their weights, two rows at a
        // time: s scale log2(e) + lv - reference, -infinity where the row does not
        // see the key.
        auto exponent2 = [&](auto masked, uint32_t s0, uint32_t s1, int r, const float* minus, float& t0, float& t1) {
          const uint64_t s2 = f32x2_pack(__uint_as_float(s0), __uint_as_float(s1));
          const float2 m = minus ? *reinterpret_cast<const float2*>(minus + r) : make_float2(0.f, 0.f);
          if constexpr (F8) {
            const float2 f = *reinterpret_cast<const float2*>(fac + r);
            f32x2_unpack(f32x2_fma(f32x2_mul(s2, f32x2_pack(km, km)), f32x2_pack(f.x, f.y),
                                   f32x2_add(f32x2_pack(lv, lv), f32x2_pack(m.x, m.y))),
                         t0, t1);
          } else {
            f32x2_unpack(f32x2_fma(s2, f32x2_pack(p.scale_log2, p.scale_log2), f32x2_pack(m.x, m.y)), t0, t1);
          }
          if constexpr (decltype(masked)::value) {
            const int wd = u >> 5 & 1, bit = u & 31;
            t0 = in && (u < 0 || (words32[2 * r + wd] >> bit & 1)) ? t0 : -INFINITY;
            t1 = in && (u < 0 || (words32[2 * r + 2 + wd] >> bit & 1)) ? t1 : -INFINITY;
          }
        };
        auto tile = [&](auto masked) {
          bool move = first;
          // (16-bit rows beyond 16: the registers of this way in cost every tile more
          // than it gains, 102 against 94 us for 64 rows over 128K)
          constexpr bool kQuick = F8 || NR == 16;
          const bool quick = kQuick && first && j0 < w.ctx;
#pragma unroll 1
          for (int pass = 0; pass < 2; ++pass) {
            if (quick && pass == 0) {
              // A segment's first tile: a reference near the rows' maxima will do, the
              // largest of one warp's 32 keys.  Each warp gives a quarter of the rows
              // theirs; in a tile with drafted keys the first warp, which has keys of
              // the context, gives all of them.
              constexpr int kQ = NR / 4, kLd = kQ < 8 ? kQ : 8;
              const bool all = decltype(masked)::value;
              const int ra = all ? 0 : (warp & 3) * kQ, rz = !all ? ra + kQ : (warp & 3) == 0 ? NR : 0;
#pragma unroll 1
              for (int c0 = ra; c0 < rz; c0 += kLd) {
                uint32_t s[kLd], lo[kLd];
                ask(c0, s, lo);
                take(s, lo);
#pragma unroll
                for (int c = 0; c < kLd; c += 2) {
                  float t0, t1;
                  exponent2(masked, s[c], s[c + 1], c0 + c, nullptr, t0, t1);
                  t0 = -fmaxf(warp_max(t0) - C::kOff, kFloor);
                  t1 = -fmaxf(warp_max(t1) - C::kOff, kFloor);
                  if (lane == 0) *reinterpret_cast<float2*>(nref + c0 + c) = make_float2(t0, t1);
                }
              }
              named_bar_sync(bar_wg, 128);
            } else if (move) {
              // move the references up to the largest scores seen; O^T and l follow
              if (!first) {
                mbar_wait_or_abort(&pv_done[wg], (uses - 1) & 1, abort, p.status, 124);
                tc_fence_after();
                named_bar_sync(bar_wg, 128);
              }
              if (tid < NR) nwas[tid] = first ? 0.f : nref[tid];
              named_bar_sync(bar_wg, 128);
#pragma unroll 1
              for (int c0 = 0; c0 < NR; c0 += 8) {
                uint32_t s[8], lo[8];
                ask(c0, s, lo);
                take(s, lo);
                float mine = 0.f;
#pragma unroll
                for (int c = 0; c < 8; c += 2) {
                  float t0, t1;
                  exponent2(masked, s[c], s[c + 1], c0 + c, nwas, t0, t1);
                  t0 = warp_max(t0);
                  t1 = warp_max(t1);
                  if (lane == c) mine = t0;
                  if (lane == c + 1) mine = t1;
                }
                if (lane < 8) wmax[(warp & 3) * NR + c0 + lane] = mine;
              }
              named_bar_sync(bar_wg, 128);
              if (tid < NR) {
                // the largest, above the former reference (above 0 in the first tile)
                const float up = fmaxf(fmaxf(wmax[tid], wmax[NR + tid]), fmaxf(wmax[2 * NR + tid], wmax[3 * NR + tid])) -
                                 C::kOff;
                if (first) {
                  nref[tid] = -fmaxf(up, kFloor);
                } else {
                  const float now = fmaxf(-nwas[tid] + up, -nwas[tid]);
                  nref[tid] = -now;
                  shrink[tid] = fast_exp2(-nwas[tid] - now);
                }
              }
              named_bar_sync(bar_wg, 128);
              if (first) {
                if constexpr (kQuick) {  // the first pass's sums
#pragma unroll
                  for (int r = 0; r < NR / 2; ++r) l[r] = 0ull;
                }
              } else {
#pragma unroll 1
                for (int c0 = 0; c0 < C::kOCols; c0 += 8) {
                  uint32_t o[8];
                  tmem_ld(o_col + c0, o);
                  tmem_landed(o);
#pragma unroll
                  for (int c = 0; c < 8; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * shrink[c0 % NR + c]);
                  tmem_st(o_col + c0, o);
                }
                tmem_wait_st();
                // l without the weights that the first pass added: they are formed
                // again.  Both are still sums of 2^s in the former reference, so the
                // difference is off by a rounding of what is formed again at most.
                // Where they overflow, the weight is above 2^127, and what was there
                // before it, weights up to 2^15 times 2^80 each, does not count.
#pragma unroll
                for (int c0 = 0; c0 < NR; c0 += 16) {
                  uint32_t s[16], lo[16];
                  ask(c0, s, lo);
                  take(s, lo);
#pragma unroll
                  for (int c = 0; c < 16; c += 2) {
                    const int r = c0 + c;
                    float t0, t1, l0, l1;
                    exponent2(masked, s[c], s[c + 1], r, nwas, t0, t1);
                    f32x2_unpack(l[r / 2], l0, l1);
                    l0 = without(l0, fast_exp2(t0) * inv) * shrink[r];
                    l1 = without(l1, fast_exp2(t1) * inv) * shrink[r + 1];
                    l[r / 2] = f32x2_pack(l0, l1);
                    asm volatile("" ::: "memory");  // one pair's factors at a time (8-bit, 64 rows: 384 bytes spilled without)
                  }
                }
              }
              named_bar_sync(bar_wg, 128);  // the scratch is the P buffer
            }
            // the weights, to shared memory as the B operand: [NR / 16 bytes][128 keys][16 bytes]
            if (!first && pass == 0) mbar_wait_or_abort(&pv_done[wg], (uses - 1) & 1, abort, p.status, 125);  // P is free
            float top = -INFINITY;
#pragma unroll
            for (int c0 = 0; c0 < NR; c0 += C::kCh) {
              uint32_t s[C::kCh], lo[C::kCh];
              ask(c0, s, lo);
              take(s, lo);
              constexpr int kStep = F8 ? 16 : 8;
#pragma unroll
              for (int g = 0; g < C::kCh; g += kStep) {
                uint32_t out[C::kPParts][4];
#pragma unroll
                for (int c = 0; c < kStep; c += 4) {
                  uint32_t h[2];  // four weights as pairs of bf16, or of half
#pragma unroll
                  for (int x = 0; x < 2; ++x) {
                    const int r = c0 + g + c + 2 * x;
                    float t0, t1;
                    exponent2(masked, s[g + c + 2 * x], s[g + c + 2 * x + 1], r, nref, t0, t1);
                    top = fmaxf(top, fmaxf(t0, t1));
                    const float p0 = fast_exp2(t0), p1 = fast_exp2(t1);
                    if constexpr (F8) {
                      l[r / 2] = f32x2_fma(f32x2_pack(p0, p1), f32x2_pack(inv, inv), l[r / 2]);
                      const __half2 two = __floats2half2_rn(p0, p1);
                      h[x] = *reinterpret_cast<const uint32_t*>(&two);
                    } else {
                      l[r / 2] = f32x2_add(l[r / 2], f32x2_pack(p0, p1));
                      h[x] = pack_bf16x2(p0, p1);
                    }
                  }
                  if constexpr (F8) {
                    // e5m2 is the upper byte of a half: each part is the remainder
                    // rounded there (half a step up, in magnitude), and leaves an
                    // exact remainder, of which 16 times is the next part, so that
                    // the last reaches down to a half's lowest step (no part is
                    // above 2^15: a remainder is at most an eighth).  A NaN weight
                    // may be lost here, not in l.
                    const __half2 up = __float2half2_rn(1.f / C::kPartScale);
#pragma unroll
                    for (int q = 0; q < 3; ++q) {
                      const uint32_t a = h[0] + 0x00800080u, b = h[1] + 0x00800080u;
                      out[q][c / 4] = __byte_perm(a, b, 0x7531);
                      const uint32_t ta = a & 0xff00ff00u, tb = b & 0xff00ff00u;
                      const __half2 ra = __hmul2(up, __hsub2(*reinterpret_cast<const __half2*>(&h[0]), *reinterpret_cast<const __half2*>(&ta)));
                      const __half2 rb = __hmul2(up, __hsub2(*reinterpret_cast<const __half2*>(&h[1]), *reinterpret_cast<const __half2*>(&tb)));
                      h[0] = *reinterpret_cast<const uint32_t*>(&ra);
                      h[1] = *reinterpret_cast<const uint32_t*>(&rb);
                    }
                  } else {
                    out[0][c / 2] = h[0];
                    out[0][c / 2 + 1] = h[1];
                  }
                }
#pragma unroll
                for (int q = 0; q < C::kPParts; ++q)
                  *reinterpret_cast<uint4*>(pbuf + q * C::kPPart + (c0 + g) / kStep * 2048 + tid * 16) =
                      make_uint4(out[q][0], out[q][1], out[q][2], out[q][3]);
              }
            }
            // a first tile's references from all of its keys are the largest scores
            if ((first && !quick) || pass == 1 || bar_and(bar_wg, 128, !(top > C::kTop))) break;
            move = true;
          }
          if (decltype(masked)::value && !in) {
            // what lies behind the sequence's end may be anything: zero weight
            // needs a finite value
            uint8_t* v = value_row();
#pragma unroll
            for (int x = 0; x < C::kRegions; ++x)
#pragma unroll
              for (int o = 0; o < C::kPitch; o += 16)
                *reinterpret_cast<uint4*>(v + x * C::kRegion + o) = make_uint4(0, 0, 0, 0);
          }
        };
        if (j0 + 128 > w.ctx) tile(std::true_type{});
        else tile(std::false_type{});
        first = false;
        fence_proxy_async();
        tc_fence_before();
        mbar_arrive(&p_full[wg]);
        ++uses;
      }

      // ---- the segment's end: sums over the keys, the two warpgroups joined
      if (!first) {
        mbar_wait_or_abort(&pv_done[wg], (uses - 1) & 1, abort, p.status, 127);
        constexpr int kSum = NR < 32 ? 16 : 32;
#pragma unroll
        for (int c0 = 0; c0 < NR; c0 += kSum) {
          float v[kSum];
#pragma unroll
          for (int c = 0; c < kSum; c += 2) f32x2_unpack(l[(c0 + c) / 2], v[c], v[c + 1]);
          const float t = lane_totals<kSum>(v);
          if (kSum == 32 || (lane & 1) == 0) lsum[(warp & 3) * NR + c0 + (kSum == 32 ? lane : lane / 2)] = t;
        }
      }
      tc_fence_before();
      named_bar_sync(bar_all, C::kSoft);
      tc_fence_after();
      // whether warpgroup v had a tile of this segment
      auto has = [&](int v) { return n >= C::kWG || (v - (it - n) % C::kWG + C::kWG) % C::kWG < n; };
      const bool whole = w.t0 == 0 && w.t1 == w.nt;  // all of the sequence's tiles
      // a partial segment's sums go to the block's first or second place
      float* part = p.part + (2ll * blockIdx.x + (w.t0 == 0 ? 1 : 0)) * NR * (D + 2);
      for (int r = threadIdx.x; r < rows; r += C::kSoft) {
        float f[C::kWG], M = -INFINITY, L = 0.f;
#pragma unroll
        for (int v = 0; v < C::kWG; ++v) {
          f[v] = has(v) ? -nref_all[v * NR + r] : -INFINITY;
          M = fmaxf(M, f[v]);
        }
#pragma unroll
        for (int v = 0; v < C::kWG; ++v) {
          f[v] = has(v) ? fast_exp2(f[v] - M) : 0.f;
          const float* x = reinterpret_cast<const float*>(smem + C::kOffP + v * C::kPB) + r;
          if (has(v)) L += ((x[0] + x[NR]) + (x[2 * NR] + x[3 * NR])) * f[v];
        }
        if (whole) {
          const float by = L == 0.f ? 0.f : 1.f / L;  // a row that saw nothing: 0, -infinity
#pragma unroll
          for (int v = 0; v < C::kWG; ++v) f[v] *= by;
          if (p.lse) p.lse[qb + row_at[r]] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
        } else {
          part[r * (D + 2) + D] = M;
          part[r * (D + 2) + D + 1] = L;
        }
#pragma unroll
        for (int v = 0; v < C::kWG; ++v) weight[v * NR + r] = f[v];
      }
      named_bar_sync(bar_all, C::kSoft);
      // lane = element of the value; the warpgroups take turns at eight rows
#pragma unroll 1
      for (int c0 = wg * 8; c0 < rows; c0 += C::kWG * 8) {
        float x[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] = 0.f;
#pragma unroll
        for (int v = 0; v < C::kWG; ++v) {
          if (!has(v)) continue;  // its O^T is not of this segment
#pragma unroll
          for (int q = 0; q < C::kPStack; ++q) {
            const float scale = q == 0 ? 1.f : q == 1 ? C::kPartScale : C::kPartScale * C::kPartScale;
            uint32_t o[8];
            tmem_ld(lanes + C::kOffO + v * C::kOCols + q * NR + c0, o);
            tmem_landed(o);
#pragma unroll
            for (int c = 0; c < 8; ++c) x[c] = fmaf(__uint_as_float(o[c]) * scale, weight[v * NR + c0 + c], x[c]);
          }
        }
        if (tid < D) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const int r = c0 + c;
            if (r >= rows) break;
            if (whole) p.o[(qb + row_at[r]) * D + tid] = __float2bfloat16(x[c]);
            else part[r * (D + 2) + tid] = x[c];
          }
        }
      }
      tc_fence_before();
      named_bar_sync(bar_all, C::kSoft);  // Q, P and the references are the next segment's
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// Joins the parts of the segments that several blocks shared: one block per row,
// in 256 / D groups of threads that take every so manieth part, then added in
// order.
template <int D>
__global__ void __launch_bounds__(256) tree_join_kernel(const TreeParams p, int nr) {
  constexpr int G = 256 / D;
  __shared__ float wt[kMaxBlocks], acc[G][D], red[8];
  const int bh = blockIdx.y, b = bh / p.c.Hkv, h = bh % p.c.Hkv;
  const int rg = blockIdx.x / nr, r = blockIdx.x % nr;  // nr rows of each row group
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  launch_dependents();
  int ctx;
  const int nd = new_tokens(p, b, ctx), nt = tiles(ctx, nd);
  int c0 = 0;
  const int d0 = lane < p.B ? new_tokens(p, lane, c0) : 0;
  const Cut cut = make_cut(p, c0, d0);
  int before = 0;  // units of the sequences before b
  for (int i = lane; i < b; i += 32) before += cut.units(tiles_of(p, i));
  before = __reduce_add_sync(0xFFFFFFFFu, before) * p.c.Hkv;
  // the segment's first block and their number
  const int units = cut.units(nt), s0 = before + h * units;
  const int first = cut.pieces ? s0 : s0 / cut.per;
  const int n = cut.pieces ? units : nt > 0 ? (s0 + nt - 1) / cut.per - first + 1 : 0;
  wait_prerequisite();  // every block: the launches that follow rely on this one being over last
  if (rg * nr + r >= nd * p.group || n <= 1) return;
  auto part_of = [&](int i) {
    const long long slot = 2ll * ((first + i) * p.groups + rg) + (i == 0 ? 1 : 0);
    return p.part + (slot * p.rows + r) * (D + 2);
  };
  // the first parts' sums are on their way while the weights are formed
  constexpr int kAhead = 8;
  const int g = threadIdx.x / D, e = threadIdx.x % D;
  float x[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) x[i] = g + i * G < n ? part_of(g + i * G)[e] : 0.f;
  float m = -INFINITY, l = 0.f;
  if (threadIdx.x < n) {
    m = part_of(threadIdx.x)[D];
    l = part_of(threadIdx.x)[D + 1];
  }
  const float wm = warp_max(m);
  if (lane == 0) red[warp] = wm;
  __syncthreads();
  float M = red[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) M = fmaxf(M, red[i]);
  const float f = threadIdx.x < n ? fast_exp2(m - M) : 0.f;
  if (threadIdx.x < n) wt[threadIdx.x] = f;
  float L = threadIdx.x < n ? l * f : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, o);
  __syncthreads();
  if (lane == 0) red[warp] = L;
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (g + i * G < n) a = fmaf(x[i], wt[g + i * G], a);
#pragma unroll 8
  for (int i = g + kAhead * G; i < n; i += G) a = fmaf(part_of(i)[e], wt[i], a);
  acc[g][e] = a;
  __syncthreads();
  if (g > 0) return;
#pragma unroll
  for (int i = 1; i < G; ++i) a += acc[i][e];
  L = red[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) L += red[i];
  const int t = (rg * nr + r) / p.group, hq = (rg * nr + r) % p.group;
  const long long row = ((long long)b * p.Hq + h * p.group + hq) * p.T + t;
  p.o[row * D + e] = __float2bfloat16(L == 0.f ? 0.f : a / L);
  if (e == 0 && p.lse) p.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

int rows_per_block(long long rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

template <int D, bool F8, int NR>
cudaError_t launch_rows(const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p, cudaStream_t stream) {
  using C = Cfg<D, F8, NR>;
  cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel<D, F8, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_early(tree_attn_kernel<D, F8, NR>, dim3(p.lanes * p.groups), C::kThreads, C::kSmem, stream, tk, tv, p);
}

template <int D, bool F8>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, TreeParams p, cudaStream_t stream) {
  const long long rows = (long long)p.T * p.group, bh = (long long)p.B * p.c.Hkv;
  const long long most = (((long long)p.c.max_pages << p.c.log_page) + 127) / 128 * bh;  // tiles
  p.rows = rows_per_block(rows);
  p.groups = (int)((rows + p.rows - 1) / p.rows);
  if (p.groups > kMaxBlocks || bh > 65535 || most >= (1ll << 30)) return cudaErrorInvalidConfiguration;
  p.lanes = (int)std::min<long long>(kMaxBlocks / p.groups, most);
  cudaError_t e = p.rows == 16   ? launch_rows<D, F8, 16>(tk, tv, p, stream)
                  : p.rows == 32 ? launch_rows<D, F8, 32>(tk, tv, p, stream)
                  : p.rows == 64 ? launch_rows<D, F8, 64>(tk, tv, p, stream)
                                 : tree_wide_launch(D, tk, tv, p, stream);
  if (e != cudaSuccess) return e;
  const int nr = (int)std::min<long long>(p.rows, rows);
  return launch_early(tree_join_kernel<D>, dim3((unsigned)(p.groups * nr), (unsigned)bh), 256, 0, stream, p, nr);
}

}  // namespace

size_t tree_part_floats(int Hq, int Hkv, int T, int d) {
  return 2ull * kMaxBlocks * rows_per_block((long long)T * (Hq / Hkv)) * (d + 2);
}
bool tree_rows_supported(int Hq, int Hkv, int T) {
  const long long rows = (long long)T * (Hq / Hkv);
  const int nr = rows_per_block(rows);
  return (rows + nr - 1) / nr <= kMaxBlocks;
}

cudaError_t tree_attn_launch(int d, const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p,
                             cudaStream_t stream) {
  if (d == 128) return p.c.ke ? launch<128, true>(tk, tv, p, stream) : launch<128, false>(tk, tv, p, stream);
  if (d == 64) return p.c.ke ? launch<64, true>(tk, tv, p, stream) : launch<64, false>(tk, tv, p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace minf
