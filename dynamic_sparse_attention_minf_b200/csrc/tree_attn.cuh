// What the cache attention kernels share: how the work is cut into the blocks'
// shares, and the warps that bring the cache's tiles in (tree_attn.cu has the
// overview).
#pragma once

#include "serve_device.cuh"
#include "serve_internal.h"

namespace minf {

constexpr int kMaxBlocks = 148;  // one block per SM
constexpr float kFloor = -1e30f; // reference of a row that has seen nothing
// Stored exponents of 8-bit values: of a row of zeros (and of rows with their
// largest in (224, 448]), and the least one.
constexpr uint32_t kZeroExp = 127, kLeastExp = 127 - 80;

// Whether the 8-bit values of a row in shared memory are all zeros.
template <int Bytes>
__device__ __forceinline__ bool zero_row(const uint8_t* row) {
  uint32_t any = 0;
#pragma unroll
  for (int o = 0; o < Bytes; o += 16) {
    const uint4 x = *reinterpret_cast<const uint4*>(row + o);
    any |= x.x | x.y | x.z | x.w;
  }
  return (any & 0x7f7f7f7fu) == 0;
}

__device__ __forceinline__ int new_tokens(const TreeParams& p, int b, int& ctx) {
  ctx = load(p.ctx + b);
  const int nd = p.ndraft ? load(p.ndraft + b) : p.T;
  const bool ok = ctx >= 0 && nd >= 0 && nd <= p.T && (long long)ctx + nd <= ((long long)p.c.max_pages << p.c.log_page);
  return ok ? nd : -1;
}
// 128-key tiles of one KV head of sequence b (0: no new tokens, or bad lengths)
__device__ __forceinline__ int tiles(int ctx, int nd) { return nd > 0 ? (ctx + nd + 127) >> 7 : 0; }
__device__ __forceinline__ int tiles_of(const TreeParams& p, int b) {
  int ctx;
  const int nd = new_tokens(p, b, ctx);
  return tiles(ctx, nd);
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (unsigned)(a + b - 1) / (unsigned)b; }

// How the work is cut, for a whole warp: in runs of `per` tiles of the list
// (sequence-major, then KV head, then tile), or, with at most one sequence and
// head per block, each of these into pieces of at most `per` tiles.  `units` of
// a sequence's head are its tiles or its pieces.
struct Cut {
  int per, total;  // total: tiles of the list
  bool pieces, bad;  // bad: a sequence has bad lengths (and counts as empty)
  __device__ __forceinline__ int units(int nt) const { return pieces ? ceil_div(nt, per) : nt; }
};
// ctx0, nd0: lengths of sequence `lane` (read by the caller; 0 without one)
__device__ __forceinline__ Cut make_cut(const TreeParams& p, int ctx0, int nd0) {
  const int lane = threadIdx.x & 31, n0 = tiles(ctx0, nd0);
  int total = n0, live = n0 > 0;
  bool bad = nd0 < 0;
  for (int b = lane + 32; b < p.B; b += 32) {
    int ctx;
    const int nd = new_tokens(p, b, ctx), n = tiles(ctx, nd);
    total += n;
    live += n > 0;
    bad = bad || nd < 0;
  }
  total = __reduce_add_sync(0xFFFFFFFFu, total) * p.c.Hkv;
  live = __reduce_add_sync(0xFFFFFFFFu, live) * p.c.Hkv;
  Cut c{max(1, ceil_div(total, p.lanes)), total, live <= p.lanes, (bool)__any_sync(0xFFFFFFFFu, bad)};
  while (c.pieces) {  // longer pieces, by a sixteenth at least, until there is a block for each
    int k = ceil_div(n0, c.per);
    for (int b = lane + 32; b < p.B; b += 32) k += ceil_div(tiles_of(p, b), c.per);
    k = __reduce_add_sync(0xFFFFFFFFu, k) * p.c.Hkv;
    if (k <= p.lanes) break;
    // per * k is at most the list's 2^30 tiles and one piece of 2^24 more for each of 148
    c.per = max(c.per + c.per / 16 + 1, (int)(((unsigned)c.per * (unsigned)k + p.lanes - 1) / (unsigned)p.lanes));
  }
  return c;
}

// A block's share, walked one (sequence, head) segment at a time; every role of
// the block walks it by itself.
struct Walk {
  int g, g1, base;     // the run [g, g1) of the tile list; base: first tile of sequence b
  int b, nt, ctx, nd;  // sequence b: tiles per head, context and new tokens
  int h, t0, t1;       // the current segment: tiles [t0, t1) of KV head h
  bool pieces;         // one segment only, set up already
  __device__ __forceinline__ bool next(const TreeParams& p) {
    if (g >= g1) return false;
    if (pieces) {
      g = g1;
      return true;
    }
    while (g >= base + nt * p.c.Hkv) {
      base += nt * p.c.Hkv;
      ++b;
      nd = new_tokens(p, b, ctx);
      nt = tiles(ctx, nd);
    }
    const unsigned x = g - base;
    h = x / (unsigned)nt;
    t0 = x - h * nt;
    t1 = min(nt, t0 + (g1 - g));
    g += t1 - t0;
    return true;
  }
};

// The share of blocks with this index among a row group's, for a whole warp
// (lane i looks at sequences i, i + 32, ...; a batch of up to 32 is read once).
__device__ __forceinline__ Walk block_share(const TreeParams& p, int part_lane) {
  const int lane = threadIdx.x & 31;
  int ctx = 0, nd = lane < p.B ? new_tokens(p, lane, ctx) : 0;
  int n = tiles(ctx, nd);
  const Cut cut = make_cut(p, ctx, nd);
  if (cut.bad && blockIdx.x == 0 && lane == 0) report(p.status, MINF_ERR_DEVICE_BOUNDS, 110);
  const int target = part_lane * (cut.pieces ? 1 : cut.per);  // first unit of the share
  Walk w{};
  w.pieces = cut.pieces;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    if (b0 > 0) {
      nd = b0 + lane < p.B ? new_tokens(p, b0 + lane, ctx) : 0;
      n = tiles(ctx, nd);
    }
    const int mine = cut.units(n);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += up;
    }
    const unsigned past = __ballot_sync(0xFFFFFFFFu, w.base + incl * p.c.Hkv > target);
    if (past) {
      const int at = __ffs(past) - 1, units = __shfl_sync(0xFFFFFFFFu, mine, at);
      w.b = b0 + at;
      w.nt = __shfl_sync(0xFFFFFFFFu, n, at);
      w.base += (__shfl_sync(0xFFFFFFFFu, incl, at) - units) * p.c.Hkv;
      w.ctx = __shfl_sync(0xFFFFFFFFu, ctx, at);
      w.nd = __shfl_sync(0xFFFFFFFFu, nd, at);
      if (cut.pieces) {  // piece x of head h's `units`, as even as they come
        w.h = (unsigned)(target - w.base) / (unsigned)units;
        const int x = target - w.base - w.h * units;
        w.t0 = (unsigned)x * (unsigned)w.nt / (unsigned)units;  // at most 148 * 2^24
        w.t1 = (unsigned)(x + 1) * (unsigned)w.nt / (unsigned)units;
        w.g1 = 1;
      } else {
        w.g = target;
        w.g1 = min(target + cut.per, cut.total);
      }
      break;
    }
    w.base += __shfl_sync(0xFFFFFFFFu, incl, 31) * p.c.Hkv;
  }
  return w;
}

// One warp loads the K tiles and one the V tiles, each tile page by page
// (lane i < pages loads page i): a box costs its warp about 100 cycles to
// issue, and with pages of 16 rows a tile has 8 or 16 boxes of each.  With K
// go, in 8 bits, the exponents of the tile's keys and values, four keys per
// lane.  No load is waited for: page ids come 32 at a time, a batch ahead.
template <class C, bool F8, int NR>
__device__ __forceinline__ void load_tiles(const TreeParams& p, const CUtensorMap& map, bool is_k, uint8_t* smem,
                                           uint64_t* full, uint64_t* empty, int rg, Walk w, volatile int* abort) {
  const int lane = threadIdx.x & 31;
  const int stages = is_k ? C::kKStages : C::kVStages;
  uint8_t* ring = smem + (is_k ? C::kOffK : C::kOffV);
  int n = 0;
  // failure-detection test hook: the first block withholds its key tiles, so its
  // bounded waits run out and the call reports a timeout
  bool live = p.status->withhold == 0 || blockIdx.x != 0;
  while (live && w.next(p)) {
    if (rg * NR >= w.nd * p.group) continue;
    const int len = w.ctx + w.nd;
    const int log = p.c.log_page, per_tile = 128 >> log, per_batch = 32 / per_tile;
    const int first = w.t0 * per_tile, end = min(w.t1 * per_tile, (len + (1 << log) - 1) >> log);  // pages
    const int32_t* table = p.c.pages + (long long)w.b * p.c.max_pages;
    auto fetch = [&](int pg) { return pg + lane < end ? load(table + pg + lane) : 0; };
    int row = 0, ids = fetch(first);  // first pool row of this lane's page of the batch; the next batch
    for (int t = w.t0; t < w.t1; ++t, ++n) {
      const int at = (t - w.t0) % per_batch * per_tile, pages = min(per_tile, end - t * per_tile);
      if (at == 0) {
        if (ids < 0 || ids >= p.c.n_pages) {  // reported, and page 0 read instead
          report(p.status, MINF_ERR_DEVICE_BOUNDS, 111);
          ids = 0;
        }
        row = (ids * p.c.Hkv + w.h) << log;
        ids = fetch(t * per_tile + 32);
      }
      const int st = n % stages;
      if (n >= stages)
        mbar_wait_or_abort(&empty[st], ((n / stages) - 1) & 1, abort, p.status, is_k ? 113 : 114);
      if (__any_sync(0xFFFFFFFFu, *abort)) {
        live = false;
        break;
      }
      if (F8 && is_k) {
        const int pg = (4 * lane) >> log;
        const int from = __shfl_sync(0xFFFFFFFFu, row, at + pg) + ((4 * lane) & ((1 << log) - 1));
        if (pg < pages) {
          const uint32_t e = smem_u32(smem + C::kOffExp + st * C::kExpB + lane * 4);
          cp_async4(e, p.c.ke + from);
          cp_async4(e + 128, p.c.ve + from);
        }
        cp_async_mbar_arrive(&full[st]);
        __syncwarp();
      }
      if (lane == 0) mbar_arrive_expect_tx(&full[st], (pages << log) * C::kRowB);
      const int from = __shfl_sync(0xFFFFFFFFu, row, (at + lane) & 31);
      if (lane < pages) {
        uint8_t* dst = ring + st * C::kTileB + (lane << log) * C::kPitch;
#pragma unroll
        for (int r = 0; r < C::kRegions; ++r) tma_load_2d(dst + r * C::kRegion, &map, &full[st], r * 64, from);
      }
      __syncwarp();
    }
  }
  if (lane == 0) {  // never exit with copies in flight
    int dummy = 0;
    for (int i = max(0, n - stages); i < n; ++i)
      mbar_wait(&full[i % stages], (i / stages) & 1, &dummy, p.status, is_k ? 115 : 116);
  }
  __syncwarp();
}

}  // namespace minf
