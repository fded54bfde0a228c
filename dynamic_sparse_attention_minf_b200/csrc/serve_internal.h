// Internal declarations of the serving operators (head norm and rotation,
// paged key-value cache, attention over the cache): the launch parameters
// shared by their host entry points (serve_api.cu) and kernels.  Not part of
// the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/minf.h"

namespace minf {

struct DevStatus;

struct RopeParams {
  const __nv_bfloat16* x;  // rows of (Hq + 2 Hkv) * d
  long long sb, sn;        // element strides of batch and token
  const int32_t* pos;      // [B, N] or NULL (row n has position n)
  const double* inv_freq;  // [rot / 2] or NULL (no rotation)
  const __nv_bfloat16* qw; // [d] or NULL (no norm)
  const __nv_bfloat16* kw;
  __nv_bfloat16 *q, *k, *v;  // v NULL: the value heads are not copied
  int B, N, Hq, Hkv, rot, interleaved;
  float eps;
};
cudaError_t rope_launch(int d, const RopeParams& p, cudaStream_t stream);

// A sequence's pages: position j is row j % page of page pages[b][j / page].
struct KvView {
  void *k, *v;
  uint8_t *ke, *ve;  // NULL: the rows are bf16
  const int32_t* pages;
  int n_pages, Hkv, log_page, max_pages;
};

struct KvWriteParams {
  KvView c;
  const __nv_bfloat16 *k, *v;
  long long ksb, ksh, ksn, vsb, vsh, vsn;  // element strides of batch, head, row
  const int32_t* start;   // [B]
  const int32_t* count;   // [B] or NULL (N)
  const int32_t* rows;    // [B, N] source rows or NULL (0 .. N-1)
  int B, N, M;            // M source rows
  DevStatus* status;
};
cudaError_t kv_write_launch(int d, const KvWriteParams& p, cudaStream_t stream);

struct KvReadParams {
  KvView c;
  __nv_bfloat16 *k, *v;   // [B, Hkv, N, d]
  const int32_t* lens;    // [B]
  int B, N;
  DevStatus* status;
};
cudaError_t kv_read_launch(int d, const KvReadParams& p, cudaStream_t stream);

struct TreeParams {
  KvView c;
  const __nv_bfloat16* q;  // [B, Hq, T, d]
  __nv_bfloat16* o;
  float* lse;              // [B, Hq, T] or NULL
  const int32_t* ctx;      // [B]
  const int32_t* ndraft;   // [B] or NULL (T)
  const unsigned long long* mask;  // [B, T] or NULL (a chain: token t sees 0 .. t)
  int B, Hq, T, group;
  float scale_log2;
  float* part;             // workspace
  DevStatus* status;
  // set by the launch: row groups of `rows` rows, and the number of runs that
  // the tile list is cut into
  int groups, rows, lanes;
};
size_t tree_part_floats(int Hq, int Hkv, int T, int d);
bool tree_rows_supported(int Hq, int Hkv, int T);
// tk, tv: the pools as [n_pages * Hkv * page, d] with boxes of one page by 128
// bytes (64 with rows of 64 bytes), swizzled over that width.
cudaError_t tree_attn_launch(int d, const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p,
                             cudaStream_t stream);
// The blocks' part of it for groups of 128 rows (tree_wide.cu).
cudaError_t tree_wide_launch(int d, const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p,
                             cudaStream_t stream);

}  // namespace minf
