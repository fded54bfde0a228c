// Host side of the serving entry points of the libminf C ABI: argument checks,
// workspace carving and dispatch.  See include/minf.h for their contracts.
#include <cmath>
#include <mutex>

#include "minf_device.cuh"
#include "serve_internal.h"

using namespace minf;

namespace {

constexpr size_t kStatusBytes = 256;

minf_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MINF_OK : MINF_ERR_CUDA; }
bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

minf_status check_ws(const void* ws, size_t bytes, size_t need) {
  if (!ws || ((uintptr_t)ws & 15)) return MINF_ERR_INVALID_ARG;
  return bytes < need ? MINF_ERR_WORKSPACE_TOO_SMALL : MINF_OK;
}

// Checks a cache and a batch's page table, and fills the kernels' view of them.
minf_status cache_view(const minf_kv_cache* c, const int32_t* pages, int B, int max_pages, KvView& v) {
  if (!c || !c->k || !c->v || !pages) return MINF_ERR_INVALID_ARG;
  if (c->type != MINF_KV_BF16 && c->type != MINF_KV_E4M3) return MINF_ERR_UNSUPPORTED;
  if (c->d != 64 && c->d != 128) return MINF_ERR_UNSUPPORTED;
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return MINF_ERR_UNSUPPORTED;
  if (c->n_pages < 1 || c->Hkv < 1 || B < 1 || max_pages < 1) return MINF_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v)) return MINF_ERR_INVALID_ARG;
  if (c->type == MINF_KV_E4M3 && (!c->k_exp || !c->v_exp || !aligned16(c->k_exp) || !aligned16(c->v_exp)))
    return MINF_ERR_INVALID_ARG;
  // rows are addressed by 32-bit tile coordinates, positions by 32-bit lengths
  if ((long long)c->n_pages * c->Hkv * c->page >= (1ll << 31)) return MINF_ERR_UNSUPPORTED;
  if ((long long)max_pages * c->page >= (1ll << 31)) return MINF_ERR_UNSUPPORTED;
  v.k = c->k;
  v.v = c->v;
  v.ke = c->type == MINF_KV_E4M3 ? c->k_exp : nullptr;
  v.ve = c->type == MINF_KV_E4M3 ? c->v_exp : nullptr;
  v.pages = pages;
  v.n_pages = c->n_pages;
  v.Hkv = c->Hkv;
  v.log_page = c->page == 16 ? 4 : c->page == 32 ? 5 : c->page == 64 ? 6 : 7;
  v.max_pages = max_pages;
  return MINF_OK;
}

bool strides_ok(const int64_t* s) {
  for (int i = 0; i < 3; ++i)
    if (s[i] < 0 || s[i] % 8 != 0) return false;
  return true;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encode() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  });
  return fn;
}

// A pool as [n_pages * Hkv * page, d] with boxes of one page by 128 bytes (64
// with rows of 64 bytes), swizzled over that width.
bool make_pool_map(CUtensorMap* m, void* ptr, const minf_kv_cache* c) {
  EncodeTiledFn enc = get_encode();
  if (!enc) return false;
  const bool f8 = c->type == MINF_KV_E4M3;
  const int row_bytes = c->d * (f8 ? 1 : 2), box_bytes = row_bytes < 128 ? row_bytes : 128;
  cuuint64_t dims[2] = {(cuuint64_t)c->d, (cuuint64_t)c->n_pages * c->Hkv * c->page};
  cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  cuuint32_t box[2] = {(cuuint32_t)(f8 ? box_bytes : box_bytes / 2), (cuuint32_t)c->page};
  cuuint32_t es[2] = {1, 1};
  return enc(m, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, ptr, dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" {

minf_status minf_qkv_norm_rope(const minf_bf16* X, int B, int N, int Hq, int Hkv, int d, int64_t batch_stride,
                               int64_t row_stride, const int32_t* pos, const double* inv_freq, int rot_dim,
                               int interleaved, const minf_bf16* q_weight, const minf_bf16* k_weight, float eps,
                               minf_bf16* Q, minf_bf16* K, minf_bf16* V, void* stream) {
  if (B < 1 || N < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return MINF_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return MINF_ERR_UNSUPPORTED;
  if (N == 0) return MINF_OK;  // empty tensors may have no address
  if (!X || !Q || !K) return MINF_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(q_weight) || !aligned16(k_weight))
    return MINF_ERR_INVALID_ARG;
  const long long heads = (long long)Hq + 2ll * Hkv;
  if (heads > 65535 || (long long)B * N * heads >= (1ll << 31)) return MINF_ERR_UNSUPPORTED;
  if (row_stride < heads * d || row_stride % 8 != 0 || batch_stride < 0 || batch_stride % 8 != 0)
    return MINF_ERR_INVALID_ARG;
  if (inv_freq) {
    if (rot_dim < 2 || rot_dim > d || ((uintptr_t)inv_freq & 7)) return MINF_ERR_INVALID_ARG;
    if (rot_dim % 16 != 0) return MINF_ERR_UNSUPPORTED;
  }
  if (!(eps >= 0.f)) return MINF_ERR_INVALID_ARG;
  RopeParams p;
  p.x = reinterpret_cast<const __nv_bfloat16*>(X);
  p.sb = batch_stride;
  p.sn = row_stride;
  p.pos = pos;
  p.inv_freq = inv_freq;
  p.qw = reinterpret_cast<const __nv_bfloat16*>(q_weight);
  p.kw = reinterpret_cast<const __nv_bfloat16*>(k_weight);
  p.q = reinterpret_cast<__nv_bfloat16*>(Q);
  p.k = reinterpret_cast<__nv_bfloat16*>(K);
  p.v = reinterpret_cast<__nv_bfloat16*>(V);
  p.B = B;
  p.N = N;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.rot = inv_freq ? rot_dim : 0;
  p.interleaved = interleaved;
  p.eps = eps;
  return cuda_status(rope_launch(d, p, (cudaStream_t)stream));
}

minf_status minf_kv_write(const minf_kv_cache* cache, const minf_bf16* K, const minf_bf16* V, int B, int N, int M,
                          const int64_t* k_strides, const int64_t* v_strides, const int32_t* pages, int max_pages,
                          const int32_t* start, const int32_t* count, const int32_t* rows, void* ws, size_t ws_bytes,
                          void* stream) {
  KvWriteParams p;
  minf_status st = cache_view(cache, pages, B, max_pages, p.c);
  if (st != MINF_OK) return st;
  if (N < 0 || M < 0) return MINF_ERR_INVALID_ARG;
  if (N == 0) return MINF_OK;  // empty tensors may have no address
  if (!K || !V || !k_strides || !v_strides || !start) return MINF_ERR_INVALID_ARG;
  if (!rows && M < N) return MINF_ERR_INVALID_ARG;
  if (!aligned16(K) || !aligned16(V) || !strides_ok(k_strides) || !strides_ok(v_strides)) return MINF_ERR_INVALID_ARG;
  if ((long long)B * cache->Hkv * N >= (1ll << 31)) return MINF_ERR_UNSUPPORTED;
  if ((st = check_ws(ws, ws_bytes, kStatusBytes)) != MINF_OK) return st;
  p.k = reinterpret_cast<const __nv_bfloat16*>(K);
  p.v = reinterpret_cast<const __nv_bfloat16*>(V);
  p.ksb = k_strides[0];
  p.ksh = k_strides[1];
  p.ksn = k_strides[2];
  p.vsb = v_strides[0];
  p.vsh = v_strides[1];
  p.vsn = v_strides[2];
  p.start = start;
  p.count = count;
  p.rows = rows;
  p.B = B;
  p.N = N;
  p.M = M;
  p.status = reinterpret_cast<DevStatus*>(ws);
  return cuda_status(kv_write_launch(cache->d, p, (cudaStream_t)stream));
}

minf_status minf_kv_read(const minf_kv_cache* cache, const int32_t* pages, int B, int max_pages, const int32_t* lens,
                         int N, minf_bf16* K, minf_bf16* V, void* ws, size_t ws_bytes, void* stream) {
  KvReadParams p;
  minf_status st = cache_view(cache, pages, B, max_pages, p.c);
  if (st != MINF_OK) return st;
  if (N < 0) return MINF_ERR_INVALID_ARG;
  if (N == 0) return MINF_OK;  // empty tensors may have no address
  if (!lens || !K || !V || !aligned16(K) || !aligned16(V)) return MINF_ERR_INVALID_ARG;
  if ((long long)B * cache->Hkv * N >= (1ll << 31)) return MINF_ERR_UNSUPPORTED;
  if ((st = check_ws(ws, ws_bytes, kStatusBytes)) != MINF_OK) return st;
  p.k = reinterpret_cast<__nv_bfloat16*>(K);
  p.v = reinterpret_cast<__nv_bfloat16*>(V);
  p.lens = lens;
  p.B = B;
  p.N = N;
  p.status = reinterpret_cast<DevStatus*>(ws);
  return cuda_status(kv_read_launch(cache->d, p, (cudaStream_t)stream));
}

size_t minf_tree_attn_workspace(int B, int Hq, int Hkv, int T, int d) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || T < 1 || T > 64 || (d != 64 && d != 128)) return 0;
  if ((long long)B * Hq * T >= (1ll << 31)) return 0;
  if (!tree_rows_supported(Hq, Hkv, T)) return 0;
  return kStatusBytes + tree_part_floats(Hq, Hkv, T, d) * sizeof(float);
}

minf_status minf_tree_attn(const minf_kv_cache* cache, const minf_bf16* Q, int B, int Hq, int T, float scale,
                           const int32_t* pages, int max_pages, const int32_t* ctx_lens, const int32_t* n_draft,
                           const uint64_t* tree_mask, minf_bf16* O, float* lse, void* ws, size_t ws_bytes,
                           void* stream) {
  TreeParams p;
  minf_status st = cache_view(cache, pages, B, max_pages, p.c);
  if (st != MINF_OK) return st;
  if (!Q || !O || !ctx_lens || Hq < 1 || Hq % cache->Hkv != 0 || T < 1) return MINF_ERR_INVALID_ARG;
  if (T > 64 || !tree_rows_supported(Hq, cache->Hkv, T) || (long long)B * cache->Hkv > 65535)
    return MINF_ERR_UNSUPPORTED;
  if (((long long)max_pages * cache->page + 127) / 128 * B * cache->Hkv >= (1ll << 30)) return MINF_ERR_UNSUPPORTED;
  if (!aligned16(Q) || !aligned16(O) || ((uintptr_t)tree_mask & 7)) return MINF_ERR_INVALID_ARG;
  if ((long long)B * Hq * T >= (1ll << 31)) return MINF_ERR_UNSUPPORTED;
  if ((st = check_ws(ws, ws_bytes, minf_tree_attn_workspace(B, Hq, cache->Hkv, T, cache->d))) != MINF_OK) return st;
  p.q = reinterpret_cast<const __nv_bfloat16*>(Q);
  p.o = reinterpret_cast<__nv_bfloat16*>(O);
  p.lse = lse;
  p.ctx = ctx_lens;
  p.ndraft = n_draft;
  p.mask = reinterpret_cast<const unsigned long long*>(tree_mask);
  p.B = B;
  p.Hq = Hq;
  p.T = T;
  p.group = Hq / cache->Hkv;
  p.scale_log2 = (scale > 0.f ? scale : 1.0f / std::sqrt((float)cache->d)) * 1.4426950408889634f;
  p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + kStatusBytes);
  p.status = reinterpret_cast<DevStatus*>(ws);
  CUtensorMap tk, tv;
  if (!make_pool_map(&tk, cache->k, cache) || !make_pool_map(&tv, cache->v, cache)) return MINF_ERR_CUDA;
  return cuda_status(tree_attn_launch(cache->d, tk, tv, p, (cudaStream_t)stream));
}

}  // extern "C"
