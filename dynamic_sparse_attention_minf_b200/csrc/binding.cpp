// Python binding of the serving entry points of include/minf.h: argument checks
// (type, shape, device, contiguity; the C ABI sees bare pointers), missing
// outputs, and the call on the tensors' device and its current stream.  These
// calls run once or more per generated token, where a few microseconds of
// marshalling count; the rest of the ABI is bound with ctypes.
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include <optional>
#include <string>

#include "../../include/minf.h"

namespace {

using at::Tensor;
using OptTensor = std::optional<Tensor>;

PyObject* g_error = nullptr;  // the package's MinfError(what, status)

[[noreturn]] void fail(const std::string& what, int status) {
  PyErr_SetObject(g_error, py::make_tuple(what, status).ptr());
  throw py::error_already_set();
}
void need(bool ok, const char* fn, const char* what) {
  if (!ok) fail(std::string(fn) + " (" + what + ")", MINF_ERR_INVALID_ARG);
}
void done(const char* fn, minf_status st) {
  if (st != MINF_OK) fail(fn, st);
}

// Refuses a tensor that is not dense, of this shape and type, on `dev`.
void same(const char* fn, const char* name, const Tensor& t, at::IntArrayRef shape, at::Device dev, at::ScalarType type) {
  if (t.scalar_type() == type && t.sizes() == shape && t.is_contiguous() && t.device() == dev) return;
  std::string s = std::string(name) + ": contiguous " + c10::toString(type) + " [";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  fail(std::string(fn) + " (" + s + "] on " + dev.str() + ")", MINF_ERR_INVALID_ARG);
}
void same(const char* fn, const char* name, const OptTensor& t, at::IntArrayRef shape, at::Device dev,
          at::ScalarType type) {
  if (t) same(fn, name, *t, shape, dev, type);
}

template <class T>
T* ptr(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
template <class T>
T* ptr(const OptTensor& t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

// The tensors' device, made current, and its current stream.
struct On {
  c10::cuda::CUDAGuard guard;
  void* stream;
  static at::Device checked(at::Device dev) {
    need(dev.is_cuda(), "serving call", "tensors in device memory");
    return dev;
  }
  explicit On(at::Device dev) : guard(checked(dev)), stream(c10::cuda::getCurrentCUDAStream(dev.index()).stream()) {}
};

Tensor out(const char* fn, const char* name, const OptTensor& t, at::IntArrayRef shape, at::Device dev,
           at::ScalarType type = at::kBFloat16) {
  if (!t) return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
  same(fn, name, *t, shape, dev, type);
  return *t;
}

// The workspace: the caller's, or a new zeroed one of `bytes`.
Tensor workspace(const char* fn, const OptTensor& ws, size_t bytes, at::Device dev) {
  if (!ws) return at::zeros({(int64_t)bytes}, at::TensorOptions().dtype(at::kByte).device(dev));
  need(ws->scalar_type() == at::kByte && ws->is_contiguous() && ws->device() == dev, fn,
       "ws: contiguous uint8 on the tensors' device");
  return *ws;
}

const minf_kv_cache* handle(int64_t addr) { return reinterpret_cast<const minf_kv_cache*>(addr); }

int table(const char* fn, const Tensor& pages, int64_t B, at::Device dev) {
  need(pages.dim() == 2, fn, "pages: [B, max_pages]");
  same(fn, "pages", pages, {B, pages.size(1)}, dev, at::kInt);
  need(pages.size(1) <= INT32_MAX && B <= INT32_MAX, fn, "pages: [B, max_pages]");
  return (int)pages.size(1);
}

py::tuple qkv_norm_rope(const Tensor& x, int64_t Hq, int64_t Hkv, const OptTensor& pos, const OptTensor& inv_freq,
                        const OptTensor& qw, const OptTensor& kw, double eps, bool interleaved, bool want_v,
                        const OptTensor& q, const OptTensor& k, const OptTensor& v) {
  const char* fn = "minf_qkv_norm_rope";
  const at::Device dev = x.device();
  need(x.scalar_type() == at::kBFloat16 && x.dim() == 3 && Hq > 0 && Hkv > 0 && Hq < 65536 && Hkv < 65536 &&
           x.size(2) % (Hq + 2 * Hkv) == 0 && x.stride(2) == 1 && x.size(0) <= INT32_MAX && x.size(1) <= INT32_MAX,
       fn, "qkv: bf16 [B, N, (Hq + 2 Hkv) * d], d contiguous");
  const int64_t B = x.size(0), N = x.size(1), C = x.size(2), d = C / (Hq + 2 * Hkv);
  const int64_t half = inv_freq ? inv_freq->numel() : 0;
  same(fn, "pos", pos, {B, N}, dev, at::kInt);
  same(fn, "inv_freq", inv_freq, {half}, dev, at::kDouble);
  same(fn, "q_weight", qw, {d}, dev, at::kBFloat16);
  same(fn, "k_weight", kw, {d}, dev, at::kBFloat16);
  On on(dev);
  Tensor oq = out(fn, "q", q, {B, Hq, N, d}, dev), ok = out(fn, "k", k, {B, Hkv, N, d}, dev), ov;
  if (want_v || v) ov = out(fn, "v", v, {B, Hkv, N, d}, dev);
  done(fn, minf_qkv_norm_rope(ptr<minf_bf16>(x), (int)B, (int)N, (int)Hq, (int)Hkv, (int)std::min<int64_t>(d, 1 << 20),
                              B > 1 ? x.stride(0) : 0, N > 1 ? x.stride(1) : C, ptr<int32_t>(pos), ptr<double>(inv_freq),
                              (int)std::min<int64_t>(2 * half, 1 << 20), interleaved, ptr<minf_bf16>(qw),
                              ptr<minf_bf16>(kw), (float)eps, ptr<minf_bf16>(oq), ptr<minf_bf16>(ok),
                              ov.defined() ? ptr<minf_bf16>(ov) : nullptr, on.stream));
  return py::make_tuple(oq, ok, ov.defined() ? py::cast(ov) : py::object(py::none()));
}

void kv_write(const Tensor& k, const Tensor& v, int64_t cache, const Tensor& pool, const Tensor& pages,
              const Tensor& start, const OptTensor& count, const OptTensor& rows, const OptTensor& ws) {
  const char* fn = "minf_kv_write";
  const minf_kv_cache* c = handle(cache);
  const at::Device dev = pool.device();
  need(k.dim() == 4 && k.sizes() == v.sizes() && k.scalar_type() == at::kBFloat16 && v.scalar_type() == at::kBFloat16 &&
           k.device() == dev && v.device() == dev && k.size(1) == c->Hkv && k.size(3) == c->d && k.stride(3) == 1 &&
           v.stride(3) == 1 && k.size(0) <= INT32_MAX && k.size(2) <= INT32_MAX,
       fn, "k, v: bf16 [B, Hkv, M, d] of the cache's Hkv, d and device, d contiguous");
  const int64_t B = k.size(0), M = k.size(2);
  const int mp = table(fn, pages, B, dev);
  same(fn, "start", start, {B}, dev, at::kInt);
  same(fn, "count", count, {B}, dev, at::kInt);
  int64_t N = M;
  if (rows) {
    need(rows->dim() == 2 && rows->size(1) <= INT32_MAX, fn, "rows: [B, N]");
    N = rows->size(1);
    same(fn, "rows", rows, {B, N}, dev, at::kInt);
  }
  int64_t ks[3], vs[3];  // the stride of a single one does not matter
  for (int i = 0; i < 3; ++i) {
    ks[i] = k.size(i) > 1 ? k.stride(i) : 0;
    vs[i] = v.size(i) > 1 ? v.stride(i) : 0;
  }
  On on(dev);
  const Tensor w = workspace(fn, ws, 256, dev);
  done(fn, minf_kv_write(c, ptr<minf_bf16>(k), ptr<minf_bf16>(v), (int)B, (int)N, (int)M, ks, vs, ptr<int32_t>(pages), mp,
                         ptr<int32_t>(start), ptr<int32_t>(count), ptr<int32_t>(rows), w.data_ptr(), w.numel(),
                         on.stream));
}

py::tuple kv_read(int64_t cache, const Tensor& pool, const Tensor& pages, const Tensor& lens, int64_t N,
                  const OptTensor& k, const OptTensor& v, const OptTensor& ws) {
  const char* fn = "minf_kv_read";
  const minf_kv_cache* c = handle(cache);
  const at::Device dev = pool.device();
  need(pages.dim() == 2 && N >= 0 && N <= INT32_MAX, fn, "pages: [B, max_pages], N >= 0");
  const int64_t B = pages.size(0);
  const int mp = table(fn, pages, B, dev);
  same(fn, "lens", lens, {B}, dev, at::kInt);
  On on(dev);
  Tensor ok = out(fn, "k", k, {B, c->Hkv, N, c->d}, dev), ov = out(fn, "v", v, {B, c->Hkv, N, c->d}, dev);
  const Tensor w = workspace(fn, ws, 256, dev);
  done(fn, minf_kv_read(c, ptr<int32_t>(pages), (int)B, mp, ptr<int32_t>(lens), (int)N, ptr<minf_bf16>(ok),
                        ptr<minf_bf16>(ov), w.data_ptr(), w.numel(), on.stream));
  return py::make_tuple(ok, ov);
}

py::tuple tree_attn(const Tensor& q, int64_t cache, const Tensor& pool, const Tensor& pages, const Tensor& ctx,
                    const OptTensor& n_draft, const OptTensor& mask, const OptTensor& o, const OptTensor& lse,
                    bool want_lse, double scale, const OptTensor& ws) {
  const char* fn = "minf_tree_attn";
  const minf_kv_cache* c = handle(cache);
  const at::Device dev = pool.device();
  need(q.dim() == 4 && q.scalar_type() == at::kBFloat16 && q.is_contiguous() && q.device() == dev && q.size(3) == c->d &&
           q.size(0) <= INT32_MAX && q.size(1) <= INT32_MAX && q.size(2) <= INT32_MAX,
       fn, "q: contiguous bf16 [B, Hq, T, d] of the cache's d and device");
  const int64_t B = q.size(0), Hq = q.size(1), T = q.size(2);
  const int mp = table(fn, pages, B, dev);
  same(fn, "ctx_lens", ctx, {B}, dev, at::kInt);
  same(fn, "n_draft", n_draft, {B}, dev, at::kInt);
  same(fn, "tree_mask", mask, {B, T}, dev, at::kLong);
  On on(dev);
  Tensor oo = out(fn, "o", o, q.sizes(), dev), ol;
  if (want_lse || lse) ol = out(fn, "lse", lse, {B, Hq, T}, dev, at::kFloat);
  Tensor w;
  if (ws) {
    w = workspace(fn, ws, 0, dev);
  } else {
    const size_t bytes = minf_tree_attn_workspace((int)B, (int)Hq, c->Hkv, (int)T, c->d);
    if (bytes == 0) fail(fn, T > 64 ? MINF_ERR_UNSUPPORTED : MINF_ERR_INVALID_ARG);
    w = workspace(fn, ws, bytes, dev);
  }
  done(fn, minf_tree_attn(c, ptr<minf_bf16>(q), (int)B, (int)Hq, (int)T, (float)scale, ptr<int32_t>(pages), mp,
                          ptr<int32_t>(ctx), ptr<int32_t>(n_draft), ptr<uint64_t>(mask), ptr<minf_bf16>(oo),
                          ol.defined() ? ptr<float>(ol) : nullptr, w.data_ptr(), w.numel(), on.stream));
  return py::make_tuple(oo, ol.defined() ? py::cast(ol) : py::object(py::none()));
}

}  // namespace

PYBIND11_MODULE(_binding, m) {
  m.def("set_error", [](py::object e) { g_error = e.release().ptr(); });
  m.def("qkv_norm_rope", &qkv_norm_rope);
  m.def("kv_write", &kv_write);
  m.def("kv_read", &kv_read);
  m.def("tree_attn", &tree_attn);
}
