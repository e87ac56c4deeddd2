// Argument marshalling of the attention operators for PyTorch tensors: checks, outputs from
// torch's allocator, and one call into the loaded library on the tensors' device and its current
// stream.  Small calls are bound by the host's time; the same marshalling through ctypes took
// 7 to 10 us a call more.  Nothing is computed here.
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <dlfcn.h>

#include <cmath>
#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>

#include "bitlinear.h"

namespace py = pybind11;
using at::Tensor;
using MaybeTensor = std::optional<Tensor>;

namespace {

// The library's functions, found in the library that the package has loaded (and no other: each
// copy of it has a status word of its own).
struct Library {
  decltype(&::bl_qk_norm_rope) qk_norm_rope;
  decltype(&::bl_qk_norm_rope_append) qk_norm_rope_append;
  decltype(&::bl_qk_norm_rope_backward) qk_norm_rope_backward;
  decltype(&::bl_qk_norm_rope_backward_workspace_size) qk_norm_rope_backward_workspace_size;
  decltype(&::bl_attention_ex) attention_ex;
  decltype(&::bl_attention_backward_ex) attention_backward_ex;
  decltype(&::bl_attention_backward_workspace_size) attention_backward_workspace_size;
  decltype(&::bl_paged_attention) paged_attention;
  decltype(&::bl_paged_attention_workspace_size) paged_attention_workspace_size;
} lib = {};
template <typename F> void find(void* handle, const char* name, F& f) {
  f = reinterpret_cast<F>(dlsym(handle, name));
  if (!f) throw std::runtime_error(std::string(name) + " is not in the loaded library");
}
void use(uintptr_t handle) {
  void* h = reinterpret_cast<void*>(handle);
  find(h, "bl_qk_norm_rope", lib.qk_norm_rope);
  find(h, "bl_qk_norm_rope_append", lib.qk_norm_rope_append);
  find(h, "bl_qk_norm_rope_backward", lib.qk_norm_rope_backward);
  find(h, "bl_qk_norm_rope_backward_workspace_size", lib.qk_norm_rope_backward_workspace_size);
  find(h, "bl_attention_ex", lib.attention_ex);
  find(h, "bl_attention_backward_ex", lib.attention_backward_ex);
  find(h, "bl_attention_backward_workspace_size", lib.attention_backward_workspace_size);
  find(h, "bl_paged_attention", lib.paged_attention);
  find(h, "bl_paged_attention_workspace_size", lib.paged_attention_workspace_size);
}

struct StatusError {
  const char* fn;
  int code;
};
void check(const char* fn, bl_status s) {
  if (s != BL_OK) throw StatusError{fn, int(s)};
}

[[noreturn]] void refuse(const std::string& what) { throw py::value_error(what); }

std::string describe(const Tensor& t) {
  std::ostringstream o;
  o << t.scalar_type() << " " << t.sizes() << " strides " << t.strides() << " on " << t.device();
  return o.str();
}

int cuda_device(const Tensor& t, const char* name) {
  if (!t.defined() || !t.is_cuda()) refuse(std::string(name) + " must be on a CUDA device");
  return t.get_device();
}

// The pointer of a contiguous tensor of this type and shape on device `dev`.
void* need(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, int dev) {
  if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || !t.sizes().equals(shape) || !t.is_contiguous()) {
    std::ostringstream o;
    o << name << ": expected a contiguous " << type << " tensor of shape " << shape << " on cuda:" << dev << ", got "
      << describe(t);
    refuse(o.str());
  }
  return t.data_ptr();
}

bl_dtype half_type(const Tensor& t, const char* name) {
  if (t.scalar_type() == at::kHalf) return BL_T_F16;
  if (t.scalar_type() == at::kBFloat16) return BL_T_BF16;
  refuse(std::string(name) + ": expected float16 or bfloat16, got " + describe(t));
}
at::ScalarType scalar_of(int code) {
  if (code == BL_T_F32) return at::kFloat;
  if (code == BL_T_F16) return at::kHalf;
  if (code == BL_T_BF16) return at::kBFloat16;
  refuse("unsupported dtype");
}
int code_of(const Tensor& t) {
  if (t.scalar_type() == at::kFloat) return BL_T_F32;
  return half_type(t, "gradients");
}

Tensor make(at::IntArrayRef shape, at::ScalarType type, int dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, c10::DeviceIndex(dev))));
}

void* workspace(const MaybeTensor& ws, Tensor& own, size_t bytes, int dev, size_t& have) {
  if (ws) {
    if (!ws->is_cuda() || ws->get_device() != dev || !ws->is_contiguous())
      refuse("ws: expected a contiguous tensor on cuda:" + std::to_string(dev) + ", got " + describe(*ws));
    have = ws->nbytes();
    return ws->data_ptr();
  }
  own = make({int64_t(bytes)}, at::kByte, dev);
  have = bytes;
  return bytes ? own.data_ptr() : nullptr;
}

cudaStream_t stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(dev)).stream(); }

// ---- norms and rotation ----------------------------------------------------------------
// float32 rows [m, width] whose elements are contiguous: pointer and stride.
const float* rows2(const Tensor& t, int64_t m, int64_t width, int dev, int64_t& ld) {
  if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(0) != m ||
      t.size(1) != width || (width > 1 && t.stride(1) != 1))
    refuse("qkv: expected float32 rows [" + std::to_string(m) + ", " + std::to_string(width) + "] on cuda:" +
           std::to_string(dev) + ", got " + describe(t));
  ld = m > 1 ? t.stride(0) : width;
  return static_cast<const float*>(t.data_ptr());
}

// The rows of a fused projection [M, (heads + 2 kv_heads) dim] or of three separate ones.
bl_qkv_rows qkv_rows(const py::object& qkv, int64_t heads, int64_t kv_heads, int64_t dim, const MaybeTensor& pos,
                     const MaybeTensor& table, const MaybeTensor& gq, const MaybeTensor& gk, double eps, bool interleaved,
                     bool values, int& dev) {
  if (heads < 1 || heads > 65535 || kv_heads < 1 || kv_heads > 65535 || dim < 1 || dim > 65535) refuse("heads, kv_heads or dim out of range");
  const int64_t wq = heads * dim, wk = kv_heads * dim;
  bl_qkv_rows r = {};
  r.Hq = int32_t(heads);
  r.Hkv = int32_t(kv_heads);
  r.D = int32_t(dim);
  r.eps = float(eps);
  r.interleaved = interleaved ? 1 : 0;
  if (THPVariable_Check(qkv.ptr())) {
    const Tensor& t = THPVariable_Unpack(qkv.ptr());
    dev = cuda_device(t, "qkv");
    if (t.dim() != 2) refuse("qkv: expected [M, (heads + 2 kv_heads) dim] rows, got " + describe(t));
    r.M = t.size(0);
    r.q = rows2(t, r.M, wq + 2 * wk, dev, r.ldq);
    r.k = r.q + wq;
    r.v = r.k + wk;
    r.ldk = r.ldv = r.ldq;
  } else {
    const py::tuple parts = py::reinterpret_borrow<py::object>(qkv);
    if (parts.size() != 3) refuse("qkv: one tensor or three");
    const Tensor q = py::cast<Tensor>(parts[0]), k = py::cast<Tensor>(parts[1]);
    dev = cuda_device(q, "qkv");
    if (q.dim() != 2) refuse("qkv: expected [M, heads dim] rows, got " + describe(q));
    r.M = q.size(0);
    r.q = rows2(q, r.M, wq, dev, r.ldq);
    r.k = rows2(k, r.M, wk, dev, r.ldk);
    if (values || !parts[2].is_none()) r.v = rows2(py::cast<Tensor>(parts[2]), r.M, wk, dev, r.ldv);
  }
  if (table) {
    if (table->dim() != 2) refuse("table is [positions, rotated elements]");
    r.P = table->size(0);
    r.R = int32_t(table->size(1));
    r.table = static_cast<const float*>(need(*table, "table", at::kFloat, {r.P, int64_t(r.R)}, dev));
    if (!pos) refuse("pos: needed with a table");
    r.pos = static_cast<const int32_t*>(need(*pos, "pos", at::kInt, {r.M}, dev));
  }
  if (gq) r.gq = static_cast<const float*>(need(*gq, "gq", at::kFloat, {dim}, dev));
  if (gk) r.gk = static_cast<const float*>(need(*gk, "gk", at::kFloat, {dim}, dev));
  return r;
}

py::tuple qk_norm_rope(const py::object& qkv, int64_t heads, int64_t kv_heads, int64_t dim, const MaybeTensor& pos,
                       const MaybeTensor& table, const MaybeTensor& gq, const MaybeTensor& gk, double eps, int dtype,
                       bool interleaved) {
  int dev;
  const bl_qkv_rows r = qkv_rows(qkv, heads, kv_heads, dim, pos, table, gq, gk, eps, interleaved, true, dev);
  const at::ScalarType type = scalar_of(dtype);
  Tensor q = make({r.M, heads, dim}, type, dev), k = make({r.M, kv_heads, dim}, type, dev), v = make({r.M, kv_heads, dim}, type, dev);
  const c10::cuda::CUDAGuard guard{c10::DeviceIndex(dev)};
  check("bl_qk_norm_rope", lib.qk_norm_rope(&r, bl_dtype(dtype), q.data_ptr(), k.data_ptr(), v.data_ptr(), stream_of(dev)));
  return py::make_tuple(q, k, v);
}

// A cache [pages, kv_heads, page, dim].
bl_kv_pages cache_of(const Tensor& k, const Tensor& v, int dev) {
  if (k.dim() != 4) refuse("a cache is [pages, kv_heads, page, dim]");
  bl_kv_pages c = {};
  c.t = half_type(k, "kcache");
  c.k = need(k, "kcache", k.scalar_type(), k.sizes(), dev);
  c.v = need(v, "vcache", k.scalar_type(), k.sizes(), dev);
  if (k.size(1) > 65535 || k.size(2) >= (int64_t(1) << 31) || k.size(3) > 65535) refuse("kcache: too large a dimension");
  c.pages = k.size(0);
  c.Hkv = int32_t(k.size(1));
  c.page = int32_t(k.size(2));
  c.D = int32_t(k.size(3));
  return c;
}

Tensor qk_norm_rope_append(const py::object& qkv, int64_t heads, int64_t kv_heads, int64_t dim, const MaybeTensor& pos,
                           const MaybeTensor& table, const MaybeTensor& gq, const MaybeTensor& gk, const Tensor& kcache,
                           const Tensor& vcache, const Tensor& slots, double eps, bool interleaved) {
  int dev;
  const bl_qkv_rows r = qkv_rows(qkv, heads, kv_heads, dim, pos, table, gq, gk, eps, interleaved, true, dev);
  const bl_kv_pages c = cache_of(kcache, vcache, dev);
  const auto* at_ = static_cast<const int64_t*>(need(slots, "slots", at::kLong, {r.M}, dev));
  Tensor q = make({r.M, heads, dim}, kcache.scalar_type(), dev);
  const c10::cuda::CUDAGuard guard{c10::DeviceIndex(dev)};
  check("bl_qk_norm_rope_append", lib.qk_norm_rope_append(&r, q.data_ptr(), &c, at_, stream_of(dev)));
  return q;
}

py::tuple qk_norm_rope_backward(const Tensor& dq, const Tensor& dk, const Tensor& dv, const py::object& qkv, int64_t heads,
                                int64_t kv_heads, int64_t dim, const MaybeTensor& pos, const MaybeTensor& table,
                                const MaybeTensor& gq, const MaybeTensor& gk, double eps, bool interleaved,
                                const MaybeTensor& ws) {
  int dev;
  const bl_qkv_rows r = qkv_rows(qkv, heads, kv_heads, dim, pos, table, gq, gk, eps, interleaved, false, dev);
  const int code = code_of(dq);
  const at::ScalarType type = dq.scalar_type();
  const void* pq = need(dq, "dq", type, {r.M, heads, dim}, dev);
  const void* pk = need(dk, "dk", type, {r.M, kv_heads, dim}, dev);
  const void* pv = need(dv, "dv", type, {r.M, kv_heads, dim}, dev);
  const int64_t wq = heads * dim, wk = kv_heads * dim, wide = wq + 2 * wk;
  Tensor dx = make({r.M, wide}, at::kFloat, dev), dgq = make({dim}, at::kFloat, dev), dgk = make({dim}, at::kFloat, dev), own;
  size_t have = 0;
  void* w = workspace(ws, own, ws ? 0 : lib.qk_norm_rope_backward_workspace_size(&r), dev, have);
  float* x = static_cast<float*>(dx.data_ptr());
  const c10::cuda::CUDAGuard guard{c10::DeviceIndex(dev)};
  check("bl_qk_norm_rope_backward",
        lib.qk_norm_rope_backward(&r, bl_dtype(code), pq, pk, pv, x, wide, x + wq, wide, x + wq + wk, wide,
                                 static_cast<float*>(dgq.data_ptr()), static_cast<float*>(dgk.data_ptr()), w, have,
                                 stream_of(dev)));
  return py::make_tuple(dx, dgq, dgk);
}

// ---- attention over packed sequences ----------------------------------------------------
// [tokens, heads, D] rows whose heads are D apart: pointer and elements between tokens.
const void* rows3(const Tensor& t, const char* name, at::ScalarType type, int dev, int64_t& ld) {
  if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || t.dim() != 3)
    refuse(std::string(name) + ": expected [tokens, heads, D] of one type and device, got " + describe(t));
  const int64_t n = t.size(0), h = t.size(1), d = t.size(2);
  if (t.is_contiguous()) {
    ld = h * d;
  } else {
    if (t.stride(2) != 1 || (h > 1 && t.stride(1) != d))
      refuse(std::string(name) + ": the heads of a token must be contiguous, got " + describe(t));
    ld = n > 1 ? t.stride(0) : h * d;
  }
  return t.data_ptr();
}

int32_t int32_of(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " does not fit 32 bits");
  return int32_t(v);
}

bl_attn_call attn_call(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu_q, const Tensor& cu_k,
                       int64_t max_q, int64_t max_k, int64_t window, int64_t sinks, const std::optional<double>& scale,
                       int& dev) {
  dev = cuda_device(q, "q");
  const at::ScalarType type = q.scalar_type();
  bl_attn_call c = {};
  c.t = half_type(q, "q");
  c.q = rows3(q, "q", type, dev, c.ldq);
  c.k = rows3(k, "k", type, dev, c.ldk);
  c.v = rows3(v, "v", type, dev, c.ldv);
  if (!k.sizes().equals(v.sizes()) || k.size(2) != q.size(2))
    refuse("q, k and v do not fit together: " + describe(q) + ", " + describe(k) + ", " + describe(v));
  c.Tq = q.size(0);
  c.Tk = k.size(0);
  c.Hq = int32_of(q.size(1), "heads");
  c.Hkv = int32_of(k.size(1), "kv_heads");
  c.D = int32_of(q.size(2), "D");
  if (cu_q.dim() != 1 || cu_q.size(0) < 1) refuse("cu_q holds at least one offset");
  c.cu_q = static_cast<const int32_t*>(need(cu_q, "cu_q", at::kInt, cu_q.sizes(), dev));
  c.cu_k = static_cast<const int32_t*>(need(cu_k, "cu_k", at::kInt, cu_q.sizes(), dev));
  c.B = int32_of(cu_q.size(0) - 1, "sequences");
  c.max_q = int32_of(max_q, "max_q");
  c.max_k = int32_of(max_k, "max_k");
  c.window = int32_of(window, "window");
  c.sinks = int32_of(sinks, "sinks");
  c.scale = scale ? float(*scale) : float(1.0 / std::sqrt(double(c.D)));
  return c;
}

py::tuple attention(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& cu_q, const Tensor& cu_k, int64_t max_q,
                    int64_t window, int64_t sinks, const std::optional<double>& scale, const MaybeTensor& out,
                    const MaybeTensor& lse) {
  int dev;
  const bl_attn_call c = attn_call(q, k, v, cu_q, cu_k, max_q, 0, window, sinks, scale, dev);
  Tensor o = out ? *out : make(q.sizes(), q.scalar_type(), dev);
  Tensor l = lse ? *lse : make({q.size(1), q.size(0)}, at::kFloat, dev);
  void* po = need(o, "out", q.scalar_type(), q.sizes(), dev);
  auto* pl = static_cast<float*>(need(l, "lse", at::kFloat, {q.size(1), q.size(0)}, dev));
  const c10::cuda::CUDAGuard guard{c10::DeviceIndex(dev)};
  // rows of no sequence: what a caller's tensor holds stays, what comes from the allocator is cleared
  const int clear = (out ? 0 : BL_CLEAR_OUT) | (lse ? 0 : BL_CLEAR_LSE);
  check("bl_attention", lib.attention_ex(&c, po, pl, clear, stream_of(dev)));
  return py::make_tuple(o, l);
}

py::tuple attention_backward(const Tensor& dout, const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& out,
                             const Tensor& lse, const Tensor& cu_q, const Tensor& cu_k, int64_t max_q, int64_t max_k,
                             int64_t window, int64_t sinks, const std::optional<double>& scale, const MaybeTensor& ws,
                             const MaybeTensor& gq, const MaybeTensor& gk, const MaybeTensor& gv) {
  int dev;
  const bl_attn_call c = attn_call(q, k, v, cu_q, cu_k, max_q, max_k, window, sinks, scale, dev);
  const at::ScalarType type = q.scalar_type();
  const void* po = need(out, "out", type, q.sizes(), dev);
  const void* pg = need(dout, "dout", type, q.sizes(), dev);
  const auto* pl = static_cast<const float*>(need(lse, "lse", at::kFloat, {q.size(1), q.size(0)}, dev));
  Tensor dq = gq ? *gq : make(q.sizes(), type, dev), dk = gk ? *gk : make(k.sizes(), type, dev),
         dv = gv ? *gv : make(k.sizes(), type, dev), own;
  void* pq = need(dq, "dq", type, q.sizes(), dev);
  void* pk = need(dk, "dk", type, k.sizes(), dev);
  void* pv = need(dv, "dv", type, k.sizes(), dev);
  size_t have = 0;
  void* w = workspace(ws, own, ws ? 0 : lib.attention_backward_workspace_size(&c), dev, have);
  const c10::cuda::CUDAGuard guard{c10::DeviceIndex(dev)};
  const int clear = (gq ? 0 : BL_CLEAR_DQ) | (gk ? 0 : BL_CLEAR_DK) | (gv ? 0 : BL_CLEAR_DV);
  check("bl_attention_backward", lib.attention_backward_ex(&c, po, pl, pg, pq, pk, pv, w, have, clear, stream_of(dev)));
  return py::make_tuple(dq, dk, dv);
}

// ---- paged -----------------------------------------------------------------------------------
Tensor paged_attention(const Tensor& q, const Tensor& kcache, const Tensor& vcache, const Tensor& pages, const Tensor& lens,
                       int64_t window, int64_t sinks, const std::optional<double>& scale, int out_dtype,
                       const MaybeTensor& ws, const MaybeTensor& out) {
  const int dev = cuda_device(q, "q");
  const bl_kv_pages c = cache_of(kcache, vcache, dev);
  if (q.dim() != 3 || q.size(2) != c.D) refuse("q is [batch, heads, " + std::to_string(c.D) + "], got " + describe(q));
  const int64_t b = q.size(0), h = q.size(1);
  const at::ScalarType type = scalar_of(out_dtype);
  const void* pq = need(q, "q", kcache.scalar_type(), q.sizes(), dev);
  if (pages.dim() != 2 || pages.size(0) != b) refuse("pages is [batch, n], got " + describe(pages));
  const auto* pp = static_cast<const int32_t*>(need(pages, "pages", at::kInt, pages.sizes(), dev));
  const auto* pl = static_cast<const int32_t*>(need(lens, "lens", at::kInt, {b}, dev));
  Tensor o = out ? *out : make(q.sizes(), type, dev), own;
  void* po = need(o, "out", type, q.sizes(), dev);
  const c10::cuda::CUDAGuard guard{c10::DeviceIndex(dev)};
  size_t have = 0;
  void* w;
  if (ws) {
    w = workspace(ws, own, 0, dev, have);
  } else {                                             // its counters have to be zero
    have = lib.paged_attention_workspace_size(b, int32_of(h, "heads"), &c);
    own = at::zeros({int64_t(have)}, at::TensorOptions().dtype(at::kByte).device(q.device()));
    w = own.data_ptr();
  }
  check("bl_paged_attention",
        lib.paged_attention(pq, b, int32_of(h, "heads"), &c, pp, pages.size(1), pl, int32_of(window, "window"),
                           int32_of(sinks, "sinks"), scale ? float(*scale) : float(1.0 / std::sqrt(double(c.D))),
                           bl_dtype(out_dtype), po, w, have, stream_of(dev)));
  return o;
}

}  // namespace

PYBIND11_MODULE(_binding, m) {
  py::register_exception_translator([](std::exception_ptr p) {
    try {
      if (p) std::rethrow_exception(p);
    } catch (const StatusError& e) {
      const py::object cls = py::module_::import("int8_row_absmax_b200").attr("BitLinearError");
      PyErr_SetObject(cls.ptr(), cls(e.fn, e.code).ptr());
    }
  });
  m.attr("built_for") = BL_BUILT_FOR;                  // looked for in the file before it is loaded
  m.def("use", &use);
  m.def("qk_norm_rope", &qk_norm_rope);
  m.def("qk_norm_rope_append", &qk_norm_rope_append);
  m.def("qk_norm_rope_backward", &qk_norm_rope_backward);
  m.def("attention", &attention);
  m.def("attention_backward", &attention_backward);
  m.def("paged_attention", &paged_attention);
}
