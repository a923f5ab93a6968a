// The operators on torch tensors: argument checks, output allocation and the calls of the
// C ABI (include/moe_tsg.h), as the functions of the Python module _torch_ops that ops.py
// documents. No computation here. In C++ because the host's part is what a small call costs:
// with the same checks in Python over ctypes it was 14 us (routing, linear), 19 (layer norm)
// and 24 to 32 (backward passes) on a Grace host, here 5 to 10, 6 to 12 and 11 to 18 by the machine.
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include <optional>
#include <sstream>
#include <string>
#include <tuple>

#include "../../include/moe_tsg.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

PyObject* g_moe_error = nullptr;  // capi.MoeError

// A call of the C ABI, without the interpreter's lock: a launch may wait for room in the
// device's queue.
template <typename F>
void call(const char* what, F f) {
  int rc;
  {
    py::gil_scoped_release free;
    rc = f();
  }
  if (rc == MOE_OK) return;
  const char* name = rc == MOE_ERR_ARG           ? "MOE_ERR_ARG"
                     : rc == MOE_ERR_WORKSPACE   ? "MOE_ERR_WORKSPACE"
                     : rc == MOE_ERR_CUDA        ? "MOE_ERR_CUDA"
                     : rc == MOE_ERR_UNSUPPORTED ? "MOE_ERR_UNSUPPORTED"
                                                 : "unknown error";
  PyErr_SetString(g_moe_error != nullptr ? g_moe_error : PyExc_RuntimeError,
                  (std::string(what) + " failed: " + name).c_str());
  throw py::error_already_set();
}

template <typename... A>
[[noreturn]] void refuse(const A&... parts) {
  std::ostringstream s;
  (s << ... << parts);
  throw py::value_error(s.str());
}

int type_of(at::ScalarType t) {
  return t == at::kBFloat16 ? MOE_BF16 : t == at::kHalf ? MOE_FP16 : t == at::kFloat ? MOE_FP32 : -1;
}
int checked_type(const Tensor& t, const char* what, bool half_only = false) {
  const int d = type_of(t.scalar_type());
  if (d < 0 || (half_only && d == MOE_FP32))
    refuse(what, " has type ", t.scalar_type(), ": expected bfloat16",
           half_only ? " or float16" : ", float16 or float32");
  return d;
}

struct Rows {
  int64_t n, c, ld;
};
// A tensor as a matrix: its last dimension contiguous, the others one run of rows.
Rows rows_of(const Tensor& t, const char* what, int64_t cols = -1) {
  const auto sizes = t.sizes();
  const auto strides = t.strides();
  const int64_t dim = t.dim();
  bool ok = dim > 0;
  Rows r{1, dim > 0 ? sizes[dim - 1] : 0, 0};
  if (t.numel() == 0) {  // no elements: whatever the strides
    for (int64_t d = 0; d < dim - 1; ++d) r.n *= sizes[d];
    if (cols >= 0 && r.c != cols) refuse(what, " has rows of ", r.c, " elements: expected ", cols);
    r.ld = r.c;
    return r;
  }
  if (ok) ok = r.c <= 1 || strides[dim - 1] == 1;
  // The dimensions of more than one element before the last: each spans the one after it.
  int64_t step = -1;
  for (int64_t d = dim - 2; ok && d >= 0; --d) {
    if (sizes[d] == 1) continue;
    if (step < 0) {
      r.ld = strides[d];
      ok = r.ld >= r.c;
    } else {
      ok = strides[d] == step;
    }
    step = strides[d] * sizes[d];
    r.n *= sizes[d];
  }
  if (!ok)
    refuse(what, " must be rows of contiguous elements, got shape ", sizes, " and strides ", strides);
  if (cols >= 0 && r.c != cols) refuse(what, " has rows of ", r.c, " elements: expected ", cols);
  if (r.n <= 1) r.ld = r.c;
  return r;
}
void same_device(const Tensor& t, const Tensor& x, const char* what) {
  if (t.device() != x.device()) refuse(what, " is on ", t.device(), ": expected ", x.device());
}
// A contiguous vector of `size` elements of x's type or (also) fp32, beside x.
void check_vector(const Tensor& t, const char* what, int64_t size, at::ScalarType type,
                  const Tensor& x) {
  if (t.dim() != 1 || t.size(0) != size || !t.is_contiguous() ||
      (t.scalar_type() != type && t.scalar_type() != at::kFloat) || t.device() != x.device())
    refuse(what, " must be ", size, " contiguous elements of ", type,
           type == at::kFloat ? "" : " or float32", " beside the rows, got ", t.sizes(), " of ",
           t.scalar_type(), " on ", t.device());
}
void same_shape(const Tensor& t, at::IntArrayRef shape, const Tensor& x, const char* what) {
  if (t.sizes() != shape || t.scalar_type() != x.scalar_type())
    refuse(what, " must be ", shape, " of ", x.scalar_type(), ", got ", t.sizes(), " of ",
           t.scalar_type());
  same_device(t, x, what);
}
// Rows of a matrix that the tensor maps read: on 16 bytes.
Rows operand(const Tensor& t, const char* what, int64_t cols, const Tensor& x) {
  const Rows r = rows_of(t, what, cols);
  if (t.scalar_type() != x.scalar_type())
    refuse(what, " has type ", t.scalar_type(), ": expected ", x.scalar_type());
  same_device(t, x, what);
  const auto at = reinterpret_cast<uintptr_t>(t.data_ptr()) % 16;
  if (at != 0 || (r.n > 1 && r.ld % 8 != 0))
    refuse(what, " must have rows that start on 16 bytes (a row stride that is a multiple of 8 ",
           "elements), got a stride of ", r.ld, " and an address of ", at, " modulo 16");
  return r;
}

// A size in an int's field; what it cannot hold is beyond every limit of such a field.
int as_int(int64_t v) { return (int)std::min<int64_t>(v, INT32_MAX); }
void* ptr(const OptTensor& t) { return t.has_value() ? t->data_ptr() : nullptr; }
Tensor empty(at::IntArrayRef shape, at::ScalarType type, const Tensor& x) {
  return at::empty(shape, x.options().dtype(type));
}
std::vector<int64_t> with_last(const Tensor& t, int64_t last) {
  std::vector<int64_t> s(t.sizes().begin(), t.sizes().end());
  s.back() = last;
  return s;
}

// The device of a call, current while it runs, and its stream.
struct Launch {
  c10::cuda::CUDAGuard guard;
  moe_stream_t stream;
  static c10::Device device(const Tensor& x) {
    if (!x.is_cuda()) refuse("tensors must be on a CUDA device, got ", x.device());
    return x.device();
  }
  explicit Launch(const Tensor& x)
      : guard(device(x)),
        stream(c10::cuda::getCurrentCUDAStream(x.device().index()).stream()) {}
};

int score_of(const std::string& s) {
  if (s == "softmax") return MOE_SCORE_SOFTMAX;
  if (s == "sigmoid") return MOE_SCORE_SIGMOID;
  refuse("score '", s, "': expected one of softmax, sigmoid");
}
int act_of(const std::string& s) {
  static const char* const names[] = {"none", "relu", "gelu", "gelu_tanh", "silu"};
  for (int i = 0; i < 5; ++i)
    if (s == names[i]) return i;
  refuse("act '", s, "': expected one of none, relu, gelu, gelu_tanh, silu");
}
static_assert(MOE_ACT_NONE == 0 && MOE_ACT_RELU == 1 && MOE_ACT_GELU == 2 && MOE_ACT_GELU_TANH == 3 &&
                  MOE_ACT_SILU == 4,
              "the names' order");

// ------------------------------------------------------------------------------ routing
std::tuple<Tensor, Tensor> route(const Tensor& logits, int topk, const std::string& score,
                                 const OptTensor& bias, int groups, int topk_groups, int group_top,
                                 bool renorm, float scale) {
  const Rows r = rows_of(logits, "logits");
  const int dt = checked_type(logits, "logits");
  if (bias.has_value()) check_vector(*bias, "bias", r.c, at::kFloat, logits);
  const moe_router_cfg cfg{as_int(r.c), topk, score_of(score), groups, topk_groups, group_top,
                           renorm ? 1 : 0, scale};
  const Launch l(logits);
  const auto shape = with_last(logits, std::max(topk, 0));
  Tensor ids = empty(shape, at::kInt, logits), w = empty(shape, at::kFloat, logits);
  call("moe_router", [&] {
    return moe_router(nullptr, &cfg, logits.data_ptr(), dt, r.n, r.ld,
                      static_cast<const float*>(ptr(bias)), static_cast<int32_t*>(ids.data_ptr()),
                      static_cast<float*>(w.data_ptr()), l.stream);
  });
  return {ids, w};
}

// The routing of a layer's tokens into its ids and weights, on the stream of that handle.
void route_plan(uintptr_t plan, int64_t n, int E, int topk, int score, int groups, int topk_groups,
                int group_top, int renorm, float scale, const Tensor& logits, const OptTensor& bias,
                const Tensor& ids, const Tensor& w, uintptr_t stream) {
  const Rows r = rows_of(logits, "logits");
  const int dt = checked_type(logits, "logits");
  if (r.c != E || r.n != n)
    refuse("logits hold ", r.n, " rows of ", r.c, ": expected ", n, " rows of ", E);
  if (bias.has_value()) check_vector(*bias, "bias", E, at::kFloat, logits);
  same_device(logits, ids, "logits");
  const moe_router_cfg cfg{E, topk, score, groups, topk_groups, group_top, renorm, scale};
  const c10::cuda::CUDAGuard guard(Launch::device(logits));
  call("moe_router", [&] {
    return moe_router(reinterpret_cast<moe_plan*>(plan), &cfg, logits.data_ptr(), dt, n, r.ld,
                      static_cast<const float*>(ptr(bias)), static_cast<int32_t*>(ids.data_ptr()),
                      static_cast<float*>(w.data_ptr()), reinterpret_cast<moe_stream_t>(stream));
  });
}

Tensor route_backward(const Tensor& d_w, const Tensor& logits, const Tensor& ids,
                      const std::string& score, bool renorm, float scale) {
  const Rows r = rows_of(logits, "logits");
  const int dt = checked_type(logits, "logits");
  const int64_t k = ids.dim() > 0 ? ids.size(-1) : 0;
  const auto shape = with_last(logits, k);
  auto beside = [&](const Tensor& t, const char* what, at::ScalarType type) {
    if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(shape) || !t.is_contiguous() ||
        t.device() != logits.device())
      refuse(what, " must be contiguous ", type, " of shape ", shape, " beside the logits, got ",
             t.sizes(), " of ", t.scalar_type(), " on ", t.device());
  };
  beside(ids, "ids", at::kInt);
  beside(d_w, "d_w", at::kFloat);
  const moe_router_cfg cfg{as_int(r.c), as_int(k), score_of(score), 1, 1, 1, renorm ? 1 : 0, scale};
  const Launch l(logits);
  Tensor d = empty(logits.sizes(), logits.scalar_type(), logits);
  call("moe_router_backward", [&] {
    return moe_router_backward(&cfg, static_cast<const float*>(d_w.data_ptr()), logits.data_ptr(),
                               static_cast<const int32_t*>(ids.data_ptr()), dt, r.n, r.ld,
                               d.data_ptr(), r.c, l.stream);
  });
  return d;
}

// --------------------------------------------------------------------------- layer norm
std::tuple<Tensor, Tensor, OptTensor, OptTensor> layer_norm(const Tensor& x, const OptTensor& weight,
                                                           const OptTensor& bias, float eps,
                                                           const OptTensor& residual, bool stats) {
  const Rows r = rows_of(x, "x");
  const int dt = checked_type(x, "x");
  if (weight.has_value()) check_vector(*weight, "weight", r.c, x.scalar_type(), x);
  if (bias.has_value()) check_vector(*bias, "bias", r.c, x.scalar_type(), x);
  if (weight.has_value() && bias.has_value() && weight->scalar_type() != bias->scalar_type())
    refuse("weight and bias differ in type: ", weight->scalar_type(), " and ", bias->scalar_type());
  Rows rr{};
  if (residual.has_value()) {
    same_shape(*residual, x.sizes(), x, "residual");
    rr = rows_of(*residual, "residual", r.c);
  }
  const Launch l(x);
  Tensor y = empty(x.sizes(), x.scalar_type(), x);
  Tensor z = residual.has_value() ? empty(x.sizes(), x.scalar_type(), x) : x;
  OptTensor mean, rstd;
  if (stats) {
    mean = empty(x.sizes().slice(0, x.dim() - 1), at::kFloat, x);
    rstd = empty(x.sizes().slice(0, x.dim() - 1), at::kFloat, x);
  }
  moe_norm_args a{};
  a.n = r.n;
  a.D = as_int(r.c);
  a.dtype = dt;
  a.wtype = weight.has_value() ? type_of(weight->scalar_type())
            : bias.has_value() ? type_of(bias->scalar_type())
                               : dt;
  a.eps = eps;
  a.x = x.data_ptr();
  a.r = ptr(residual);
  a.w = ptr(weight);
  a.b = ptr(bias);
  a.y = y.data_ptr();
  a.z = residual.has_value() ? z.data_ptr() : nullptr;
  a.mean = static_cast<float*>(ptr(mean));
  a.rstd = static_cast<float*>(ptr(rstd));
  a.ld_x = r.ld;
  a.ld_r = rr.ld;
  a.ld_y = a.ld_z = r.c;
  call("moe_layer_norm", [&] { return moe_layer_norm(&a, l.stream); });
  return {y, z, mean, rstd};
}

std::tuple<Tensor, OptTensor, OptTensor> layer_norm_backward(const Tensor& dy, const Tensor& z,
                                                            const OptTensor& weight, const Tensor& mean,
                                                            const Tensor& rstd, const OptTensor& dz,
                                                            bool bias) {
  const Rows r = rows_of(z, "z");
  const int dt = checked_type(z, "z");
  if (weight.has_value()) check_vector(*weight, "weight", r.c, z.scalar_type(), z);
  same_shape(dy, z.sizes(), z, "dy");
  const Rows rdy = rows_of(dy, "dy", r.c);
  Rows rdz{};
  if (dz.has_value()) {
    same_shape(*dz, z.sizes(), z, "dz");
    rdz = rows_of(*dz, "dz", r.c);
  }
  const auto shape = z.sizes().slice(0, z.dim() - 1);
  auto stat = [&](const Tensor& t, const char* what) {
    if (t.sizes() != shape || t.scalar_type() != at::kFloat || !t.is_contiguous() ||
        t.device() != z.device())
      refuse(what, " must be contiguous float32 of shape ", shape, ", got ", t.sizes(), " of ",
             t.scalar_type(), " on ", t.device());
  };
  stat(mean, "mean");
  stat(rstd, "rstd");
  const at::ScalarType wt = weight.has_value() ? weight->scalar_type() : z.scalar_type();
  const Launch l(z);
  Tensor dx = empty(z.sizes(), z.scalar_type(), z);
  OptTensor dw, db;
  if (weight.has_value()) dw = empty({r.c}, wt, z);
  if (bias) db = empty({r.c}, wt, z);
  const int D = as_int(r.c);
  const size_t size = moe_layer_norm_workspace(r.n, D);
  Tensor work = empty({(int64_t)size}, at::kByte, z);
  moe_norm_args a{};
  a.n = r.n;
  a.D = D;
  a.dtype = dt;
  a.wtype = type_of(wt);
  a.w = ptr(weight);
  a.z = z.data_ptr();
  a.mean = static_cast<float*>(mean.data_ptr());
  a.rstd = static_cast<float*>(rstd.data_ptr());
  a.dy = dy.data_ptr();
  a.dz = ptr(dz);
  a.dx = dx.data_ptr();
  a.dw = ptr(dw);
  a.db = ptr(db);
  a.ld_z = r.ld;
  a.ld_dy = rdy.ld;
  a.ld_dz = rdz.ld;
  a.ld_dx = r.c;
  call("moe_layer_norm_backward",
       [&] { return moe_layer_norm_backward(&a, work.data_ptr(), size, l.stream); });
  return {dx, dw, db};
}

// ------------------------------------------------------------------------------- linear
// The type named by a torch.dtype that is x's type or fp32, or `none` for None.
at::ScalarType x_or_fp32(const py::object& t, const char* what, const Tensor& x, at::ScalarType none) {
  if (t.is_none()) return none;
  if (THPDtype_Check(t.ptr())) {
    const at::ScalarType s = reinterpret_cast<THPDtype*>(t.ptr())->scalar_type;
    if (s == x.scalar_type() || s == at::kFloat) return s;
  }
  refuse(what, " ", std::string(py::str(t)), ": expected ", x.scalar_type(), " or float32");
}

std::tuple<Tensor, OptTensor> linear(const Tensor& x, const Tensor& weight, const OptTensor& bias,
                                     const std::string& act, const OptTensor& residual, bool preact,
                                     const py::object& out_dtype) {
  const int dt = checked_type(x, "x", true);
  const Rows rx = operand(x, "x", -1, x);
  if (weight.dim() != 2) refuse("weight must be [N, K], got ", weight.sizes());
  const Rows rw = operand(weight, "weight", rx.c, x);
  moe_linear_args a{};
  a.act = act_of(act);
  const at::ScalarType yt = x_or_fp32(out_dtype, "out_dtype", x, x.scalar_type());
  if (bias.has_value()) check_vector(*bias, "bias", rw.n, x.scalar_type(), x);
  const auto shape = with_last(x, rw.n);
  Rows rr{};
  if (residual.has_value()) {
    same_shape(*residual, shape, x, "residual");
    rr = rows_of(*residual, "residual", rw.n);
  }
  const Launch l(x);
  Tensor y = empty(shape, yt, x);
  OptTensor z;
  if (preact) z = empty(shape, x.scalar_type(), x);
  a.M = rx.n;
  a.N = rw.n;
  a.K = rx.c;
  a.dtype = a.dwtype = dt;
  a.ytype = type_of(yt);
  a.btype = bias.has_value() ? type_of(bias->scalar_type()) : dt;
  a.x = x.data_ptr();
  a.w = weight.data_ptr();
  a.b = ptr(bias);
  a.r = ptr(residual);
  a.y = y.data_ptr();
  a.z = ptr(z);
  a.ld_x = rx.ld;
  a.ld_w = rw.ld;
  a.ld_r = rr.ld;
  a.ld_y = a.ld_z = rw.n;
  call("moe_linear", [&] { return moe_linear(&a, l.stream); });
  return {y, z};
}

std::tuple<OptTensor, OptTensor, OptTensor> linear_backward(
    const Tensor& dy, const Tensor& x, const Tensor& weight, const OptTensor& z,
    const std::string& act, const py::object& bias, const py::object& dw_dtype, bool need_dx,
    bool need_dw) {
  const int dt = checked_type(x, "x", true);
  const Rows rx = operand(x, "x", -1, x);
  if (weight.dim() != 2) refuse("weight must be [N, K], got ", weight.sizes());
  const Rows rw = operand(weight, "weight", rx.c, x);
  moe_linear_args a{};
  a.act = act_of(act);
  if (z.has_value() == (a.act == MOE_ACT_NONE)) refuse("z is needed with an activation, and only then");
  const auto shape = with_last(x, rw.n);
  same_shape(dy, shape, x, "dy");
  const Rows rdy = rows_of(dy, "dy", rw.n);
  Rows rz{};
  if (z.has_value()) {
    same_shape(*z, shape, x, "z");
    rz = rows_of(*z, "z", rw.n);
  }
  const at::ScalarType wt = x_or_fp32(dw_dtype, "dw_dtype", x, x.scalar_type());
  const at::ScalarType bt = x_or_fp32(bias, "bias", x, at::ScalarType::Undefined);
  const Launch l(x);
  OptTensor dx, dw, db;
  if (need_dx) dx = empty(x.sizes(), x.scalar_type(), x);
  if (need_dw) dw = empty({rw.n, rx.c}, wt, x);
  if (bt != at::ScalarType::Undefined) db = empty({rw.n}, bt, x);
  const size_t size = moe_linear_workspace(rx.n, rw.n);
  Tensor work = empty({(int64_t)size}, at::kByte, x);
  a.M = rx.n;
  a.N = rw.n;
  a.K = rx.c;
  a.dtype = a.ytype = dt;
  a.btype = db.has_value() ? type_of(bt) : dt;
  a.dwtype = type_of(wt);
  a.x = x.data_ptr();
  a.w = weight.data_ptr();
  a.z = ptr(z);
  a.dy = dy.data_ptr();
  a.dx = ptr(dx);
  a.dw = ptr(dw);
  a.db = ptr(db);
  a.ld_x = rx.ld;
  a.ld_w = rw.ld;
  a.ld_z = rz.ld;
  a.ld_dy = rdy.ld;
  a.ld_dx = a.ld_dw = rx.c;
  call("moe_linear_backward", [&] { return moe_linear_backward(&a, work.data_ptr(), size, l.stream); });
  return {dx, dw, db};
}

}  // namespace

PYBIND11_MODULE(_torch_ops, m) {
  m.def("set_error", [](py::object e) { g_moe_error = e.release().ptr(); });
  m.def("route", torch::wrap_pybind_function(&route));
  m.def("route_plan", torch::wrap_pybind_function(&route_plan));
  m.def("route_backward", torch::wrap_pybind_function(&route_backward));
  m.def("layer_norm", torch::wrap_pybind_function(&layer_norm));
  m.def("layer_norm_backward", torch::wrap_pybind_function(&layer_norm_backward));
  m.def("linear", torch::wrap_pybind_function(&linear));
  m.def("linear_backward", torch::wrap_pybind_function(&linear_backward));
}
