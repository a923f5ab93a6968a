// The operators on torch tensors: argument checks, output allocation and the calls of the
// C ABI (include/moe_tsg.h), as the functions of the Python module _torch_ops that ops.py
// documents. No computation here. In C++ because the host's part is what a small call costs:
// with the same checks in Python over ctypes it was 14 us (routing, linear), 19 (layer norm)
// and 24 to 32 (backward passes) on a Grace host, here 5 to 10, 6 to 12 and 11 to 18 by the machine.
#include <ATen/cuda/EmptyTensor.h>
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
// A tensor beside x (which is on a CUDA device), without the dispatcher: each is a good part of a
// small call's time.
Tensor empty(at::IntArrayRef shape, at::ScalarType type, const Tensor& x) {
  return Tensor(at::detail::empty_cuda(shape, type, x.device(), std::nullopt));
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

// Codes and scales of an 8-bit checkpoint.
void check_kept(const Tensor& codes, const Tensor& scales, const char* what, const Tensor& beside) {
  if (codes.scalar_type() != at::kFloat8_e4m3fn || codes.dim() < 1 || !codes.is_contiguous())
    refuse(what, "'s codes must be contiguous float8_e4m3fn, got ", codes.sizes(), " of ",
           codes.scalar_type());
  const auto shape = with_last(codes, (codes.size(-1) + 31) / 32);
  if (scales.scalar_type() != at::kByte || scales.sizes() != at::IntArrayRef(shape) ||
      !scales.is_contiguous())
    refuse(what, "'s scales must be contiguous uint8 of shape ", shape, ", got ", scales.sizes(), " of ",
           scales.scalar_type());
  same_device(codes, beside, what);
  same_device(scales, beside, what);
}
// A matrix from its checkpoint, on the stream of `l`.
Tensor restored(const Tensor& codes, const Tensor& scales, at::ScalarType type, const Launch& l) {
  Tensor x = empty(codes.sizes(), type, codes);
  const int64_t c = codes.size(-1);
  if (x.numel() == 0) return x;
  moe_checkpoint_args a{};
  a.n = codes.numel() / c;
  a.c = c;
  a.dtype = type_of(type);
  a.x = x.data_ptr();
  a.codes = codes.data_ptr();
  a.scales = static_cast<uint8_t*>(scales.data_ptr());
  a.ld_x = a.ld_codes = c;
  a.ld_scales = (c + 31) / 32;
  call("moe_restore", [&] { return moe_restore(&a, l.stream); });
  return x;
}

// x and z: matrices, or (with scales) the codes of their checkpoints.
std::tuple<OptTensor, OptTensor, OptTensor> linear_backward(
    const Tensor& dy, const Tensor& kept_x, const OptTensor& x_scales, const Tensor& weight,
    const OptTensor& z, const OptTensor& z_scales, const std::string& act, const py::object& bias,
    const py::object& dw_dtype, bool need_dx, bool need_dw) {
  const Tensor& x = x_scales.has_value() ? dy : kept_x;  // of the type and device that all have
  const int dt = checked_type(x, x_scales.has_value() ? "dy" : "x", true);
  Rows rx;
  if (x_scales.has_value()) {
    check_kept(kept_x, *x_scales, "x", dy);
    rx = rows_of(kept_x, "x");
    if (rx.c % 8 != 0) refuse("x has rows of ", rx.c, " elements: expected a multiple of 8 for a checkpoint");
  } else {
    rx = operand(x, "x", -1, x);
  }
  if (weight.dim() != 2) refuse("weight must be [N, K], got ", weight.sizes());
  const Rows rw = operand(weight, "weight", rx.c, x);
  moe_linear_args a{};
  a.act = act_of(act);
  if (z.has_value() == (a.act == MOE_ACT_NONE)) refuse("z is needed with an activation, and only then");
  const auto shape = with_last(kept_x, rw.n);
  same_shape(dy, shape, x, "dy");
  const Rows rdy = rows_of(dy, "dy", rw.n);
  Rows rz{};
  if (z_scales.has_value()) {
    check_kept(*z, *z_scales, "z", x);
    if (z->sizes() != at::IntArrayRef(shape)) refuse("z must be ", shape, ", got ", z->sizes());
    rz = {0, rw.n, rw.n};
  } else if (z.has_value()) {
    same_shape(*z, shape, x, "z");
    rz = rows_of(*z, "z", rw.n);
  }
  const at::ScalarType wt = x_or_fp32(dw_dtype, "dw_dtype", x, x.scalar_type());
  const at::ScalarType bt = x_or_fp32(bias, "bias", x, at::ScalarType::Undefined);
  const Launch l(x);
  OptTensor dx, dw, db;
  if (need_dx) dx = empty(kept_x.sizes(), x.scalar_type(), x);
  if (need_dw) dw = empty({rw.n, rx.c}, wt, x);
  if (bt != at::ScalarType::Undefined) db = empty({rw.n}, bt, x);
  const size_t size =
      moe_linear_workspace(rx.n, rw.n) + (x_scales.has_value() && need_dw ? moe_linear_kept_bytes(rx.n, rx.c) : 0);
  Tensor work = empty({(int64_t)size}, at::kByte, x);
  a.M = rx.n;
  a.N = rw.n;
  a.K = rx.c;
  a.dtype = a.ytype = dt;
  a.btype = db.has_value() ? type_of(bt) : dt;
  a.dwtype = type_of(wt);
  a.x = kept_x.data_ptr();
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
  a.z_scales = static_cast<const uint8_t*>(ptr(z_scales));
  a.x_scales = static_cast<const uint8_t*>(ptr(x_scales));
  call("moe_linear_backward", [&] { return moe_linear_backward(&a, work.data_ptr(), size, l.stream); });
  return {dx, dw, db};
}

// ------------------------------------------------------------------------------- expert rows
// The order of a batch: rows [..., topk] and offsets [E + 1].
struct Order {
  int64_t n, T, topk, E;
};
Order order_of(const Tensor& rows, const Tensor& offsets, const Tensor& beside) {
  if (rows.scalar_type() != at::kInt || rows.dim() < 1 || !rows.is_contiguous())
    refuse("the order's rows must be contiguous int32 [..., topk], got ", rows.sizes(), " of ",
           rows.scalar_type());
  if (offsets.scalar_type() != at::kInt || offsets.dim() != 1 || offsets.size(0) < 2 ||
      !offsets.is_contiguous())
    refuse("offsets must be contiguous int32 [E + 1], got ", offsets.sizes(), " of ",
           offsets.scalar_type());
  same_device(rows, beside, "the order");
  same_device(offsets, beside, "offsets");
  const int64_t topk = rows.size(-1);
  if (topk < 1 || topk > 32) refuse("the order's rows have ", topk, " choices: expected 1 to 32");
  return {rows.numel(), rows.numel() / topk, topk, offsets.size(0) - 1};
}
moe_rows_args rows_args(const Order& o, const Tensor& rows, const Tensor& offsets, int dtype, int64_t D) {
  moe_rows_args a{};
  a.T = o.T;
  a.D = D;
  a.topk = as_int(o.topk);
  a.E = as_int(o.E);
  a.dtype = dtype;
  a.rows = static_cast<const int32_t*>(rows.data_ptr());
  a.offsets = static_cast<const int32_t*>(offsets.data_ptr());
  return a;
}
void check_weights(const Tensor& w, const Tensor& rows) {
  if (w.scalar_type() != at::kFloat || w.sizes() != rows.sizes() || !w.is_contiguous() ||
      w.device() != rows.device())
    refuse("w must be contiguous float32 of shape ", rows.sizes(), " beside the order, got ", w.sizes(),
           " of ", w.scalar_type(), " on ", w.device());
}
void check_tokens(const Tensor& x, const Tensor& rows, const char* what) {
  if (x.dim() != rows.dim() || x.sizes().slice(0, x.dim() - 1) != rows.sizes().slice(0, rows.dim() - 1))
    refuse(what, " has shape ", x.sizes(), " for an order of rows ", rows.sizes());
}
// n rows of the matrix r.
Rows expert_matrix(const Tensor& r, const char* what, int64_t n) {
  const Rows m = rows_of(r, what);
  if (m.n != n) refuse(what, " has ", m.n, " rows: expected ", n, ", one for every slot");
  return m;
}

std::tuple<Tensor, Tensor, Tensor> sort_experts(const Tensor& ids, int64_t E) {
  if (ids.scalar_type() != at::kInt || ids.dim() < 1 || !ids.is_contiguous())
    refuse("ids must be contiguous int32 [..., topk], got ", ids.sizes(), " of ", ids.scalar_type());
  if (E < 1 || E > 1024) refuse("E is ", E, ": expected 1 to 1024");
  const Launch l(ids);
  const int64_t n = ids.numel();
  Tensor slots = empty({n}, at::kInt, ids), rows = empty(ids.sizes(), at::kInt, ids),
         offsets = empty({E + 1}, at::kInt, ids), work;
  const size_t size = moe_sort_experts_workspace(n, (int)E);
  if (size > 0) work = empty({(int64_t)size}, at::kByte, ids);
  call("moe_sort_experts", [&] {
    return moe_sort_experts(static_cast<const int32_t*>(ids.data_ptr()), n, (int)E,
                            static_cast<int32_t*>(slots.data_ptr()), static_cast<int32_t*>(rows.data_ptr()),
                            static_cast<int32_t*>(offsets.data_ptr()), size > 0 ? work.data_ptr() : nullptr,
                            size, l.stream);
  });
  return {slots, rows, offsets};
}

Tensor expert_rows(const Tensor& x, const Tensor& rows, const Tensor& offsets) {
  const Order o = order_of(rows, offsets, x);
  const Rows r = rows_of(x, "x");
  const int dt = checked_type(x, "x");
  check_tokens(x, rows, "x");
  const Launch l(x);
  Tensor out = empty({o.n, r.c}, x.scalar_type(), x);
  moe_rows_args a = rows_args(o, rows, offsets, dt, r.c);
  a.x = x.data_ptr();
  a.dr = out.data_ptr();
  a.ld_x = r.ld;
  a.ld_dr = r.c;
  call("moe_expert_rows", [&] { return moe_expert_rows(&a, l.stream); });
  return out;
}

Tensor combine_experts(const Tensor& r, const OptTensor& w, const Tensor& rows, const Tensor& offsets) {
  const Order o = order_of(rows, offsets, r);
  const int dt = checked_type(r, "r");
  const Rows m = expert_matrix(r, "r", o.n);
  if (w.has_value()) check_weights(*w, rows);
  const Launch l(r);
  Tensor y = empty(with_last(rows, m.c), r.scalar_type(), r);
  moe_rows_args a = rows_args(o, rows, offsets, dt, m.c);
  a.w = static_cast<const float*>(ptr(w));
  a.r = r.data_ptr();
  a.y = y.data_ptr();
  a.ld_r = m.ld;
  a.ld_y = m.c;
  call("moe_combine_experts", [&] { return moe_combine_experts(&a, l.stream); });
  return y;
}

std::tuple<Tensor, Tensor> combine_experts_backward(const Tensor& dy, const Tensor& r, const OptTensor& scales,
                                                    const OptTensor& weights, const Tensor& rows,
                                                    const Tensor& offsets) {
  if (!weights.has_value()) refuse("w is None: without weights the gradient of r is expert_rows(dy, order)");
  const Tensor& w = *weights;
  const Order o = order_of(rows, offsets, dy);
  const int dt = checked_type(dy, "dy");
  const Rows d = rows_of(dy, "dy");
  check_tokens(dy, rows, "dy");
  check_weights(w, rows);
  if (scales.has_value())
    check_kept(r, *scales, "r", dy);
  else if (r.scalar_type() != dy.scalar_type())
    refuse("r has type ", r.scalar_type(), ": expected ", dy.scalar_type(), " or a checkpoint");
  same_device(r, dy, "r");
  const Rows m = expert_matrix(r, "r", o.n);
  if (m.c != d.c) refuse("r has rows of ", m.c, " elements: expected ", d.c);
  const Launch l(dy);
  Tensor dr = empty({o.n, d.c}, dy.scalar_type(), dy), dw = empty(rows.sizes(), at::kFloat, dy);
  moe_rows_args a = rows_args(o, rows, offsets, dt, d.c);
  a.w = static_cast<const float*>(w.data_ptr());
  a.x = dy.data_ptr();
  a.r = r.data_ptr();
  a.r_scales = static_cast<const uint8_t*>(ptr(scales));
  a.dr = dr.data_ptr();
  a.dw = static_cast<float*>(dw.data_ptr());
  a.ld_x = d.ld;
  a.ld_r = m.ld;
  a.ld_scales = (d.c + 31) / 32;
  a.ld_dr = d.c;
  call("moe_combine_experts_backward", [&] { return moe_combine_experts_backward(&a, l.stream); });
  return {dr, dw};
}

// ------------------------------------------------------------------------------- expert linear
// Weights [E, N, K]: rows on 16 bytes, experts a multiple of 8 elements apart.
struct Experts {
  int64_t N, K, ld, stride;
};
Experts expert_weights(const Tensor& w, const Tensor& x, const Tensor& offsets) {
  if (offsets.scalar_type() != at::kInt || offsets.dim() != 1 || !offsets.is_contiguous() ||
      offsets.size(0) < 2)
    refuse("offsets must be contiguous int32 [E + 1], got ", offsets.sizes(), " of ", offsets.scalar_type());
  same_device(offsets, x, "offsets");
  if (w.dim() != 3 || w.size(0) != offsets.size(0) - 1)
    refuse("weight must be [E, N, K] with E = ", offsets.size(0) - 1, ", got ", w.sizes());
  if (w.scalar_type() != x.scalar_type())
    refuse("weight has type ", w.scalar_type(), ": expected ", x.scalar_type());
  same_device(w, x, "weight");
  const Experts e{w.size(1), w.size(2), w.stride(1), w.stride(0)};
  if (e.N % 8 != 0 || e.K % 8 != 0 || e.N < 1 || e.K < 1)
    refuse("weight must have N and K that are multiples of 8, got ", w.sizes());
  if (w.stride(2) != 1 || e.ld % 8 != 0 || e.ld < e.K ||
      (w.size(0) > 1 && (e.stride % 8 != 0 || e.stride < (e.N - 1) * e.ld + e.K)) ||
      reinterpret_cast<uintptr_t>(w.data_ptr()) % 16 != 0)
    refuse("weight must have contiguous rows that start on 16 bytes, got strides ", w.strides());
  return e;
}
moe_expert_linear_args expert_args(const Experts& e, const Tensor& w, const Tensor& offsets, int dtype,
                                   int64_t n) {
  moe_expert_linear_args a{};
  a.n = n;
  a.N = e.N;
  a.K = e.K;
  a.E = as_int(w.size(0));
  a.dtype = a.dwtype = dtype;
  a.offsets = static_cast<const int32_t*>(offsets.data_ptr());
  a.w = w.data_ptr();
  a.ld_w = e.ld;
  a.stride_w = e.stride;
  return a;
}

// A workspace of a call, which may need none.
struct Scratch {
  Tensor t;
  void* p = nullptr;
  size_t size;
  Scratch(size_t bytes, const Tensor& x) : size(bytes) {
    if (bytes == 0) return;
    t = empty({(int64_t)bytes}, at::kByte, x);
    p = t.data_ptr();
  }
};

Tensor expert_linear(const Tensor& x, const Tensor& weight, const Tensor& offsets) {
  const int dt = checked_type(x, "x", true);
  const Experts e = expert_weights(weight, x, offsets);
  const Rows r = operand(x, "x", e.K, x);
  const Launch l(x);
  Tensor y = empty(with_last(x, e.N), x.scalar_type(), x);
  moe_expert_linear_args a = expert_args(e, weight, offsets, dt, r.n);
  a.x = x.data_ptr();
  a.y = y.data_ptr();
  a.ld_x = r.ld;
  a.ld_y = e.N;
  const Scratch work(moe_expert_linear_workspace(a.n, a.N, a.K, a.E), x);
  call("moe_expert_linear", [&] { return moe_expert_linear(&a, work.p, work.size, l.stream); });
  return y;
}

// x: needed for dw alone.
std::tuple<OptTensor, OptTensor> expert_linear_backward(const Tensor& dy, const OptTensor& rows, const Tensor& weight,
                                                        const Tensor& offsets, const OptTensor& add,
                                                        const py::object& dw_dtype, bool need_dx, bool need_dw) {
  const int dt = checked_type(dy, "dy", true);
  const Experts e = expert_weights(weight, dy, offsets);
  const Rows d = operand(dy, "dy", e.N, dy);
  const auto shape = with_last(dy, e.K);
  Rows r{d.n, e.K, 0};
  if (rows.has_value()) {
    same_shape(*rows, shape, dy, "x");
    r = operand(*rows, "x", e.K, dy);
  } else if (need_dw) {
    refuse("x is needed for dweight");
  }
  const Tensor& x = dy;  // whose type and device all have
  Rows ra{};
  if (add.has_value()) {
    if (!need_dx) refuse("add is a part of dx, which is not asked for");
    same_shape(*add, shape, x, "add");
    ra = operand(*add, "add", e.K, x);
  }
  const at::ScalarType wt = x_or_fp32(dw_dtype, "dw_dtype", x, x.scalar_type());
  const Launch l(x);
  OptTensor dx, dw;
  moe_expert_linear_args a = expert_args(e, weight, offsets, dt, r.n);
  if (need_dx) dx = empty(shape, x.scalar_type(), x);
  if (need_dw) dw = empty(weight.sizes(), wt, x);
  a.dwtype = type_of(wt);
  a.x = ptr(rows);
  a.dy = dy.data_ptr();
  a.add = ptr(add);
  a.dx = ptr(dx);
  a.dw = ptr(dw);
  a.ld_x = r.ld;
  a.ld_dy = d.ld;
  a.ld_add = ra.ld;
  a.ld_dx = a.ld_dw = e.K;
  a.stride_dw = e.N * e.K;
  const Scratch work(need_dx ? moe_expert_linear_workspace(a.n, a.K, a.N, a.E) : 0, x);
  call("moe_expert_linear_backward",
       [&] { return moe_expert_linear_backward(&a, work.p, work.size, l.stream); });
  return {dx, dw};
}

// ------------------------------------------------------------------------------- checkpoints
std::tuple<Tensor, Tensor> checkpoint(const Tensor& x) {
  const Rows r = rows_of(x, "x");
  const int dt = checked_type(x, "x");
  const Launch l(x);
  Tensor codes = empty(x.sizes(), at::kFloat8_e4m3fn, x), scales = empty(with_last(x, (r.c + 31) / 32), at::kByte, x);
  if (x.numel() == 0) return {codes, scales};
  moe_checkpoint_args a{};
  a.n = r.n;
  a.c = r.c;
  a.dtype = dt;
  a.x = x.data_ptr();
  a.codes = codes.data_ptr();
  a.scales = static_cast<uint8_t*>(scales.data_ptr());
  a.ld_x = r.ld;
  a.ld_codes = r.c;
  a.ld_scales = (r.c + 31) / 32;
  call("moe_checkpoint", [&] { return moe_checkpoint(&a, l.stream); });
  return {codes, scales};
}

Tensor restore(const Tensor& codes, const Tensor& scales, const py::object& dtype) {
  check_kept(codes, scales, "the checkpoint", codes);
  at::ScalarType t = at::ScalarType::Undefined;
  if (THPDtype_Check(dtype.ptr())) t = reinterpret_cast<THPDtype*>(dtype.ptr())->scalar_type;
  if (type_of(t) < 0) refuse("dtype ", std::string(py::str(dtype)), ": expected bfloat16, float16 or float32");
  const Launch l(codes);
  return restored(codes, scales, t, l);
}

// ------------------------------------------------------------------------------- gated
moe_gated_args gated_args(const Tensor& beside, int64_t n, int64_t c, const std::string& act) {
  moe_gated_args a{};
  a.n = n;
  a.c = c;
  a.dtype = type_of(beside.scalar_type());
  a.act = act_of(act);
  return a;
}

std::tuple<Tensor, OptTensor, OptTensor, OptTensor, OptTensor> gated(const Tensor& gate, const Tensor& up,
                                                                    const std::string& act, bool keep) {
  checked_type(gate, "gate", true);
  const Rows g = rows_of(gate, "gate");
  same_shape(up, gate.sizes(), gate, "up");
  const Rows u = rows_of(up, "up", g.c);
  moe_gated_args a = gated_args(gate, g.n, g.c, act);
  const Launch l(gate);
  Tensor h = empty(gate.sizes(), gate.scalar_type(), gate);
  OptTensor gc, gs, uc, us;
  if (keep) {
    const auto blocks = with_last(gate, (g.c + 31) / 32);
    gc = empty(gate.sizes(), at::kFloat8_e4m3fn, gate);
    uc = empty(gate.sizes(), at::kFloat8_e4m3fn, gate);
    gs = empty(blocks, at::kByte, gate);
    us = empty(blocks, at::kByte, gate);
  }
  if (h.numel() == 0) return {h, gc, gs, uc, us};
  a.gate = gate.data_ptr();
  a.up = up.data_ptr();
  a.h = h.data_ptr();
  a.gate_codes = ptr(gc);
  a.up_codes = ptr(uc);
  a.gate_scales = static_cast<uint8_t*>(ptr(gs));
  a.up_scales = static_cast<uint8_t*>(ptr(us));
  a.ld_gate = g.ld;
  a.ld_up = u.ld;
  a.ld_h = g.c;
  call("moe_gated", [&] { return moe_gated(&a, l.stream); });
  return {h, gc, gs, uc, us};
}

std::tuple<Tensor, Tensor, OptTensor> gated_backward(const Tensor& dh, const Tensor& gate,
                                                     const OptTensor& gate_scales, const Tensor& up,
                                                     const OptTensor& up_scales, const std::string& act,
                                                     bool need_h) {
  checked_type(dh, "dh", true);
  const Rows d = rows_of(dh, "dh");
  if (gate_scales.has_value() != up_scales.has_value())
    refuse("gate and up must be both matrices or both checkpoints");
  Rows g{0, d.c, d.c}, u = g;
  if (gate_scales.has_value()) {
    check_kept(gate, *gate_scales, "gate", dh);
    check_kept(up, *up_scales, "up", dh);
    if (gate.sizes() != dh.sizes() || up.sizes() != dh.sizes())
      refuse("gate and up must be ", dh.sizes(), ", got ", gate.sizes(), " and ", up.sizes());
  } else {
    same_shape(gate, dh.sizes(), dh, "gate");
    same_shape(up, dh.sizes(), dh, "up");
    g = rows_of(gate, "gate", d.c);
    u = rows_of(up, "up", d.c);
  }
  moe_gated_args a = gated_args(dh, d.n, d.c, act);
  const Launch l(dh);
  Tensor dg = empty(dh.sizes(), dh.scalar_type(), dh), du = empty(dh.sizes(), dh.scalar_type(), dh);
  OptTensor h;
  if (need_h) h = empty(dh.sizes(), dh.scalar_type(), dh);
  if (dh.numel() == 0) return {dg, du, h};
  a.gate = gate.data_ptr();
  a.up = up.data_ptr();
  a.gate_scales = static_cast<uint8_t*>(ptr(gate_scales));
  a.up_scales = static_cast<uint8_t*>(ptr(up_scales));
  a.dh = dh.data_ptr();
  a.dgate = dg.data_ptr();
  a.dup = du.data_ptr();
  a.h = ptr(h);
  a.ld_gate = g.ld;
  a.ld_up = u.ld;
  a.ld_dh = d.ld;
  a.ld_dgate = a.ld_dup = a.ld_h = d.c;
  call("moe_gated_backward", [&] { return moe_gated_backward(&a, l.stream); });
  return {dg, du, h};
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
  m.def("sort_experts", torch::wrap_pybind_function(&sort_experts));
  m.def("expert_rows", torch::wrap_pybind_function(&expert_rows));
  m.def("combine_experts", torch::wrap_pybind_function(&combine_experts));
  m.def("combine_experts_backward", torch::wrap_pybind_function(&combine_experts_backward));
  m.def("expert_linear", torch::wrap_pybind_function(&expert_linear));
  m.def("expert_linear_backward", torch::wrap_pybind_function(&expert_linear_backward));
  m.def("checkpoint", torch::wrap_pybind_function(&checkpoint));
  m.def("restore", torch::wrap_pybind_function(&restore));
  m.def("gated", torch::wrap_pybind_function(&gated));
  m.def("gated_backward", torch::wrap_pybind_function(&gated_backward));
}
