// Native binding of the calls whose host time matters (token movement, FP8
// products, norms, gates and the MoE layer for a few tokens, called many times per
// step on small batches): argument checks,
// output allocation and the C call without interpreter work in between.  The
// ctypes binding of the same C entry points takes 5 to 10 us more per call.
//
// Every function uses the current stream of its tensors' device.  A bad argument
// raises ValueError, a status other than NVFP4_OK the class given to set_error.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/Context.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <initializer_list>
#include <optional>
#include <stdexcept>
#include <string>

#include "../../include/nvfp4.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;      // class (name, status) of failed calls

struct BadArg : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct Failed {
  const char* name;
  int status;
};

void need(bool ok, const char* what) {
  if (!ok) throw BadArg(what);
}

const Tensor& tensor(PyObject* o, const char* what) {
  need(THPVariable_Check(o), what);
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw BadArg("expected an integer");
  }
  return v;
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw BadArg("expected a number");
  }
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    throw BadArg("expected true or false");
  }
  return v != 0;
}

int dtype_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return NVFP4_BF16;
    case at::kHalf: return NVFP4_FP16;
    case at::kFloat: return NVFP4_FP32;
    default: throw BadArg("expected BF16, FP16 or FP32 rows");
  }
}

// The device of every tensor of a call, as the current one.
struct On {
  c10::cuda::OptionalCUDAGuard guard;
  c10::Device device;
  explicit On(const Tensor& t) : device(t.device()) {
    need(t.is_cuda(), "expected a CUDA tensor");
    guard.set_device(device);
  }
  void same(const Tensor& t) const { need(t.device() == device, "tensors on different devices"); }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }
  Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    // Past the dispatcher (0.5 us less an output), but where torch takes part in allocations:
    // dispatch modes, and the fill of uninitialised memory of deterministic algorithms.
    const at::Context& torch = at::globalContext();
    if (c10::impl::TorchDispatchModeTLS::any_modes_set() ||
        (torch.deterministicAlgorithms() && torch.deterministicFillUninitializedMemory()))
      return at::empty(shape, at::TensorOptions().dtype(type).device(device));
    return at::detail::empty_cuda(shape, type, device, std::nullopt);
  }
};

// Rows [n, D] whose elements are neighbours (a copy only where they are not).
Tensor rows_of(const Tensor& t) {
  need(t.dim() == 2, "expected rows [n, D]");
  const int64_t n = t.size(0), D = t.size(1);
  need(D > 0, "rows of width 0");
  if ((D > 1 && t.stride(1) != 1) || (n > 1 && t.stride(0) < D)) return t.contiguous();
  return t;
}
// The same, with base and row stride multiples of 16 bytes (16-bit types).
Tensor rows16_of(const Tensor& t) {
  Tensor r = rows_of(t);
  if ((reinterpret_cast<uintptr_t>(r.data_ptr()) & 15u) || (r.size(0) > 1 && r.stride(0) % 8))
    return r.clone(at::MemoryFormat::Contiguous);
  return r;
}
int64_t row_stride(const Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

const int32_t* routes(const Tensor& pos) {
  need(pos.dim() == 2 && pos.size(1) > 0 && pos.scalar_type() == at::kInt && pos.is_contiguous(),
       "route_pos: expected contiguous int32 [T, topk]");
  return static_cast<const int32_t*>(pos.data_ptr());
}

// expert_offsets or None: pointer and E.
const int32_t* offsets(const On& on, PyObject* o, int* E) {
  *E = 0;
  if (o == Py_None) return nullptr;
  const Tensor& t = tensor(o, "expert_offsets: expected a tensor");
  need(t.dim() == 1 && t.numel() >= 2 && t.scalar_type() == at::kInt && t.is_contiguous(),
       "expert_offsets: expected contiguous int32 [E + 1]");
  on.same(t);
  *E = static_cast<int>(t.numel() - 1);
  return static_cast<const int32_t*>(t.data_ptr());
}

Tensor weights_of(const On& on, const Tensor& w, const Tensor& pos) {
  need(w.sizes() == pos.sizes() && w.scalar_type() == at::kFloat,
       "weights: expected FP32 of route_pos' shape");
  on.same(w);
  return w.contiguous();
}

void check(const char* name, int status) {
  if (status != NVFP4_OK) throw Failed{name, status};
}

PyObject* give(Tensor t) { return THPVariable_Wrap(std::move(t)); }

// Route-ordered rows for a kernel to write.  `zero`: rows that no route names are
// zero; with expert_offsets the kernel zeroes them, without them nothing says
// which rows those are, so all are.
Tensor route_rows(const On& on, at::IntArrayRef shape, at::ScalarType type, const int32_t* off,
                  bool zero) {
  Tensor t = on.empty(shape, type);
  if (zero && !off) t.zero_();
  return t;
}

// dispatch(x, route_pos, expert_offsets | None, R | -1, zero) -> [R, D]
PyObject* dispatch(PyObject* const* a) {
  Tensor x = tensor(a[0], "x: expected a tensor");
  const Tensor& pos = tensor(a[1], "route_pos: expected a tensor");
  const int32_t* p = routes(pos);
  need(x.dim() == 2 && x.size(0) == pos.size(0), "x: expected as many rows as route_pos");
  const int type = dtype_of(x);
  const On on(x);
  on.same(pos);
  int E;
  const int32_t* off = offsets(on, a[2], &E);
  x = rows_of(x);
  int64_t R = integer(a[3]);
  if (R < 0) R = pos.numel();
  Tensor out = route_rows(on, {R, x.size(1)}, x.scalar_type(), off, truth(a[4]));
  check("nvfp4_tokens_dispatch",
        nvfp4_tokens_dispatch(x.data_ptr(), row_stride(x), p, off, E, pos.size(0),
                              static_cast<int32_t>(pos.size(1)), R, x.size(1), type,
                              out.data_ptr(), on.stream()));
  return give(std::move(out));
}

// combine(y, route_pos, weights | None) -> [T, D]
PyObject* combine(PyObject* const* a) {
  Tensor y = tensor(a[0], "y: expected a tensor");
  const Tensor& pos = tensor(a[1], "route_pos: expected a tensor");
  const int32_t* p = routes(pos);
  const int type = dtype_of(y);
  Tensor w;
  if (a[2] != Py_None) w = tensor(a[2], "weights: expected a tensor");
  if (w.defined())
    need(w.sizes() == pos.sizes() && w.scalar_type() == at::kFloat,
         "weights: expected FP32 of route_pos' shape");
  need(y.dim() == 2, "y: expected rows [R, D]");
  const On on(y);
  on.same(pos);
  if (w.defined()) w = weights_of(on, w, pos);
  y = rows_of(y);
  Tensor out = on.empty({pos.size(0), y.size(1)}, y.scalar_type());
  check("nvfp4_tokens_combine",
        nvfp4_tokens_combine(y.data_ptr(), row_stride(y), p,
                             w.defined() ? static_cast<const float*>(w.data_ptr()) : nullptr,
                             pos.size(0), static_cast<int32_t>(pos.size(1)), y.size(0), y.size(1),
                             type, out.data_ptr(), on.stream()));
  return give(std::move(out));
}

// combine_grad(dout, y, route_pos, weights, expert_offsets | None, zero) -> (dy, dw)
PyObject* combine_grad(PyObject* const* a) {
  Tensor dout = tensor(a[0], "dout: expected a tensor");
  Tensor y = tensor(a[1], "y: expected a tensor");
  const Tensor& pos = tensor(a[2], "route_pos: expected a tensor");
  const int32_t* p = routes(pos);
  Tensor w = tensor(a[3], "weights: expected a tensor");
  need(w.sizes() == pos.sizes() && w.scalar_type() == at::kFloat,
       "weights: expected FP32 of route_pos' shape");
  need(y.dim() == 2 && dout.dim() == 2 && dout.size(0) == pos.size(0) &&
           dout.size(1) == y.size(1) && dout.scalar_type() == y.scalar_type(),
       "dout: expected [T, D] of y's width and type");
  const int type = dtype_of(dout);
  const On on(y);
  on.same(pos);
  on.same(dout);
  w = weights_of(on, w, pos);
  int E;
  const int32_t* off = offsets(on, a[4], &E);
  dout = rows_of(dout);
  y = rows_of(y);
  Tensor dy = route_rows(on, y.sizes(), y.scalar_type(), off, truth(a[5]));
  Tensor dw = on.empty(pos.sizes(), at::kFloat);
  check("nvfp4_tokens_combine_grad",
        nvfp4_tokens_combine_grad(dout.data_ptr(), row_stride(dout), y.data_ptr(), row_stride(y), p,
                                  static_cast<const float*>(w.data_ptr()), off, E, pos.size(0),
                                  static_cast<int32_t>(pos.size(1)), y.size(0), y.size(1), type,
                                  dy.data_ptr(), static_cast<float*>(dw.data_ptr()), on.stream()));
  PyObject* both = PyTuple_New(2);
  if (!both) return nullptr;
  PyTuple_SET_ITEM(both, 0, give(std::move(dy)));
  PyTuple_SET_ITEM(both, 1, give(std::move(dw)));
  return both;
}

int64_t blocks(int64_t n) { return (n + 127) / 128; }

void check_weights(int64_t K, const Tensor& w, const Tensor& scale, int dim) {
  need(w.dim() == dim && w.scalar_type() == at::kFloat8_e4m3fn && w.is_contiguous(),
       dim == 2 ? "w: expected contiguous float8_e4m3fn codes [N, K]"
                : "w: expected contiguous float8_e4m3fn codes [E, N, K]");
  need(scale.dim() == dim && scale.scalar_type() == at::kFloat && scale.is_contiguous() &&
           scale.size(dim - 1) == blocks(w.size(dim - 1)) &&
           scale.size(dim - 2) == blocks(w.size(dim - 2)) &&
           (dim == 2 || scale.size(0) == w.size(0)),
       "w_scale: expected contiguous FP32, one value per 128 x 128 block of w");
  need(K == w.size(dim - 1), "x: its columns are not the weights'");
}
void check_product(const Tensor& x, int64_t K, const Tensor& w, const Tensor& scale, int dim) {
  check_weights(K, w, scale, dim);
  need(x.scalar_type() == at::kBFloat16 || x.scalar_type() == at::kHalf,
       "x: expected BF16 or FP16");
}

// The products take no part in autograd; losing a gradient silently is worse than an
// error.  (torch.nn.Parameter requires a gradient unless told not to, scales and
// codes too.)
void no_gradient(const Tensor& x, const Tensor& w, const Tensor& scale) {
  if (c10::GradMode::is_enabled() &&
      (x.requires_grad() || w.requires_grad() || scale.requires_grad()))
    throw std::runtime_error(
        "FP8 products are not differentiable by themselves: call them in an autograd.Function "
        "(the gradient is the product with transpose_weights; the weights are frozen) or under "
        "no_grad");
}

// linear(x, w, w_scale) -> [M, N]; x [M, K]
PyObject* linear(PyObject* const* a) {
  Tensor x = tensor(a[0], "x: expected a tensor");
  const Tensor& w = tensor(a[1], "w: expected a tensor");
  const Tensor& scale = tensor(a[2], "w_scale: expected a tensor");
  no_gradient(x, w, scale);
  need(x.dim() == 2, "x: expected rows [M, K]");
  check_product(x, x.size(1), w, scale, 2);
  const On on(x);
  on.same(w);
  on.same(scale);
  x = rows16_of(x);
  const int64_t M = x.size(0), N = w.size(0), K = x.size(1);
  Tensor y = on.empty({M, N}, x.scalar_type());
  const size_t bytes = nvfp4_fp8_linear_workspace_bytes(M, K);
  Tensor ws = on.empty({static_cast<int64_t>(bytes)}, at::kByte);
  check("nvfp4_fp8_linear",
        nvfp4_fp8_linear(x.data_ptr(), M, row_stride(x), dtype_of(x),
                         static_cast<const uint8_t*>(w.data_ptr()),
                         static_cast<const float*>(scale.data_ptr()), N, K, y.data_ptr(), N,
                         ws.data_ptr(), bytes, on.stream()));
  return give(std::move(y));
}

// expert_linear(x, w, w_scale, expert_offsets, route_pos | None, R | -1, silu_mul) -> [R, N]
PyObject* expert_linear(PyObject* const* a) {
  Tensor x = tensor(a[0], "x: expected a tensor");
  const Tensor& w = tensor(a[1], "w: expected a tensor");
  const Tensor& scale = tensor(a[2], "w_scale: expected a tensor");
  no_gradient(x, w, scale);
  const bool silu = truth(a[6]);
  need(x.dim() == 2, "x: expected rows");
  const int64_t K = silu ? x.size(1) / 2 : x.size(1);
  need(!silu || x.size(1) % 2 == 0, "x: gate and up halves of one width");
  check_product(x, K, w, scale, 3);
  const Tensor& off = tensor(a[3], "expert_offsets: expected a tensor");
  need(off.dim() == 1 && off.size(0) == w.size(0) + 1 && off.scalar_type() == at::kInt &&
           off.is_contiguous(),
       "expert_offsets: expected contiguous int32 [E + 1]");
  const int32_t* p = nullptr;
  int64_t fanout = 1, R = integer(a[5]);
  if (a[4] != Py_None) {
    const Tensor& pos = tensor(a[4], "route_pos: expected a tensor");
    p = routes(pos);
    need(pos.size(0) == x.size(0), "x: expected as many rows as route_pos");
    fanout = pos.size(1);
    if (R < 0) R = pos.numel();
  } else {
    need(R < 0 || R == x.size(0), "R: without route_pos, the rows of x");
    R = x.size(0);
  }
  const On on(x);
  on.same(w);
  on.same(scale);
  on.same(off);
  if (p) on.same(THPVariable_Unpack(a[4]));
  x = rows16_of(x);
  const int64_t N = w.size(1);
  Tensor y = on.empty({R, N}, x.scalar_type());
  const size_t bytes = nvfp4_fp8_linear_workspace_bytes(R, K);
  Tensor ws = on.empty({static_cast<int64_t>(bytes)}, at::kByte);
  check("nvfp4_fp8_expert_linear",
        nvfp4_fp8_expert_linear(x.data_ptr(), x.size(0), row_stride(x), dtype_of(x),
                                silu ? NVFP4_FP8_SILU_MUL : 0u, p, static_cast<int32_t>(fanout),
                                static_cast<const uint8_t*>(w.data_ptr()),
                                static_cast<const float*>(scale.data_ptr()),
                                static_cast<const int32_t*>(off.data_ptr()),
                                static_cast<int32_t>(w.size(0)), R, N, K, y.data_ptr(), N,
                                ws.data_ptr(), bytes, on.stream()));
  return give(std::move(y));
}

// linear_codes(codes, scales, w, w_scale, nvfp4_dtype) -> [M, N]
PyObject* linear_codes(PyObject* const* a) {
  const Tensor& q = tensor(a[0], "codes: expected a tensor");
  const Tensor& sq = tensor(a[1], "scales: expected a tensor");
  const Tensor& w = tensor(a[2], "w: expected a tensor");
  const Tensor& scale = tensor(a[3], "w_scale: expected a tensor");
  const int64_t type = integer(a[4]);
  no_gradient(sq, w, scale);
  need(q.dim() == 2 && q.scalar_type() == at::kFloat8_e4m3fn && q.is_contiguous() && q.size(1) > 0,
       "codes: expected contiguous float8_e4m3fn [M, K]");
  const int64_t M = q.size(0), K = q.size(1);
  need(sq.dim() == 2 && sq.scalar_type() == at::kFloat && sq.is_contiguous() &&
           sq.size(0) == blocks(K) && sq.size(1) == M,
       "scales: expected contiguous FP32 [ceil(K / 128), M]");
  check_weights(K, w, scale, 2);
  const On on(q);
  on.same(sq);
  on.same(w);
  on.same(scale);
  const int64_t N = w.size(0);
  Tensor y = on.empty({M, N}, type == NVFP4_FP32   ? at::kFloat
                              : type == NVFP4_FP16 ? at::kHalf
                                                   : at::kBFloat16);
  check("nvfp4_fp8_gemm",
        nvfp4_fp8_gemm(static_cast<const uint8_t*>(q.data_ptr()),
                       static_cast<const float*>(sq.data_ptr()),
                       static_cast<const uint8_t*>(w.data_ptr()),
                       static_cast<const float*>(scale.data_ptr()), y.data_ptr(), M, N, K, N,
                       static_cast<int32_t>(type), on.stream()));
  return give(std::move(y));
}

PyObject* give(std::initializer_list<Tensor> ts) {
  PyObject* all = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!all) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) PyTuple_SET_ITEM(all, i++, give(t));
  return all;
}

// Weight of a norm over rows of width D.
Tensor norm_weight(const On& on, PyObject* o, const Tensor& x) {
  Tensor w = tensor(o, "weight: expected a tensor");
  need(w.dim() == 1 && w.size(0) == x.size(1) &&
           (w.scalar_type() == x.scalar_type() || w.scalar_type() == at::kFloat),
       "weight: expected [D] of the rows' type or FP32");
  on.same(w);
  return w.contiguous();
}

// Rows that lie where a dense matrix's do within 16 bytes (a copy where they do not).
Tensor norm_rows(const Tensor& t) {
  Tensor r = rows_of(t);
  const int64_t es = static_cast<int64_t>(r.element_size());
  if ((reinterpret_cast<uintptr_t>(r.data_ptr()) & 15u) ||
      (r.size(0) > 1 && (r.stride(0) - r.size(1)) * es % 16))
    return r.clone(at::MemoryFormat::Contiguous);
  return r;
}

// A second operand of x's shape and type, or None.
Tensor like_rows(const On& on, PyObject* o, const Tensor& x, const char* what) {
  if (o == Py_None) return {};
  const Tensor& t = tensor(o, what);
  need(t.sizes() == x.sizes() && t.scalar_type() == x.scalar_type(), what);
  on.same(t);
  return norm_rows(t);
}
Tensor aligned_rows(const Tensor& t) { return t.defined() ? rows16_of(t) : t; }
const void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
int64_t stride_or_0(const Tensor& t) { return t.defined() ? row_stride(t) : 0; }

float epsilon(PyObject* o) {
  const float eps = static_cast<float>(real(o));
  need(eps >= 0.f, "eps: expected a number >= 0");
  return eps;
}

// rms_norm(x, weight, residual | None, eps, fp8) -> (y, h) or (codes, scales, h);
// without a residual no h
PyObject* rms_norm(PyObject* const* a) {
  Tensor x = tensor(a[0], "x: expected a tensor");
  need(x.dim() == 2 && x.size(1) > 0, "x: expected rows [T, D]");
  const int type = dtype_of(x);
  const float eps = epsilon(a[3]);
  const bool fp8 = truth(a[4]);
  const On on(x);
  Tensor w = norm_weight(on, a[1], x);
  Tensor r = like_rows(on, a[2], x, "residual: expected rows of x's shape and type");
  x = norm_rows(x);
  const int64_t T = x.size(0), D = x.size(1);
  Tensor h;
  if (r.defined()) h = on.empty({T, D}, x.scalar_type());
  if (fp8) {
    need(type != NVFP4_FP32 && D % 16 == 0,
         "x: expected BF16 or FP16 rows whose width is a multiple of 16");
    x = rows16_of(x);
    r = aligned_rows(r);
    if (reinterpret_cast<uintptr_t>(w.data_ptr()) & 15u) w = w.clone();
    Tensor codes = on.empty({T, D}, at::kFloat8_e4m3fn);
    Tensor scales = on.empty({blocks(D), T}, at::kFloat);
    check("nvfp4_rms_norm_fp8",
          nvfp4_rms_norm_fp8(x.data_ptr(), row_stride(x), ptr(r), stride_or_0(r), T, D, type,
                             w.data_ptr(), dtype_of(w), eps, h.defined() ? h.data_ptr() : nullptr,
                             static_cast<uint8_t*>(codes.data_ptr()),
                             static_cast<float*>(scales.data_ptr()), on.stream()));
    return h.defined() ? give({codes, scales, h}) : give({codes, scales});
  }
  Tensor y = on.empty({T, D}, x.scalar_type());
  check("nvfp4_rms_norm",
        nvfp4_rms_norm(x.data_ptr(), row_stride(x), ptr(r), stride_or_0(r), T, D, type,
                       w.data_ptr(), dtype_of(w), eps, h.defined() ? h.data_ptr() : nullptr,
                       y.data_ptr(), on.stream()));
  return h.defined() ? give({y, h}) : give({y});
}

// rms_norm_grad(dy, h, weight, dh | None, eps) -> (dx, dweight)
PyObject* rms_norm_grad(PyObject* const* a) {
  Tensor h = tensor(a[1], "h: expected a tensor");
  need(h.dim() == 2 && h.size(1) > 0, "h: expected rows [T, D]");
  const int type = dtype_of(h);
  const float eps = epsilon(a[4]);
  const On on(h);
  need(a[0] != Py_None, "dy: expected rows of h's shape and type");
  Tensor dy = like_rows(on, a[0], h, "dy: expected rows of h's shape and type");
  Tensor w = norm_weight(on, a[2], h);
  Tensor dh = like_rows(on, a[3], h, "dh: expected rows of h's shape and type");
  h = norm_rows(h);
  const int64_t T = h.size(0), D = h.size(1);
  Tensor dx = on.empty({T, D}, h.scalar_type());
  Tensor dw = on.empty({D}, w.scalar_type());
  const size_t bytes = nvfp4_rms_norm_grad_workspace_bytes(T, D);
  Tensor ws = on.empty({static_cast<int64_t>(bytes)}, at::kByte);
  check("nvfp4_rms_norm_grad",
        nvfp4_rms_norm_grad(dy.data_ptr(), row_stride(dy), h.data_ptr(), row_stride(h), ptr(dh),
                            stride_or_0(dh), T, D, type, w.data_ptr(), dtype_of(w), eps,
                            dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), bytes, on.stream()));
  return give({dx, dw});
}

// flags from (sigmoid, renormalize)
uint32_t gate_flags(PyObject* sigmoid, PyObject* renormalize) {
  return (truth(sigmoid) ? NVFP4_GATE_SIGMOID : 0u) |
         (truth(renormalize) ? NVFP4_GATE_RENORMALIZE : 0u);
}

Tensor gate_bias(const On& on, PyObject* o, int64_t E) {
  if (o == Py_None) return {};
  const Tensor& b = tensor(o, "bias: expected a tensor");
  need(b.dim() == 1 && b.size(0) == E && b.scalar_type() == at::kFloat, "bias: expected FP32 [E]");
  on.same(b);
  return b.contiguous();
}

int32_t gate_topk(PyObject* o, int64_t E) {
  const int64_t k = integer(o);
  need(k > 0 && k <= E, "topk: expected 1 to E experts");
  return static_cast<int32_t>(k < 1 << 20 ? k : 1 << 20);
}

// topk_gate(logits, topk, bias | None, sigmoid, renormalize, scale) -> (ids, weights)
PyObject* topk_gate(PyObject* const* a) {
  Tensor l = tensor(a[0], "logits: expected a tensor");
  need(l.dim() == 2 && l.size(1) > 0, "logits: expected [T, E]");
  const int type = dtype_of(l);
  const int64_t T = l.size(0), E = l.size(1);
  const int32_t k = gate_topk(a[1], E);
  const On on(l);
  const Tensor bias = gate_bias(on, a[2], E);
  l = rows_of(l);
  Tensor ids = on.empty({T, k}, at::kInt), w = on.empty({T, k}, at::kFloat);
  check("nvfp4_topk_gate",
        nvfp4_topk_gate(l.data_ptr(), row_stride(l), T, static_cast<int32_t>(E < 1 << 30 ? E : 1 << 30),
                        type, k, static_cast<const float*>(ptr(bias)), gate_flags(a[3], a[4]),
                        static_cast<float>(real(a[5])), static_cast<int32_t*>(ids.data_ptr()),
                        static_cast<float*>(w.data_ptr()), on.stream()));
  return give({ids, w});
}

const Tensor& chosen(const On& on, PyObject* o, int64_t T) {
  const Tensor& ids = tensor(o, "topk_ids: expected a tensor");
  need(ids.dim() == 2 && ids.size(0) == T && ids.size(1) > 0 && ids.scalar_type() == at::kInt &&
           ids.is_contiguous(),
       "topk_ids: expected contiguous int32 [T, topk]");
  on.same(ids);
  return ids;
}

// topk_gate_grad(dweights, logits, ids, sigmoid, renormalize, scale) -> dlogits
PyObject* topk_gate_grad(PyObject* const* a) {
  Tensor l = tensor(a[1], "logits: expected a tensor");
  need(l.dim() == 2 && l.size(1) > 0, "logits: expected [T, E]");
  const int type = dtype_of(l);
  const int64_t T = l.size(0), E = l.size(1);
  const On on(l);
  const Tensor& ids = chosen(on, a[2], T);
  Tensor dw = tensor(a[0], "dweights: expected a tensor");
  need(dw.sizes() == ids.sizes() && dw.scalar_type() == at::kFloat,
       "dweights: expected FP32 of topk_ids' shape");
  on.same(dw);
  dw = dw.contiguous();
  l = rows_of(l);
  Tensor dl = on.empty({T, E}, l.scalar_type());
  check("nvfp4_topk_gate_grad",
        nvfp4_topk_gate_grad(static_cast<const float*>(dw.data_ptr()), l.data_ptr(), row_stride(l),
                             T, static_cast<int32_t>(E < 1 << 30 ? E : 1 << 30), type,
                             static_cast<int32_t>(ids.size(1)),
                             static_cast<const int32_t*>(ids.data_ptr()), gate_flags(a[3], a[4]),
                             static_cast<float>(real(a[5])), dl.data_ptr(), on.stream()));
  return give(std::move(dl));
}

// moe_layer(x, router | None, gate_up, gate_up_scale, down, down_scale, topk, bias | None,
//           sigmoid, renormalize, scale, ids | None, weights | None)
//   -> (out, ids, weights), or None for more tokens than the call takes
PyObject* moe_layer(PyObject* const* a) {
  Tensor x = tensor(a[0], "x: expected a tensor");
  const Tensor& w1 = tensor(a[2], "gate_up: expected a tensor");
  const Tensor& s1 = tensor(a[3], "gate_up scales: expected a tensor");
  const Tensor& w2 = tensor(a[4], "down: expected a tensor");
  const Tensor& s2 = tensor(a[5], "down scales: expected a tensor");
  no_gradient(x, w1, s1);
  no_gradient(x, w2, s2);
  need(x.dim() == 2, "x: expected rows [T, K]");
  check_product(x, x.size(1), w1, s1, 3);
  need(w1.size(1) % 2 == 0, "gate_up: gate and up halves of one width");
  const int64_t T = x.size(0), K = x.size(1), E = w1.size(0), I = w1.size(1) / 2;
  check_weights(I, w2, s2, 3);
  need(w2.size(0) == E, "down: expected as many experts as gate_up");
  const int64_t N = w2.size(1);
  const On on(x);
  on.same(w1);
  on.same(s1);
  on.same(w2);
  on.same(s2);
  Tensor router, bias, ids, weights;
  int32_t k;
  uint32_t flags = 0;
  float scale = 1.f;
  if (a[1] != Py_None) {
    router = tensor(a[1], "router: expected a tensor");
    need(router.dim() == 2 && router.size(0) == E && router.size(1) == K &&
             (router.scalar_type() == x.scalar_type() || router.scalar_type() == at::kFloat),
         "router: expected [E, K] of x's type or FP32");
    no_gradient(router, w1, s1);
    on.same(router);
    k = gate_topk(a[6], E);
    bias = gate_bias(on, a[7], E);
    flags = gate_flags(a[8], a[9]);
    scale = static_cast<float>(real(a[10]));
  } else {
    ids = chosen(on, a[11], T);
    weights = tensor(a[12], "topk_weights: expected a tensor");
    need(weights.sizes() == ids.sizes() && weights.scalar_type() == at::kFloat,
         "topk_weights: expected FP32 of topk_ids' shape");
    no_gradient(weights, w1, s1);
    on.same(weights);
    weights = weights.contiguous();
    need(ids.size(1) <= 1 << 20, "topk_ids: too many routes");
    k = static_cast<int32_t>(ids.size(1));
  }
  const size_t bytes = T == 0 ? 0
                              : nvfp4_fp8_moe_layer_workspace_bytes(T, k, static_cast<int32_t>(E), K,
                                                                    I, N);
  if (bytes == 0) Py_RETURN_NONE;
  x = rows16_of(x);
  if (router.defined()) {
    router = router.contiguous();
    if (reinterpret_cast<uintptr_t>(router.data_ptr()) & 15u) router = router.clone();
    ids = on.empty({T, k}, at::kInt);
    weights = on.empty({T, k}, at::kFloat);
  }
  Tensor out = on.empty({T, N}, x.scalar_type());
  Tensor ws = on.empty({static_cast<int64_t>(bytes)}, at::kByte);
  check("nvfp4_fp8_moe_layer",
        nvfp4_fp8_moe_layer(x.data_ptr(), row_stride(x), T, dtype_of(x), ptr(router),
                            router.defined() ? dtype_of(router) : dtype_of(x),
                            static_cast<const float*>(ptr(bias)), flags, scale,
                            static_cast<const uint8_t*>(w1.data_ptr()),
                            static_cast<const float*>(s1.data_ptr()),
                            static_cast<const uint8_t*>(w2.data_ptr()),
                            static_cast<const float*>(s2.data_ptr()), static_cast<int32_t>(E), k, K,
                            I, N, static_cast<int32_t*>(ids.data_ptr()),
                            static_cast<float*>(weights.data_ptr()), out.data_ptr(), N,
                            ws.data_ptr(), bytes, on.stream()));
  return give({out, ids, weights});
}

// No C++ exception leaves a Python entry.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const BadArg& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const Failed& f) {
    PyObject* e = g_error ? PyObject_CallFunction(g_error, "si", f.name, f.status) : nullptr;
    if (e) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
      PyErr_Format(PyExc_RuntimeError, "%s failed (%d)", f.name, f.status);
    }
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* cls = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    PyErr_Clear();
    PyErr_SetString(cls ? cls : PyExc_MemoryError, e.what_without_backtrace());
    Py_XDECREF(cls);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<dispatch, 5>("dispatch"),
    method<combine, 3>("combine"),
    method<combine_grad, 6>("combine_grad"),
    method<linear, 3>("linear"),
    method<expert_linear, 7>("expert_linear"),
    method<linear_codes, 5>("linear_codes"),
    method<rms_norm, 5>("rms_norm"),
    method<rms_norm_grad, 5>("rms_norm_grad"),
    method<topk_gate, 6>("topk_gate"),
    method<topk_gate_grad, 6>("topk_gate_grad"),
    method<moe_layer, 13>("moe_layer"),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods,
                        nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
