// Native binding of the calls whose host time matters (token movement and FP8
// products, called many times per step on small batches): argument checks,
// output allocation and the C call without interpreter work in between.  The
// ctypes binding of the same C entry points takes 5 to 10 us more per call.
//
// Every function uses the current stream of its tensors' device.  A bad argument
// raises ValueError, a status other than NVFP4_OK the class given to set_error.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

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
    return at::empty(shape, at::TensorOptions().dtype(type).device(device));
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
  Tensor out = route_rows(on, {R, x.size(1)}, x.scalar_type(), off, PyObject_IsTrue(a[4]) == 1);
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
  Tensor dy = route_rows(on, y.sizes(), y.scalar_type(), off, PyObject_IsTrue(a[5]) == 1);
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

void check_product(const Tensor& x, int64_t K, const Tensor& w, const Tensor& scale, int dim) {
  need(w.dim() == dim && w.scalar_type() == at::kFloat8_e4m3fn && w.is_contiguous(),
       dim == 2 ? "w: expected contiguous float8_e4m3fn codes [N, K]"
                : "w: expected contiguous float8_e4m3fn codes [E, N, K]");
  need(scale.dim() == dim && scale.scalar_type() == at::kFloat && scale.is_contiguous() &&
           scale.size(dim - 1) == blocks(w.size(dim - 1)) &&
           scale.size(dim - 2) == blocks(w.size(dim - 2)) &&
           (dim == 2 || scale.size(0) == w.size(0)),
       "w_scale: expected contiguous FP32, one value per 128 x 128 block of w");
  need(K == w.size(dim - 1), "x: its columns are not the weights'");
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
  const int silu = PyObject_IsTrue(a[6]);
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
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods,
                        nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
