// rowops_binding.cpp -- the allocation helpers of the row operators as a Python extension.
//
// A row operator on a few tokens takes 1.5 to 3 us on the device; checking its tensors,
// allocating its outputs and marshalling its arguments in Python took 11 to 40 us.  Here the
// same steps are compiled: check, at::empty, one call of the C ABI.  The entry points' addresses
// are handed over by bind(), so that this module and the ctypes binding use the same loaded
// library.  Arguments are positional (the Python helpers give them names and defaults).
#include <ATen/ATen.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <optional>
#include <vector>

#include "fp8q.h"

namespace {

#define FP8Q_ENTRIES(X)                                                                                                \
  X(fp8_layer_norm) X(fp8_layer_norm_backward) X(fp8_layer_norm_workspace) X(fp8_gated_act) X(fp8_gated_act_backward) \
  X(fp8_moe_route) X(fp8_moe_capacity) X(fp8_moe_dispatch) X(fp8_moe_combine) X(fp8_moe_combine_backward)             \
  X(fp8_rms_norm) X(fp8_rms_norm_backward) X(fp8_rms_norm_workspace) X(fp8_grouped_gemm) X(fp8_grouped_wgrad)          \
  X(fp8_grad_norm) X(fp8_clip_grad_norm) X(fp8_grad_norm_workspace)
#define X(f) decltype(&::f) p_##f = nullptr;
FP8Q_ENTRIES(X)
#undef X
PyObject* error_class = nullptr;   // FP8Error

struct Failed {};                  // a Python exception has been set

[[noreturn]] void refuse(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw Failed();
}
std::string shape_of(const at::Tensor& t) {
  std::string s = c10::toString(t.scalar_type()) + std::string(" (");
  for (int64_t i = 0; i < t.dim(); ++i)
    s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}
void check(fp8_status st, const char* fn) {
  if (st == FP8_OK) return;
  PyObject* e = PyObject_CallFunction(error_class, "si", fn, static_cast<int>(st));
  if (e != nullptr) {
    PyErr_SetObject(error_class, e);
    Py_DECREF(e);
  }
  throw Failed();
}

// Other threads run while outputs are allocated and the kernel is launched.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// The tensor of an argument, nullptr for None.
const at::Tensor* tensor(PyObject* o, const char* what) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(what) + ": a tensor is needed");
  return &THPVariable_Unpack(o);
}
const at::Tensor& needed(PyObject* o, const char* what) {
  const at::Tensor* t = tensor(o, what);
  if (t == nullptr) refuse(PyExc_TypeError, std::string(what) + ": a tensor is needed, not None");
  return *t;
}
// All tensors of a call are on one GPU.  Checked last, so that what else is wrong with a tensor is named first.
void on_gpu(std::initializer_list<PyObject*> args) {
  const at::Tensor* first = nullptr;
  for (PyObject* o : args) {
    if (o == Py_None) continue;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse(PyExc_ValueError, "a CUDA tensor is needed, not one on " + t.device().str());
    if (first == nullptr) first = &t;
    if (t.device() != first->device())
      refuse(PyExc_ValueError, "tensors of one device are needed, not of " + first->device().str() + " and " + t.device().str());
  }
}
fp8_dtype dtype_code(at::ScalarType type, const char* what) {
  if (type == at::kBFloat16) return FP8_DT_BF16;
  if (type == at::kFloat) return FP8_DT_FP32;
  refuse(PyExc_TypeError, std::string(what) + ": bfloat16 or float32 is needed, not " + c10::toString(type));
}
fp8_dtype data_type(const at::Tensor& t, const char* what) { return dtype_code(t.scalar_type(), what); }

// A 2-D tensor whose rows are contiguous (one without elements is, whatever its strides).
struct Rows {
  const at::Tensor* t = nullptr;
  int64_t rows = 0, cols = 0, ld = 0;
  void* p() const { return t == nullptr ? nullptr : t->data_ptr(); }
};
Rows rows_of(const at::Tensor& t, const char* what) {
  if (t.dim() != 2 || (t.stride(1) != 1 && t.size(1) > 1 && t.size(0) > 0))
    refuse(PyExc_ValueError, std::string(what) + ": a 2-D tensor with contiguous rows is needed, not " + shape_of(t));
  return {&t, t.size(0), t.size(1), t.stride(0)};
}
// None, or a tensor of these rows and columns and the type of `like`
Rows rows_like(PyObject* o, const at::Tensor& like, int64_t rows, int64_t cols, const char* what) {
  const at::Tensor* t = tensor(o, what);
  if (t == nullptr) return {};
  const Rows r = rows_of(*t, what);
  if (r.rows != rows || r.cols != cols || t->scalar_type() != like.scalar_type())
    refuse(PyExc_ValueError, std::string(what) + ": " + shape_of(*t) + ", expected " + c10::toString(like.scalar_type()) + " (" +
                                 std::to_string(rows) + ", " + std::to_string(cols) + ")");
  return r;
}
// None, or a dense tensor of n elements
void* vector_of(PyObject* o, int64_t n, at::ScalarType type, const char* what) {
  const at::Tensor* t = tensor(o, what);
  if (t == nullptr) return nullptr;
  if (t->numel() != n || t->scalar_type() != type || !t->is_contiguous())
    refuse(PyExc_ValueError, std::string(what) + ": " + std::to_string(n) + " contiguous " + c10::toString(type) +
                                 " elements are needed, not " + shape_of(*t));
  return t->data_ptr();
}
int64_t groups(int64_t cols) { return (cols + 127) / 128; }
// The codes and multipliers of an 8-bit copy, both or neither.
struct Copy {
  uint8_t* q = nullptr;
  float* s = nullptr;
  int64_t ld = 0;
};
Copy copy_of(PyObject* oq, PyObject* os, int64_t rows, int64_t cols, const char* what) {
  const at::Tensor* q = tensor(oq, what);
  if (q == nullptr && os == Py_None) return {};
  if (q == nullptr || os == Py_None || q->element_size() != 1 || q->dim() != 2 || q->size(0) != rows || q->size(1) != cols)
    refuse(PyExc_ValueError, std::string(what) + ": codes of one byte for every element and their multipliers are needed");
  const Rows r = rows_of(*q, what);
  return {static_cast<uint8_t*>(r.p()), static_cast<float*>(vector_of(os, rows * groups(cols), at::kFloat, what)), r.ld};
}

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}
// Outputs that live and die together (a copy's codes and multipliers, both statistics, a routing's
// arrays) are parts of one allocation: at::empty takes 1 us, a part 0.1.
at::Tensor part(const at::Tensor& whole, int64_t byte, at::ScalarType type, at::IntArrayRef shape, at::IntArrayRef strides) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(), c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_sizes_and_strides(shape, strides);
  t.unsafeGetTensorImpl()->set_storage_offset(byte / static_cast<int64_t>(c10::elementSize(type)));
  return t;
}
int64_t to16(int64_t bytes) { return (bytes + 15) / 16 * 16; }
struct NewCopy {
  at::Tensor q, s;
  int64_t ld = 0;
};
// N copies' codes, with a row stride of whole 16 bytes, and multipliers; `more` bytes behind them
// (where the returned place in the returned allocation starts)
struct Whole {
  at::Tensor t;
  int64_t rest;
};
template <int N>
Whole new_copies(NewCopy* const (&to)[N], int64_t rows, int64_t cols, const at::Tensor& like, int64_t more = 0) {
  const int64_t ld = to16(cols), g = groups(cols), codes = rows * ld, scales = to16(rows * g * 4), rest = N * (codes + scales);
  const at::Tensor whole = make({rest + more}, at::kByte, like);
  for (int i = 0; i < N; ++i) {
    to[i]->q = part(whole, i * codes, at::kByte, {rows, cols}, {ld, 1});
    to[i]->s = part(whole, N * codes + i * scales, at::kFloat, {rows, g}, {g, 1});
    to[i]->ld = ld;
  }
  return {whole, rest};
}
template <typename T>
T* ptr(const at::Tensor& t) {
  return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}
PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
template <typename... Ts>
PyObject* wrap_all(const Ts&... ts) {
  PyObject* out = PyTuple_New(sizeof...(ts));
  if (out == nullptr) throw Failed();
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(out, i++, wrap(ts)), ...);
  return out;
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Failed();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Failed();
  return v != 0;
}
// A number for an int32_t of the C ABI, which refuses what lies outside its range there too.
int32_t small(int64_t v) { return static_cast<int32_t>(std::min<int64_t>(std::max<int64_t>(v, -1), INT32_MAX)); }
// Where a call runs.  The tensors' device is current meanwhile: the library launches on the
// current device, whose number need not be the tensors'.
struct Place {
  c10::cuda::OptionalCUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard stream;
};
// The stream of a call.  None: the current stream of the tensors' device; else a raw stream or an
// object that has one, which `on` makes current, so that outputs and workspaces are allocated for
// the stream that writes them: a workspace is given back while its kernels may still be queued.
cudaStream_t stream_of(PyObject* o, const at::Tensor& t, Place& on) {
  if (o == Py_None) {
    on.device.set_index(t.device().index());
    return c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
  }
  PyObject* raw = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
  if (raw == nullptr) throw Failed();
  const auto s = static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(raw));
  Py_DECREF(raw);
  if (PyErr_Occurred()) throw Failed();
  on.stream.reset_stream(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(s), t.device().index()));
  return reinterpret_cast<cudaStream_t>(s);
}
fp8_format format(PyObject* o) { return static_cast<fp8_format>(small(integer(o))); }
fp8_act activation(PyObject* o) { return static_cast<fp8_act>(small(integer(o))); }

// The type code of weight and bias, of one type (either may be None).
fp8_dtype param_type(PyObject* weight, PyObject* bias) {
  const at::Tensor* t = tensor(weight, "weight");
  if (t == nullptr) t = tensor(bias, "bias");
  return t == nullptr ? FP8_DT_FP32 : data_type(*t, "weight / bias");
}
at::ScalarType scalar_type(fp8_dtype d) { return d == FP8_DT_FP32 ? at::kFloat : at::kBFloat16; }

// layer_norm(x, weight, bias, eps, checkpoint | None, stats, stream) -> (y, mean, rstd, q, s)
PyObject* layer_norm(PyObject* const* a) {
  const Rows x = rows_of(needed(a[0], "x"), "x");
  const fp8_dtype dt = data_type(*x.t, "x"), wdt = param_type(a[1], a[2]);
  void* w = vector_of(a[1], x.cols, scalar_type(wdt), "weight");
  void* b = vector_of(a[2], x.cols, scalar_type(wdt), "bias");
  on_gpu({a[0], a[1], a[2]});
  const double eps = PyFloat_AsDouble(a[3]);
  if (PyErr_Occurred()) throw Failed();
  const bool stats = truth(a[5]), keep = a[4] != Py_None;
  const fp8_format fmt = keep ? format(a[4]) : FP8_E4M3;
  Place on;
  const cudaStream_t stream = stream_of(a[6], *x.t, on);
  at::Tensor y, mean, rstd;
  NewCopy c;
  fp8_status st;
  {
    Unlocked unlocked;
    y = make({x.rows, x.cols}, x.t->scalar_type(), *x.t);
    const int64_t more = stats ? 8 * x.rows : 0;
    if (keep || stats) {
      const Whole whole = keep ? new_copies({&c}, x.rows, x.cols, *x.t, more) : Whole{make({more}, at::kByte, *x.t), 0};
      if (stats) {
        mean = part(whole.t, whole.rest, at::kFloat, {x.rows}, {1});
        rstd = part(whole.t, whole.rest + 4 * x.rows, at::kFloat, {x.rows}, {1});
      }
    }
    st = p_fp8_layer_norm(x.p(), x.rows, x.cols, x.ld, dt, w, b, wdt, static_cast<float>(eps), y.data_ptr(), x.cols,
                          ptr<float>(mean), ptr<float>(rstd), fmt, ptr<uint8_t>(c.q), c.ld, ptr<float>(c.s), stream);
  }
  check(st, "fp8_layer_norm");
  return wrap_all(y, mean, rstd, c.q, c.s);
}

// layer_norm_backward(dy, rstd, weight, x, mean, q, s, fmt, param_grads, param_dtype, stream) -> (dx, dweight, dbias)
PyObject* layer_norm_backward(PyObject* const* a) {
  const Rows dy = rows_of(needed(a[0], "dy"), "dy");
  const fp8_dtype dt = data_type(*dy.t, "dy");
  if (!THPDtype_Check(a[9])) refuse(PyExc_TypeError, "param_dtype: a torch.dtype is needed");
  const at::Tensor* weight = tensor(a[2], "weight");
  const fp8_dtype wdt = dtype_code(weight != nullptr ? weight->scalar_type() : reinterpret_cast<THPDtype*>(a[9])->scalar_type,
                                   weight != nullptr ? "weight" : "param_dtype");
  void* w = vector_of(a[2], dy.cols, scalar_type(wdt), "weight");
  const Rows x = rows_like(a[3], *dy.t, dy.rows, dy.cols, "x");
  auto* rstd = static_cast<float*>(vector_of(a[1], dy.rows, at::kFloat, "rstd"));
  auto* mean = static_cast<float*>(vector_of(a[4], dy.rows, at::kFloat, "mean"));
  const Copy c = copy_of(a[5], a[6], dy.rows, dy.cols, "q");
  on_gpu({a[0], a[1], a[2], a[3], a[4], a[5], a[6]});
  const fp8_format fmt = format(a[7]);
  const bool param_grads = truth(a[8]);
  Place on;
  const cudaStream_t stream = stream_of(a[10], *dy.t, on);
  int64_t bytes = 0;
  if (param_grads) check(p_fp8_layer_norm_workspace(dy.rows, dy.cols, &bytes), "fp8_layer_norm_workspace");
  at::Tensor dx, dw, db, ws;
  fp8_status st;
  {
    Unlocked unlocked;
    dx = make({dy.rows, dy.cols}, dy.t->scalar_type(), *dy.t);
    if (param_grads) {
      const int64_t half = to16(dy.cols * static_cast<int64_t>(c10::elementSize(scalar_type(wdt))));
      const at::Tensor whole = make({2 * half}, at::kByte, *dy.t);
      dw = part(whole, 0, scalar_type(wdt), {dy.cols}, {1});
      db = part(whole, half, scalar_type(wdt), {dy.cols}, {1});
      ws = make({bytes}, at::kByte, *dy.t);
    }
    st = p_fp8_layer_norm_backward(dy.p(), dy.rows, dy.cols, dy.ld, dt, x.p(), x.ld, mean, rstd, fmt, c.q, c.ld, c.s, w, wdt,
                                   dx.data_ptr(), dy.cols, ptr<void>(dw), ptr<void>(db), ptr<void>(ws), bytes, stream);
  }
  check(st, "fp8_layer_norm_backward");
  return wrap_all(dx, dw, db);
}

// gated_act(a, b, act, checkpoint | None, stream) -> (y, qa, sa, qb, sb)
PyObject* gated_act(PyObject* const* a) {
  const Rows x = rows_of(needed(a[0], "a"), "a");
  const fp8_dtype dt = data_type(*x.t, "a");
  const Rows b = rows_like(a[1], *x.t, x.rows, x.cols, "b");
  on_gpu({a[0], a[1]});
  const fp8_act act = activation(a[2]);
  const bool keep = a[3] != Py_None;
  const fp8_format fmt = keep ? format(a[3]) : FP8_E4M3;
  Place on;
  const cudaStream_t stream = stream_of(a[4], *x.t, on);
  at::Tensor y;
  NewCopy ca, cb;
  fp8_status st;
  {
    Unlocked unlocked;
    y = make({x.rows, x.cols}, x.t->scalar_type(), *x.t);
    if (keep && b.t != nullptr)
      new_copies({&ca, &cb}, x.rows, x.cols, *x.t);
    else if (keep)
      new_copies({&ca}, x.rows, x.cols, *x.t);
    st = p_fp8_gated_act(x.p(), x.rows, x.cols, x.ld, dt, act, b.p(), b.ld, y.data_ptr(), x.cols, fmt, ptr<uint8_t>(ca.q),
                         ptr<float>(ca.s), ptr<uint8_t>(cb.q), ptr<float>(cb.s), ca.ld, stream);
  }
  check(st, "fp8_gated_act");
  return wrap_all(y, ca.q, ca.s, cb.q, cb.s);
}

// gated_act_backward(dy, act, a, b, qa, sa, qb, sb, fmt, stream) -> (da, db)
PyObject* gated_act_backward(PyObject* const* a) {
  const Rows dy = rows_of(needed(a[0], "dy"), "dy");
  const fp8_dtype dt = data_type(*dy.t, "dy");
  const Rows x = rows_like(a[2], *dy.t, dy.rows, dy.cols, "a"), b = rows_like(a[3], *dy.t, dy.rows, dy.cols, "b");
  const Copy ca = copy_of(a[4], a[5], dy.rows, dy.cols, "qa"), cb = copy_of(a[6], a[7], dy.rows, dy.cols, "qb");
  if (ca.q != nullptr && cb.q != nullptr && ca.ld != cb.ld && dy.rows > 1)
    refuse(PyExc_ValueError, "qa and qb: one row stride is needed for both");
  on_gpu({a[0], a[2], a[3], a[4], a[5], a[6], a[7]});
  const fp8_act act = activation(a[1]);
  const fp8_format fmt = format(a[8]);
  Place on;
  const cudaStream_t stream = stream_of(a[9], *dy.t, on);
  const bool gated = b.t != nullptr || cb.q != nullptr;
  const int64_t ld = gated ? 2 * dy.cols : dy.cols;
  at::Tensor da, db;
  fp8_status st;
  {
    Unlocked unlocked;
    da = make({dy.rows, ld}, dy.t->scalar_type(), *dy.t);
    if (gated) {   // the halves of one tensor
      const at::Tensor whole = da;
      da = part(whole, 0, dy.t->scalar_type(), {dy.rows, dy.cols}, {ld, 1});
      db = part(whole, dy.cols * dy.t->element_size(), dy.t->scalar_type(), {dy.rows, dy.cols}, {ld, 1});
    }
    st = p_fp8_gated_act_backward(dy.p(), dy.rows, dy.cols, dy.ld, dt, act, x.p(), x.ld, b.p(), b.ld, fmt, ca.q, ca.s, cb.q, cb.s,
                                  ca.q != nullptr ? ca.ld : cb.ld, da.data_ptr(), ld, ptr<void>(db), ld, stream);
  }
  check(st, "fp8_gated_act_backward");
  return wrap_all(da, db);
}

// moe_route(experts, n_experts, align, stream) -> (offsets, pos, src)
PyObject* moe_route(PyObject* const* a) {
  const at::Tensor& e = needed(a[0], "experts");
  const bool wide = e.scalar_type() == at::kLong;
  if (e.dim() != 2 || (!wide && e.scalar_type() != at::kInt) || !e.is_contiguous())
    refuse(PyExc_ValueError, "experts: a contiguous [tokens, k] int32 or int64 tensor is needed, not " + shape_of(e));
  on_gpu({a[0]});
  const int64_t tokens = e.size(0);
  const int32_t k = small(e.size(1)), n_experts = small(integer(a[1])), align = small(integer(a[2]));
  Place on;
  const cudaStream_t stream = stream_of(a[3], e, on);
  int64_t capacity = 0;
  check(p_fp8_moe_capacity(tokens, k, n_experts, align, &capacity), "fp8_moe_capacity");
  at::Tensor offsets, pos, src;
  fp8_status st;
  {
    Unlocked unlocked;
    const int64_t at_pos = to16(4 * (int64_t{n_experts} + 1)), at_src = at_pos + to16(4 * tokens * k);
    const at::Tensor whole = make({at_src + 4 * capacity}, at::kByte, e);
    offsets = part(whole, 0, at::kInt, {n_experts + 1}, {1});
    pos = part(whole, at_pos, at::kInt, {tokens, k}, {k, 1});
    src = part(whole, at_src, at::kInt, {capacity}, {1});
    st = p_fp8_moe_route(e.data_ptr(), wide ? 8 : 4, tokens, k, n_experts, align, ptr<int32_t>(offsets), ptr<int32_t>(pos),
                         ptr<int32_t>(src), capacity, stream);
  }
  check(st, "fp8_moe_route");
  return wrap_all(offsets, pos, src);
}

// the pos of a routing, [tokens, k] (any number of tokens with tokens < 0)
const at::Tensor& choices(PyObject* o, int64_t tokens) {
  const at::Tensor& t = needed(o, "pos");
  if (t.dim() != 2 || t.scalar_type() != at::kInt || !t.is_contiguous() || (tokens >= 0 && t.size(0) != tokens))
    refuse(PyExc_ValueError, "pos: a contiguous int32 [tokens, k] tensor is needed, not " + shape_of(t));
  return t;
}

// moe_dispatch(x, pos, src, stream) -> xs
PyObject* moe_dispatch(PyObject* const* a) {
  const Rows x = rows_of(needed(a[0], "x"), "x");
  const fp8_dtype dt = data_type(*x.t, "x");
  const at::Tensor& pos = choices(a[1], x.rows);
  const int64_t capacity = needed(a[2], "src").numel();
  auto* src = static_cast<int32_t*>(vector_of(a[2], capacity, at::kInt, "src"));
  on_gpu({a[0], a[1], a[2]});
  Place on;
  const cudaStream_t stream = stream_of(a[3], *x.t, on);
  at::Tensor xs;
  fp8_status st;
  {
    Unlocked unlocked;
    xs = make({capacity, x.cols}, x.t->scalar_type(), *x.t);
    st = p_fp8_moe_dispatch(x.p(), x.rows, x.cols, x.ld, dt, small(pos.size(1)), ptr<int32_t>(pos), src, capacity, xs.data_ptr(),
                            x.cols, stream);
  }
  check(st, "fp8_moe_dispatch");
  return wrap(xs);
}

// moe_combine(ys, pos, weights, stream) -> y
PyObject* moe_combine(PyObject* const* a) {
  const Rows ys = rows_of(needed(a[0], "ys"), "ys");
  const fp8_dtype dt = data_type(*ys.t, "ys");
  const at::Tensor& pos = choices(a[1], -1);
  auto* w = static_cast<float*>(vector_of(a[2], pos.numel(), at::kFloat, "weights"));
  on_gpu({a[0], a[1], a[2]});
  Place on;
  const cudaStream_t stream = stream_of(a[3], *ys.t, on);
  at::Tensor y;
  fp8_status st;
  {
    Unlocked unlocked;
    y = make({pos.size(0), ys.cols}, ys.t->scalar_type(), *ys.t);
    st = p_fp8_moe_combine(ys.p(), ys.rows, ys.cols, ys.ld, dt, pos.size(0), small(pos.size(1)), ptr<int32_t>(pos), w,
                           y.data_ptr(), ys.cols, stream);
  }
  check(st, "fp8_moe_combine");
  return wrap(y);
}

// moe_combine_backward(dy, ys, pos, src, weights, stream) -> (dys, dweights)
PyObject* moe_combine_backward(PyObject* const* a) {
  const Rows dy = rows_of(needed(a[0], "dy"), "dy");
  const fp8_dtype dt = data_type(*dy.t, "dy");
  const at::Tensor& pos = choices(a[2], dy.rows);
  const int64_t capacity = needed(a[3], "src").numel();
  auto* src = static_cast<int32_t*>(vector_of(a[3], capacity, at::kInt, "src"));
  auto* w = static_cast<float*>(vector_of(a[4], pos.numel(), at::kFloat, "weights"));
  const bool weighted = a[4] != Py_None;
  const Rows ys = weighted ? rows_like(a[1], *dy.t, capacity, dy.cols, "ys") : Rows{};
  on_gpu({a[0], a[2], a[3], a[4], weighted ? a[1] : Py_None});
  Place on;
  const cudaStream_t stream = stream_of(a[5], *dy.t, on);
  at::Tensor dys, dw;
  fp8_status st;
  {
    Unlocked unlocked;
    dys = make({capacity, dy.cols}, dy.t->scalar_type(), *dy.t);
    if (weighted) dw = make(pos.sizes(), at::kFloat, pos);
    st = p_fp8_moe_combine_backward(dy.p(), dy.rows, dy.cols, dy.ld, dt, small(pos.size(1)), ptr<int32_t>(pos), src, w, ys.p(),
                                    ys.ld, capacity, dys.data_ptr(), dy.cols, ptr<float>(dw), stream);
  }
  check(st, "fp8_moe_combine_backward");
  return wrap_all(dys, dw);
}

constexpr int64_t kTogether = 64 * 1024;   // bytes

fp8_recipe recipe_of(PyObject* o) { return static_cast<fp8_recipe>(small(integer(o))); }
bool is_mx(fp8_recipe r) { return r >= FP8_MX_1x32; }
bool is_tiled(fp8_recipe r) { return r == FP8_MX_1x32_TILED || r == FP8_MX_1x32_FLOOR_TILED; }

// rms_norm(x, weight, residual, eps, recipe | None, fmt, scale, amax_out, keep_y, stats, stream) -> (y, h, rstd, q, s)
PyObject* rms_norm(PyObject* const* a) {
  const Rows x = rows_of(needed(a[0], "x"), "x");
  const fp8_dtype dt = data_type(*x.t, "x"), wdt = param_type(a[1], Py_None);
  void* w = vector_of(a[1], x.cols, scalar_type(wdt), "weight");
  const Rows res = rows_like(a[2], *x.t, x.rows, x.cols, "residual");
  auto* scale = static_cast<float*>(vector_of(a[6], 1, at::kFloat, "scale"));
  auto* amax = static_cast<float*>(vector_of(a[7], 1, at::kFloat, "amax_out"));
  on_gpu({a[0], a[1], a[2], a[6], a[7]});
  const double eps = PyFloat_AsDouble(a[3]);
  if (PyErr_Occurred()) throw Failed();
  const bool copy = a[4] != Py_None, keep_y = truth(a[8]), stats = truth(a[9]);
  const fp8_recipe recipe = copy ? recipe_of(a[4]) : FP8_TENSOR;
  const fp8_format fmt = format(a[5]);
  Place on;
  const cudaStream_t stream = stream_of(a[10], *x.t, on);
  at::Tensor y, h, rstd, q, s;
  const int64_t ldq = to16(x.cols);
  fp8_status st;
  {
    Unlocked unlocked;
    // the codes and their multipliers in one allocation; with little data (a few tokens) all outputs are.  The statistics, which
    // a backward pass holds long after the codes were used, are apart from much of them: with h, which it holds too, or alone.
    int64_t shape[3] = {1, 1, 1}, dims = 1, scales = 0;
    if (copy) {
      if (is_tiled(recipe)) {
        dims = 3, shape[0] = (x.rows + 127) / 128, shape[1] = groups(x.cols), shape[2] = 512;
      } else if (recipe != FP8_TENSOR) {
        dims = 2, shape[0] = x.rows, shape[1] = is_mx(recipe) ? x.cols / 32 : groups(x.cols);
      }
      scales = to16(shape[0] * shape[1] * shape[2] * (is_mx(recipe) ? 1 : 4));
    }
    const int64_t codes = copy ? to16(x.rows * ldq) : 0, rest = stats ? to16(4 * x.rows) : 0;
    const int64_t data = to16(x.rows * x.cols * static_cast<int64_t>(x.t->element_size()));
    const int64_t wide = (keep_y ? data : 0) + (res.t != nullptr ? data : 0);
    const bool together = wide + codes + scales + rest <= kTogether;
    at::Tensor whole;
    if (together || codes + scales > 0) whole = make({(together ? wide + rest : 0) + codes + scales}, at::kByte, *x.t);
    int64_t at = 0;
    auto matrix = [&](bool wanted) -> at::Tensor {
      if (!wanted) return {};
      if (!together) return make({x.rows, x.cols}, x.t->scalar_type(), *x.t);
      at += data;
      return part(whole, at - data, x.t->scalar_type(), {x.rows, x.cols}, {x.cols, 1});
    };
    y = matrix(keep_y);
    if (!together && stats && res.t != nullptr) {
      const at::Tensor kept = make({data + rest}, at::kByte, *x.t);
      h = part(kept, 0, x.t->scalar_type(), {x.rows, x.cols}, {x.cols, 1});
      rstd = part(kept, data, at::kFloat, {x.rows}, {1});
    } else {
      h = matrix(res.t != nullptr);
    }
    if (copy) {
      const int64_t strides[3] = {dims == 1 ? 1 : shape[1] * shape[2], dims == 2 ? 1 : shape[2], 1};
      q = part(whole, at, at::kByte, {x.rows, x.cols}, {ldq, 1});
      s = part(whole, at + codes, is_mx(recipe) ? at::kByte : at::kFloat, {shape, static_cast<size_t>(dims)},
               {strides, static_cast<size_t>(dims)});
    }
    if (stats && !rstd.defined())
      rstd = together ? part(whole, at + codes + scales, at::kFloat, {x.rows}, {1}) : make({x.rows}, at::kFloat, *x.t);
    st = p_fp8_rms_norm(x.p(), x.rows, x.cols, x.ld, dt, res.p(), res.ld, w, wdt, static_cast<float>(eps), ptr<void>(h), x.cols,
                        ptr<void>(y), x.cols, ptr<float>(rstd), recipe, fmt, scale, amax, ptr<uint8_t>(q), ldq, ptr<void>(s),
                        stream);
  }
  check(st, "fp8_rms_norm");
  return wrap_all(y, h, rstd, q, s);
}

// rms_norm_backward(dy, h, rstd, weight, dh, param_grads, param_dtype, stream) -> (dx, dweight)
PyObject* rms_norm_backward(PyObject* const* a) {
  const Rows dy = rows_of(needed(a[0], "dy"), "dy");
  const fp8_dtype dt = data_type(*dy.t, "dy");
  needed(a[1], "h");
  needed(a[2], "rstd");
  const Rows h = rows_like(a[1], *dy.t, dy.rows, dy.cols, "h"), dh = rows_like(a[4], *dy.t, dy.rows, dy.cols, "dh");
  if (!THPDtype_Check(a[6])) refuse(PyExc_TypeError, "param_dtype: a torch.dtype is needed");
  const at::Tensor* weight = tensor(a[3], "weight");
  const fp8_dtype wdt = dtype_code(weight != nullptr ? weight->scalar_type() : reinterpret_cast<THPDtype*>(a[6])->scalar_type,
                                   weight != nullptr ? "weight" : "param_dtype");
  void* w = vector_of(a[3], dy.cols, scalar_type(wdt), "weight");
  auto* rstd = static_cast<float*>(vector_of(a[2], dy.rows, at::kFloat, "rstd"));
  on_gpu({a[0], a[1], a[2], a[3], a[4]});
  const bool param_grads = truth(a[5]);
  Place on;
  const cudaStream_t stream = stream_of(a[7], *dy.t, on);
  int64_t bytes = 0;
  if (param_grads) check(p_fp8_rms_norm_workspace(dy.rows, dy.cols, &bytes), "fp8_rms_norm_workspace");
  at::Tensor dx, dw, ws;
  fp8_status st;
  {
    Unlocked unlocked;
    dx = make({dy.rows, dy.cols}, dy.t->scalar_type(), *dy.t);
    if (param_grads) {
      dw = make({dy.cols}, scalar_type(wdt), *dy.t);
      ws = make({bytes}, at::kByte, *dy.t);
    }
    st = p_fp8_rms_norm_backward(dy.p(), dy.rows, dy.cols, dy.ld, dt, h.p(), h.ld, rstd, dh.p(), dh.ld, w, wdt, dx.data_ptr(),
                                 dy.cols, ptr<void>(dw), ptr<void>(ws), bytes, stream);
  }
  check(st, "fp8_rms_norm_backward");
  return wrap_all(dx, dw);
}

// One operand of the grouped products: dense codes and their multipliers.
struct Operand {
  const at::Tensor* t;
  int64_t rows, cols, n_scales;
  void* s;
  uint8_t* p() const { return static_cast<uint8_t*>(t->data_ptr()); }
};
Operand operand_of(PyObject* o, PyObject* os, fp8_recipe recipe, int64_t experts, const char* what) {
  const at::Tensor& t = needed(o, what);
  if (t.dim() != 2 || t.element_size() != 1 || !t.is_contiguous())
    refuse(PyExc_ValueError, std::string(what) + ": a dense matrix of one-byte codes is needed, not " + shape_of(t));
  const at::Tensor& s = needed(os, "scales");
  Operand r{&t, t.size(0), t.size(1), s.numel(), s.data_ptr()};
  if (is_mx(recipe)) {
    if (s.element_size() != 1 || !s.is_contiguous() || r.n_scales != (r.rows + 127) / 128 * groups(r.cols) * 512)
      refuse(PyExc_ValueError, std::string(what) + ": its tiled one-byte scales are needed, not " + shape_of(s));
  } else if (s.scalar_type() != at::kFloat || !s.is_contiguous() || (r.n_scales != 1 && r.n_scales != experts)) {
    refuse(PyExc_ValueError, std::string(what) + ": one float32 multiplier" + (experts > 1 ? " (or one an expert)" : "") +
                                 " is needed, not " + shape_of(s));
  }
  return r;
}
const at::Tensor& starts_of(PyObject* o) {
  const at::Tensor& t = needed(o, "offsets");
  if (t.dim() != 1 || t.size(0) < 2 || t.scalar_type() != at::kInt || !t.is_contiguous())
    refuse(PyExc_ValueError, "offsets: a contiguous int32 vector of n_experts + 1 is needed, not " + shape_of(t));
  return t;
}
fp8_out_dtype out_of(PyObject* o) { return static_cast<fp8_out_dtype>(small(integer(o))); }

// grouped_gemm(a, fa, ra, sa, b, fb, rb, sb, offsets, out, stacked, zero_tail, stream) -> c
PyObject* grouped_gemm(PyObject* const* v) {
  const at::Tensor& offsets = starts_of(v[8]);
  const int64_t experts = offsets.size(0) - 1;
  const fp8_recipe ra = recipe_of(v[2]), rb = recipe_of(v[6]);
  const Operand a = operand_of(v[0], v[3], ra, 1, "a"), b = operand_of(v[4], v[7], rb, experts, "b");
  const fp8_out_dtype out = out_of(v[9]);
  const fp8_format fa = format(v[1]), fb = format(v[5]);
  const auto stacked = static_cast<fp8_stacked>(small(integer(v[10])));
  const bool cols = stacked == FP8_STACKED_COLS;
  const int64_t n = cols ? b.rows : b.rows / experts, depth = a.cols;
  if (cols ? b.cols != experts * depth : b.rows != experts * n || b.cols != depth)
    refuse(PyExc_ValueError, "b: " + std::to_string(experts) + " experts' matrices of depth " + std::to_string(depth) +
                                 (cols ? " side by side" : " one below the other") + " are needed, not " + shape_of(*b.t));
  on_gpu({v[0], v[3], v[4], v[7], v[8]});
  const int32_t zero_tail = truth(v[11]) ? 2 : 0;   // the allocation's rows outside the segments, in front and behind
  Place on;
  const cudaStream_t stream = stream_of(v[12], *a.t, on);
  at::Tensor c;
  fp8_status st;
  {
    Unlocked unlocked;
    c = make({a.rows, n}, out == FP8_OUT_FP32 ? at::kFloat : at::kBFloat16, *a.t);
    st = p_fp8_grouped_gemm(a.p(), fa, ra, a.s, b.p(), fb, rb, b.s, small(b.n_scales), ptr<int32_t>(offsets),
                            small(experts), a.rows, n, depth, stacked, c.data_ptr(), out, zero_tail, stream);
  }
  check(st, "fp8_grouped_gemm");
  return wrap(c);
}

// grouped_wgrad(a, fa, ra, sa, b, fb, rb, sb, offsets, out, stream) -> c
PyObject* grouped_wgrad(PyObject* const* v) {
  const at::Tensor& offsets = starts_of(v[8]);
  const int64_t experts = offsets.size(0) - 1;
  const fp8_recipe ra = recipe_of(v[2]), rb = recipe_of(v[6]);
  const Operand a = operand_of(v[0], v[3], ra, 1, "a"), b = operand_of(v[4], v[7], rb, 1, "b");
  if (a.cols != b.cols)
    refuse(PyExc_ValueError, "a and b: the same number of rows' columns is needed, not " + shape_of(*a.t) + " and " + shape_of(*b.t));
  on_gpu({v[0], v[3], v[4], v[7], v[8]});
  const fp8_out_dtype out = out_of(v[9]);
  const fp8_format fa = format(v[1]), fb = format(v[5]);
  Place on;
  const cudaStream_t stream = stream_of(v[10], *a.t, on);
  at::Tensor c;
  fp8_status st;
  {
    Unlocked unlocked;
    c = make({experts, a.rows, b.rows}, out == FP8_OUT_FP32 ? at::kFloat : at::kBFloat16, *a.t);
    st = p_fp8_grouped_wgrad(a.p(), fa, ra, a.s, b.p(), fb, rb, b.s, ptr<int32_t>(offsets), small(experts),
                             a.cols, a.rows, b.rows, c.data_ptr(), out, stream);
  }
  check(st, "fp8_grouped_wgrad");
  return wrap(c);
}

// The elements of a sequence of tensors, held until the call returns: the caller's list may change meanwhile, in another thread
// while the interpreter is unlocked or in Python code that an argument runs, and its tensors may be dropped.
struct Items {
  PyObject* tuple;
  Items(PyObject* o, const char* what) {
    PyObject* const seq = PySequence_Fast(o, what);
    if (seq == nullptr) throw Failed();
    tuple = PySequence_Tuple(seq);
    Py_DECREF(seq);
    if (tuple == nullptr) throw Failed();
  }
  ~Items() { Py_DECREF(tuple); }
  Items(const Items&) = delete;
  Items& operator=(const Items&) = delete;
  Py_ssize_t size() const { return PyTuple_GET_SIZE(tuple); }
  PyObject* operator[](Py_ssize_t i) const { return PyTuple_GET_ITEM(tuple, i); }
};
// A gradient whose elements fill their memory without gaps, in whatever order.
const at::Tensor& dense(PyObject* o, const char* what) {
  const at::Tensor& t = needed(o, what);
  data_type(t, what);
  if (t.layout() != at::kStrided || !t.is_non_overlapping_and_dense())
    refuse(PyExc_ValueError, std::string(what) + ": dense tensors are needed, not " + shape_of(t));
  return t;
}

// The memory of a call's tensors: what one of them writes must not be part of another, whose turn may come first
// or last.  Tensors of different storages are apart if torch's allocator made both (one taken over from elsewhere, as by DLPack, may
// lie in another's memory), and those of one storage are seen to be apart on the way when they come in ascending
// order, as views into a buffer do; only others are sorted.
class Spans {
 public:
  explicit Spans(size_t n) {
    all_.reserve(n);
    size_t slots = 16;
    while (slots < 2 * n) slots *= 2;
    ends_.resize(slots);
  }
  void add(const at::Tensor& t, bool written) {
    if (t.numel() == 0) return;
    const auto lo = reinterpret_cast<uintptr_t>(t.const_data_ptr());
    const uintptr_t hi = lo + static_cast<uintptr_t>(t.numel() * t.element_size());
    all_.push_back({lo, hi, written});
    const c10::StorageImpl* const storage = t.unsafeGetTensorImpl()->unsafe_storage().unsafeGetStorageImpl();
    if (storage->data_ptr().get_deleter() != own_) sorted_ = false;
    size_t i = (reinterpret_cast<uintptr_t>(storage) >> 4) * 0x9E3779B97F4A7C15ull >> 20;
    while (true) {
      End& e = ends_[i++ & (ends_.size() - 1)];
      if (e.storage != nullptr && e.storage != storage) continue;
      if (e.storage != nullptr && lo < e.hi) sorted_ = false;
      e = {storage, hi};
      return;
    }
  }
  bool meet() {
    if (sorted_) return false;
    std::sort(all_.begin(), all_.end(), [](const Span& x, const Span& y) { return x.lo < y.lo; });
    uintptr_t any = 0, written = 0;   // ends of what lies in front
    for (const Span& x : all_) {
      if (x.lo < written || (x.written && x.lo < any)) return true;
      any = std::max(any, x.hi);
      if (x.written) written = std::max(written, x.hi);
    }
    return false;
  }

 private:
  struct Span {
    uintptr_t lo, hi;
    bool written;
  };
  struct End {
    const void* storage = nullptr;
    uintptr_t hi = 0;
  };
  const c10::DeleterFnPtr own_ = c10::cuda::CUDACachingAllocator::get()->raw_deleter();
  std::vector<Span> all_;
  std::vector<End> ends_;   // by storage, open addressing
  bool sorted_ = true;
};

// clip_grad_norm(grads, max_norm | None, out | None, stream) -> norm; max_norm None: the norm alone;
// out None: in place
PyObject* clip_grad_norm(PyObject* const* v) {
  const Items grads(v[0], "grads: a sequence of tensors is needed");
  const Py_ssize_t n = grads.size();
  const bool clip = v[1] != Py_None, in_place = v[2] == Py_None;
  const double max_norm = clip ? PyFloat_AsDouble(v[1]) : 0.0;
  if (PyErr_Occurred()) throw Failed();
  std::optional<Items> out;   // in place the gradients themselves: a generator gives its tensors once
  if (!in_place) out.emplace(v[2], "out: a sequence of tensors is needed");
  const Items& outs = in_place ? grads : *out;
  if (clip && outs.size() != n) refuse(PyExc_ValueError, "out: as many tensors as gradients are needed");
  if (n == 0) refuse(PyExc_ValueError, "grads: at least one tensor is needed");
  std::vector<fp8_gradient> table(static_cast<size_t>(n));
  const at::Tensor& first = needed(grads[0], "grads");
  Spans spans(static_cast<size_t>(in_place ? n : 2 * n));
  for (Py_ssize_t i = 0; i < n; ++i) {
    const at::Tensor& g = dense(grads[i], "grads");
    if (!g.is_cuda()) refuse(PyExc_ValueError, "a CUDA tensor is needed, not one on " + g.device().str());
    if (g.device() != first.device())
      refuse(PyExc_ValueError, "tensors of one device are needed, not of " + first.device().str() + " and " + g.device().str());
    fp8_gradient& to = table[static_cast<size_t>(i)];
    to = {g.data_ptr(), nullptr, g.numel(), data_type(g, "grads")};
    if (!clip) continue;
    const at::Tensor& o = in_place ? g : dense(outs[i], "out");
    if (!in_place) {
      if (o.scalar_type() != g.scalar_type() || o.sizes() != g.sizes() || o.strides() != g.strides() || o.device() != g.device())
        refuse(PyExc_ValueError, "out: tensors like the gradients are needed, not " + shape_of(o) + " for " + shape_of(g));
      if (o.data_ptr() != g.data_ptr()) spans.add(o, true);
    }
    to.out = o.data_ptr();
    spans.add(g, to.out == to.in);
  }
  if (spans.meet()) refuse(PyExc_ValueError, "gradients and outputs must not share memory");
  Place on;
  const cudaStream_t stream = stream_of(v[3], first, on);
  int64_t bytes = 0;
  const auto count = small(n);
  check(p_fp8_grad_norm_workspace(count, &bytes), "fp8_grad_norm_workspace");
  at::Tensor whole, norm;
  fp8_status st;
  {
    Unlocked unlocked;
    whole = make({bytes}, at::kByte, first);
    norm = make({1}, at::kFloat, first);
    st = clip ? p_fp8_clip_grad_norm(table.data(), count, static_cast<float>(max_norm), whole.data_ptr(), bytes, ptr<float>(norm), stream)
              : p_fp8_grad_norm(table.data(), count, whole.data_ptr(), bytes, ptr<float>(norm), stream);
  }
  check(st, clip ? "fp8_clip_grad_norm" : "fp8_grad_norm");
  // autograd learns of what was written, as of any operation in place
  for (Py_ssize_t i = 0; clip && i < n; ++i) {
    const at::Tensor& o = needed(outs[i], "out");
    if (!o.is_inference()) o.unsafeGetTensorImpl()->bump_version();
  }
  return wrap(norm);
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments are needed, not %zd", N, n);
    return nullptr;
  }
  if (error_class == nullptr) {
    PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Failed&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// bind({entry point: address}, FP8Error)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 2 || !PyDict_Check(args[0])) {
    PyErr_SetString(PyExc_TypeError, "bind(addresses, error class)");
    return nullptr;
  }
#define X(f)                                                             \
  {                                                                      \
    PyObject* v = PyDict_GetItemString(args[0], #f);                     \
    const uint64_t at = v != nullptr ? PyLong_AsUnsignedLongLong(v) : 0; \
    if (at == 0 || PyErr_Occurred()) {                                   \
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_KeyError, #f);        \
      return nullptr;                                                    \
    }                                                                    \
    p_##f = reinterpret_cast<decltype(&::f)>(static_cast<uintptr_t>(at)); \
  }
  FP8Q_ENTRIES(X)
#undef X
  Py_INCREF(args[1]);
  Py_XDECREF(error_class);
  error_class = args[1];
  Py_RETURN_NONE;
}

#define ENTRY(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&bind)), METH_FASTCALL, nullptr},
    ENTRY(layer_norm, 7),
    ENTRY(layer_norm_backward, 11),
    ENTRY(gated_act, 5),
    ENTRY(gated_act_backward, 10),
    ENTRY(moe_route, 4),
    ENTRY(moe_dispatch, 4),
    ENTRY(moe_combine, 4),
    ENTRY(moe_combine_backward, 6),
    ENTRY(rms_norm, 11),
    ENTRY(rms_norm_backward, 8),
    ENTRY(grouped_gemm, 13),
    ENTRY(grouped_wgrad, 11),
    ENTRY(clip_grad_norm, 4),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rowops", "Allocation helpers of the row operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rowops() { return PyModule_Create(&module); }
