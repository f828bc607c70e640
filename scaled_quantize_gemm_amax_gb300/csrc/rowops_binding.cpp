// rowops_binding.cpp -- the allocation helpers of the row operators as a Python extension.
//
// A row operator on a few tokens takes 1.5 to 3 us on the device; checking its tensors,
// allocating its outputs and marshalling its arguments in Python took 11 to 40 us.  Here the
// same steps are compiled: check, at::empty, one call of the C ABI.  The entry points' addresses
// are handed over by bind(), so that this module and the ctypes binding use the same loaded
// library.  Arguments are positional (the Python helpers give them names and defaults).
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fp8q.h"

namespace {

#define FP8Q_ENTRIES(X)                                                                                                \
  X(fp8_layer_norm) X(fp8_layer_norm_backward) X(fp8_layer_norm_workspace) X(fp8_gated_act) X(fp8_gated_act_backward) \
  X(fp8_moe_route) X(fp8_moe_capacity) X(fp8_moe_dispatch) X(fp8_moe_combine) X(fp8_moe_combine_backward)
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
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rowops", "Allocation helpers of the row operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rowops() { return PyModule_Create(&module); }
