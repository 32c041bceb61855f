// The training calls on torch tensors: a CPython module (_training) that
// checks lists of tensors, allocates the outputs and calls the C ABI.
//
// A router call looks at up to three tensors a rank and allocates five; in
// Python that took 20 us for 8 ranks, more than most such calls take on the
// GPU.  Here it takes about a third, the launch included.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/EmptyTensor.h>

#include <cstring>

#include "ar.h"

namespace {

// Raises `type` with a formatted message; for `return fail(...)`.
template <class... A> std::nullptr_t fail(PyObject* type, const char* format, A... a) {
  PyErr_Format(type, format, a...);
  return nullptr;
}

struct Ranks {
  const void* p[AR_MAX_RANKS];
};

// The tensor behind a Python object, which must be one on a GPU.
const at::Tensor* gpu_tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
    return fail(PyExc_TypeError, "%s must be GPU tensors", what);
  return &THPVariable_Unpack(o);
}

Py_ssize_t list_size(PyObject* list, const char* what) {
  if (!PyList_Check(list)) {
    fail(PyExc_TypeError, "%s must be a list", what);
    return -1;
  }
  return PyList_GET_SIZE(list);
}

// The ranks' logits: GPU tensors [tokens, experts] of one type, shape and
// strides, experts next to each other.  A stride along one element or none
// says nothing and may be any.
const at::Tensor* check_logits(PyObject* list, Ranks* at, ar_route_shape_t* s) {
  const Py_ssize_t n = list_size(list, "logits");
  if (n < 0) return nullptr;
  if (n < 1 || n > AR_MAX_RANKS)
    return fail(PyExc_ValueError, "need the logits of 1 to %d ranks", AR_MAX_RANKS);
  const at::Tensor* first = gpu_tensor(PyList_GET_ITEM(list, 0), "logits");
  if (first == nullptr) return nullptr;
  const auto type = first->scalar_type();
  if (type != at::kFloat && type != at::kBFloat16)
    return fail(PyExc_TypeError, "unsupported dtype %s", c10::toString(type));
  if (first->dim() != 2 || first->size(1) < 1)
    return fail(PyExc_ValueError, "logits must be [tokens, experts]");
  const int64_t tokens = first->size(0), experts = first->size(1);
  const int64_t row = first->stride(0), col = first->stride(1);
  if ((col != 1 && experts > 1 && tokens > 0) || (tokens > 1 && row < experts))
    return fail(PyExc_ValueError, "a token's logits must lie next to each other, tokens apart");
  for (Py_ssize_t i = 0; i < n; ++i) {
    const at::Tensor* t = gpu_tensor(PyList_GET_ITEM(list, i), "logits");
    if (t == nullptr) return nullptr;
    if (t->scalar_type() != type || t->device() != first->device())
      return fail(PyExc_TypeError, "logits must share type and device");
    if (t->sizes() != first->sizes() || (tokens > 1 && t->stride(0) != row) ||
        (tokens > 0 && experts > 1 && t->stride(1) != 1))
      return fail(PyExc_ValueError, "logits must share shape and strides");
    at->p[i] = t->const_data_ptr();
  }
  s->nranks = static_cast<int>(n);
  s->tokens = static_cast<size_t>(tokens);
  s->experts = experts > INT32_MAX ? INT32_MAX : static_cast<int>(experts);
  s->row_stride = static_cast<size_t>(row > experts ? row : experts);
  s->dtype = type == at::kFloat ? AR_FLOAT32 : AR_BFLOAT16;
  return first;
}

// One contiguous tensor a rank, or None (then *given is false).
bool check_ranks(PyObject* list, const char* what, at::ScalarType type, at::IntArrayRef size,
                 const at::Tensor& logits, int n, Ranks* at, bool* given) {
  *given = list != Py_None;
  if (!*given) return true;
  const Py_ssize_t m = list_size(list, what);
  if (m < 0) return false;
  if (m != n) {
    fail(PyExc_ValueError, "%s: %zd tensors for %d ranks", what, m, n);
    return false;
  }
  for (Py_ssize_t i = 0; i < m; ++i) {
    const at::Tensor* t = gpu_tensor(PyList_GET_ITEM(list, i), what);
    if (t == nullptr) return false;
    if (t->scalar_type() != type || t->device() != logits.device()) {
      fail(PyExc_TypeError, "%s must be %s on the logits' device", what, c10::toString(type));
      return false;
    }
    if (t->sizes() != size || !t->is_contiguous()) {
      fail(PyExc_ValueError, "%s must be contiguous and of the logits' tokens", what);
      return false;
    }
    at->p[i] = t->const_data_ptr();
  }
  return true;
}

hipStream_t stream_of(PyObject* handle) { return static_cast<hipStream_t>(PyLong_AsVoidPtr(handle)); }

bool arguments(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  fail(PyExc_TypeError, "takes %zd arguments", want);
  return false;
}

// An empty contiguous tensor on the current device, which is the logits': what
// at::empty gives without its way through the dispatcher (about 0.6 us each).
// Every output has a storage of its own, so that each can be saved, kept and
// freed by itself.
at::Tensor empty(at::IntArrayRef size, at::ScalarType type) {
  static c10::Allocator* const allocator =
      at::empty({1}, at::TensorOptions(at::kFloat).device(c10::DeviceType::CUDA)).storage().allocator();
  return at::detail::empty_generic(size, allocator, c10::DispatchKeySet(c10::DispatchKey::CUDA), type, c10::nullopt);
}

// A tuple (status, tensors...).
PyObject* result(ar_status_t status, std::initializer_list<const at::Tensor*> tensors) {
  PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(tensors.size()) + 1);
  if (out == nullptr) return nullptr;
  PyTuple_SET_ITEM(out, 0, PyLong_FromLong(status));
  Py_ssize_t i = 1;
  for (const at::Tensor* t : tensors) PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(*t));
  return out;
}

// device(list): the index of the first tensor's device.
PyObject* device(PyObject*, PyObject* list) {
  HANDLE_TH_ERRORS
  Ranks at;
  ar_route_shape_t s;
  const at::Tensor* first = check_logits(list, &at, &s);
  return first == nullptr ? nullptr : PyLong_FromLong(first->get_device());
  END_HANDLE_TH_ERRORS
}

// route(logits, top_k, mask, renormalize, workspace, stream)
//   -> (status, indices, weights, counts, loss, share)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arguments(n, 6)) return nullptr;
  Ranks logits, masks;
  ar_route_shape_t s;
  const at::Tensor* first = check_logits(a[0], &logits, &s);
  if (first == nullptr) return nullptr;
  const long k = PyLong_AsLong(a[1]);
  if (k == -1 && PyErr_Occurred()) return nullptr;
  const int most = s.experts < AR_MAX_TOP_K ? s.experts : AR_MAX_TOP_K;
  if (k < 1 || k > most || s.experts > AR_MAX_EXPERTS)
    return fail(PyExc_ValueError, "top_k must be 1 to %d of at most %d experts, not %ld of %d", most,
                AR_MAX_EXPERTS, k, s.experts);
  const int64_t tokens = static_cast<int64_t>(s.tokens);
  bool masked;
  if (!check_ranks(a[2], "mask", at::kBool, {tokens}, *first, s.nranks, &masks, &masked)) return nullptr;
  s.top_k = static_cast<int>(k);
  if ((s.renormalize = PyObject_IsTrue(a[3])) < 0) return nullptr;
  const at::Tensor indices = empty({s.nranks, tokens, k}, at::kInt);
  const at::Tensor weights = empty({s.nranks, tokens, k}, at::kFloat);
  const at::Tensor counts = empty({s.nranks, s.experts}, at::kInt);
  const at::Tensor share = empty({s.experts}, at::kFloat);
  const at::Tensor loss = empty({}, at::kFloat);
  const ar_status_t status = ar_route(
      logits.p, masked ? reinterpret_cast<const uint8_t* const*>(masks.p) : nullptr, &s,
      static_cast<int32_t*>(indices.data_ptr()), static_cast<float*>(weights.data_ptr()),
      static_cast<int32_t*>(counts.data_ptr()), static_cast<float*>(loss.data_ptr()),
      static_cast<float*>(share.data_ptr()), PyLong_AsVoidPtr(a[4]), stream_of(a[5]));
  return result(status, {&indices, &weights, &counts, &loss, &share});
  END_HANDLE_TH_ERRORS
}

// route_grad(logits, dtype, indices, share, mask, renormalize, dweights, dloss, stream)
//   -> (status, dlogits)
PyObject* route_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arguments(n, 9)) return nullptr;
  Ranks logits, masks, dweights;
  ar_route_shape_t s;
  const at::Tensor* first = check_logits(a[0], &logits, &s);
  if (first == nullptr) return nullptr;
  const at::Tensor* indices = gpu_tensor(a[2], "indices");
  const at::Tensor* share = indices == nullptr ? nullptr : gpu_tensor(a[3], "share");
  if (share == nullptr) return nullptr;
  const int64_t tokens = static_cast<int64_t>(s.tokens);
  // a Routing's tensors are plain attributes: what the kernel reads is checked here
  if (indices->dim() != 3 || indices->size(0) != s.nranks || indices->size(1) != tokens ||
      share->numel() != s.experts || indices->device() != first->device() ||
      share->device() != first->device() || !THPDtype_Check(a[1]) ||
      reinterpret_cast<THPDtype*>(a[1])->scalar_type != first->scalar_type())
    return fail(PyExc_ValueError, "these are not the logits of this routing");
  if (indices->scalar_type() != at::kInt || share->scalar_type() != at::kFloat)
    return fail(PyExc_TypeError, "need int32 indices and a float32 share, not %s and %s",
                c10::toString(indices->scalar_type()), c10::toString(share->scalar_type()));
  if (!indices->is_contiguous() || !share->is_contiguous())
    return fail(PyExc_ValueError, "indices and share must be contiguous");
  if (indices->size(2) < 1 || indices->size(2) > AR_MAX_TOP_K || indices->size(2) > s.experts)
    return fail(PyExc_ValueError, "indices must hold 1 to %d choices a token", AR_MAX_TOP_K);
  s.top_k = static_cast<int>(indices->size(2));
  if ((s.renormalize = PyObject_IsTrue(a[5])) < 0) return nullptr;
  bool masked, weighted;
  if (!check_ranks(a[4], "mask", at::kBool, {tokens}, *first, s.nranks, &masks, &masked) ||
      !check_ranks(a[6], "dweights", at::kFloat, {tokens, s.top_k}, *first, s.nranks, &dweights, &weighted))
    return nullptr;
  const at::Tensor* dloss = nullptr;
  if (a[7] != Py_None) {
    dloss = gpu_tensor(a[7], "dloss");
    if (dloss == nullptr) return nullptr;
    if (dloss->scalar_type() != at::kFloat || dloss->device() != first->device() || dloss->numel() != 1)
      return fail(PyExc_ValueError, "dloss must be one float32 on the logits' device");
  }
  const at::Tensor dlogits = at::empty({s.nranks, tokens, s.experts}, first->options());
  const ar_status_t status = ar_route_grad(
      logits.p, masked ? reinterpret_cast<const uint8_t* const*>(masks.p) : nullptr, &s,
      static_cast<const int32_t*>(indices->const_data_ptr()), static_cast<const float*>(share->const_data_ptr()),
      weighted ? reinterpret_cast<const float* const*>(dweights.p) : nullptr,
      dloss == nullptr ? nullptr : static_cast<const float*>(dloss->const_data_ptr()), dlogits.data_ptr(),
      stream_of(a[8]));
  return result(status, {&dlogits});
  END_HANDLE_TH_ERRORS
}

// dequantize(codes, scales, stream) -> (status, values)
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arguments(n, 3)) return nullptr;
  const at::Tensor* codes = gpu_tensor(a[0], "codes and scales");
  const at::Tensor* scales = codes == nullptr ? nullptr : gpu_tensor(a[1], "codes and scales");
  if (scales == nullptr) return nullptr;
  const auto type = codes->scalar_type();
  if ((type != at::kChar && type != at::kByte) || scales->scalar_type() != at::kFloat)
    return fail(PyExc_TypeError, "need int8 or uint8 codes and float32 scales, not %s and %s",
                c10::toString(type), c10::toString(scales->scalar_type()));
  const int64_t count = codes->numel(), blocks = (count + AR_ADAMW_BLOCK - 1) / AR_ADAMW_BLOCK;
  if (scales->numel() != blocks || scales->device() != codes->device())
    return fail(PyExc_ValueError, "%lld codes need %lld scales on their device", static_cast<long long>(count),
                static_cast<long long>(blocks));
  if (!codes->is_contiguous() || !scales->is_contiguous())
    return fail(PyExc_ValueError, "codes and scales must be contiguous");
  const at::Tensor out = at::empty(codes->sizes(), codes->options().dtype(at::kFloat));
  const ar_status_t status = ar_adamw_dequantize(
      codes->const_data_ptr(), static_cast<const float*>(scales->const_data_ptr()), static_cast<size_t>(count),
      type == at::kChar, static_cast<float*>(out.data_ptr()), stream_of(a[2]));
  return result(status, {&out});
  END_HANDLE_TH_ERRORS
}

// --- the experts' products ---------------------------------------------------------

// A contiguous int32 tensor on a GPU, of `count` elements where that is not negative.
const at::Tensor* int32_tensor(PyObject* o, const char* what, int64_t count) {
  const at::Tensor* t = gpu_tensor(o, what);
  if (t == nullptr) return nullptr;
  if (t->scalar_type() != at::kInt) return fail(PyExc_TypeError, "%s must be int32, not %s", what, c10::toString(t->scalar_type()));
  if (!t->is_contiguous()) return fail(PyExc_ValueError, "%s must be contiguous", what);
  if (count >= 0 && t->numel() != count)
    return fail(PyExc_ValueError, "%s must hold %lld numbers, not %lld", what, static_cast<long long>(count),
                static_cast<long long>(t->numel()));
  return t;
}

// A bfloat16 matrix whose rows lie apart, each contiguous; `rows` and `cols` where
// they are not negative.
const at::Tensor* matrix(PyObject* o, const char* what, int64_t rows, int64_t cols, size_t* stride) {
  const at::Tensor* t = gpu_tensor(o, what);
  if (t == nullptr) return nullptr;
  if (t->scalar_type() != at::kBFloat16)
    return fail(PyExc_TypeError, "%s must be bfloat16, not %s", what, c10::toString(t->scalar_type()));
  if (t->dim() != 2 || t->size(1) < 1) return fail(PyExc_ValueError, "%s must be a matrix with columns", what);
  if ((rows >= 0 && t->size(0) != rows) || (cols >= 0 && t->size(1) != cols))
    return fail(PyExc_ValueError, "%s must be [%lld, %lld], not [%lld, %lld]", what,
                static_cast<long long>(rows >= 0 ? rows : t->size(0)), static_cast<long long>(cols >= 0 ? cols : t->size(1)),
                static_cast<long long>(t->size(0)), static_cast<long long>(t->size(1)));
  if (t->size(0) > 0 && ((t->size(1) > 1 && t->stride(1) != 1) || (t->size(0) > 1 && t->stride(0) < t->size(1))))
    return fail(PyExc_ValueError, "a row of %s must lie next to each other, rows apart", what);
  *stride = static_cast<size_t>(t->size(0) > 1 ? t->stride(0) : t->size(1));
  return t;
}

// What the experts' calls need of Python: torch's current device and stream (of
// a device), the classes of an order and of a library error, attributes' names.
struct Hooks {
  PyObject *device, *stream, *order_class, *error_class;
  PyObject *order, *position, *offsets, *top_k;
} hooks;

// hooks(current device, current stream, ExpertOrder, ArError)
PyObject* set_hooks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arguments(n, 4)) return nullptr;
  for (Py_ssize_t i = 0; i < 4; ++i) Py_INCREF(a[i]);
  hooks = {a[0], a[1], a[2], a[3], PyUnicode_InternFromString("order"), PyUnicode_InternFromString("position"),
           PyUnicode_InternFromString("offsets"), PyUnicode_InternFromString("top_k")};
  Py_RETURN_NONE;
}

// The device of the calls' first tensor, if it is the current one, and its current
// stream.  Otherwise false, with an error, or without one where another device is
// current: the caller has to change to it (and gets None).
bool on_current(PyObject* first, const char* what, hipStream_t* stream) {
  const at::Tensor* t = gpu_tensor(first, what);
  if (t == nullptr) return false;
  PyObject* current = PyObject_CallNoArgs(hooks.device);
  if (current == nullptr) return false;
  const long device = PyLong_AsLong(current);
  PyObject* handle = device == t->get_device() ? PyObject_CallOneArg(hooks.stream, current) : nullptr;
  Py_DECREF(current);
  if (handle == nullptr) return false;
  *stream = stream_of(handle);
  Py_DECREF(handle);
  return !PyErr_Occurred();
}

PyObject* elsewhere() {
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

// The tensor, or an ArError.
PyObject* checked(ar_status_t status, const char* call, const at::Tensor& t) {
  if (status == AR_SUCCESS) return THPVariable_Wrap(t);
  PyObject* error = PyObject_CallFunction(hooks.error_class, "is", static_cast<int>(status), call);
  if (error != nullptr) PyErr_SetObject(hooks.error_class, error);
  Py_XDECREF(error);
  return nullptr;
}
PyObject* checked(ar_status_t status, const char* call, std::initializer_list<const at::Tensor*> tensors) {
  PyObject* out = checked(status, call, **tensors.begin());
  if (out == nullptr) return nullptr;
  PyObject* tuple = PyTuple_New(static_cast<Py_ssize_t>(tensors.size()));
  if (tuple == nullptr) {
    Py_DECREF(out);
    return nullptr;
  }
  PyTuple_SET_ITEM(tuple, 0, out);
  for (size_t i = 1; i < tensors.size(); ++i)
    PyTuple_SET_ITEM(tuple, static_cast<Py_ssize_t>(i), THPVariable_Wrap(**(tensors.begin() + i)));
  return tuple;
}

// What expert_order found.  Its attributes are plain, so what the kernels read is
// checked; their tensors are held for the call.
struct Order {
  at::Tensor order, position, offsets;
  int64_t pairs, tokens;
  int experts, top_k;
};

// An attribute that is a contiguous int32 tensor of `count` elements (any if negative).
bool attribute(PyObject* from, PyObject* name, const char* what, int64_t count, at::Tensor* to) {
  PyObject* o = PyObject_GetAttr(from, name);
  if (o == nullptr) return false;
  const at::Tensor* t = int32_tensor(o, what, count);
  if (t != nullptr) *to = *t;
  Py_DECREF(o);
  return t != nullptr;
}

bool check_order(PyObject* from, Order* o) {
  if (!PyObject_TypeCheck(from, reinterpret_cast<PyTypeObject*>(hooks.order_class))) {
    fail(PyExc_TypeError, "order must be what expert_order returned");
    return false;
  }
  PyObject* number = PyObject_GetAttr(from, hooks.top_k);
  if (number == nullptr) return false;
  const long k = PyLong_AsLong(number);
  Py_DECREF(number);
  if (k == -1 && PyErr_Occurred()) return false;
  if (!attribute(from, hooks.order, "order", -1, &o->order)) return false;
  o->pairs = o->order.numel();
  if (!attribute(from, hooks.position, "position", o->pairs, &o->position) ||
      !attribute(from, hooks.offsets, "offsets", -1, &o->offsets))
    return false;
  if (k < 1 || k > INT32_MAX || o->pairs % k != 0 || o->offsets.numel() < 2 ||
      o->offsets.numel() > AR_MAX_EXPERTS + 1 || o->position.device() != o->order.device() ||
      o->offsets.device() != o->order.device()) {
    fail(PyExc_ValueError, "this is not the order of top_k choices a token");
    return false;
  }
  o->top_k = static_cast<int>(k);
  o->tokens = o->pairs / k;
  o->experts = static_cast<int>(o->offsets.numel() - 1);
  return true;
}

bool same_device(const Order& o, std::initializer_list<const at::Tensor*> tensors) {
  for (const at::Tensor* t : tensors)
    if (t->device() != o.order.device()) {
      fail(PyExc_ValueError, "all tensors must be on the order's device");
      return false;
    }
  return true;
}

ar_expert_rows_t rows_of(const Order& o, const at::Tensor& x, size_t stride, bool gather, int64_t out) {
  ar_expert_rows_t r;
  r.x = x.const_data_ptr();
  r.x_rows = static_cast<size_t>(x.size(0));
  r.x_stride = stride;
  r.order = gather ? static_cast<const int32_t*>(o.order.const_data_ptr()) : nullptr;
  r.top_k = o.top_k;
  r.offsets = static_cast<const int32_t*>(o.offsets.const_data_ptr());
  r.pairs = static_cast<size_t>(o.pairs);
  r.experts = o.experts;
  r.in = static_cast<size_t>(x.size(1));
  r.out = static_cast<size_t>(out);
  r.dtype = AR_BFLOAT16;
  return r;
}

// The calls below return None where another device than their tensors' is current.

// expert_order(indices, experts) -> (order, position, offsets)
PyObject* expert_order(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arguments(n, 2)) return nullptr;
  hipStream_t stream;
  if (!on_current(a[0], "indices", &stream)) return elsewhere();
  const at::Tensor* indices = int32_tensor(a[0], "indices", -1);
  if (indices == nullptr) return nullptr;
  const long experts = PyLong_AsLong(a[1]);
  if (experts == -1 && PyErr_Occurred()) return nullptr;
  if (experts < 1 || experts > AR_MAX_EXPERTS)
    return fail(PyExc_ValueError, "experts must be 1 to %d, not %ld", AR_MAX_EXPERTS, experts);
  if (indices->dim() < 1 || indices->size(-1) < 1)
    return fail(PyExc_ValueError, "indices must be [..., top_k]");
  const int64_t pairs = indices->numel();
  const at::Tensor order = empty({pairs}, at::kInt), position = empty(indices->sizes(), at::kInt);
  const at::Tensor offsets = empty({experts + 1}, at::kInt);
  const size_t bytes = ar_expert_order_workspace(static_cast<size_t>(pairs), static_cast<int>(experts));
  at::Tensor workspace;
  if (bytes != 0) workspace = empty({static_cast<int64_t>(bytes)}, at::kByte);
  const ar_status_t status = ar_expert_order(
      static_cast<const int32_t*>(indices->const_data_ptr()), static_cast<size_t>(pairs), static_cast<int>(experts),
      static_cast<int32_t*>(order.data_ptr()), static_cast<int32_t*>(position.data_ptr()),
      static_cast<int32_t*>(offsets.data_ptr()), bytes != 0 ? workspace.data_ptr() : nullptr, stream);
  return checked(status, "expert_order", {&order, &position, &offsets});
  END_HANDLE_TH_ERRORS
}

// expert_matmul(x, weight, order, gather) -> y
PyObject* expert_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arguments(n, 4)) return nullptr;
  Order o;
  hipStream_t stream;
  if (!check_order(a[2], &o)) return nullptr;
  if (!on_current(a[0], "x", &stream)) return elsewhere();
  const int gather = PyObject_IsTrue(a[3]);
  if (gather < 0) return nullptr;
  size_t stride;
  const at::Tensor* x = matrix(a[0], "x", gather ? o.tokens : o.pairs, -1, &stride);
  if (x == nullptr) return nullptr;
  const at::Tensor* w = gpu_tensor(a[1], "weight");
  if (w == nullptr) return nullptr;
  if (w->scalar_type() != at::kBFloat16)
    return fail(PyExc_TypeError, "weight must be bfloat16, not %s", c10::toString(w->scalar_type()));
  if (w->dim() != 3 || w->size(0) != o.experts || w->size(1) != x->size(1) || w->size(2) < 1)
    return fail(PyExc_ValueError, "weight must be [%d experts, %lld, size]", o.experts,
                static_cast<long long>(x->size(1)));
  const int64_t in = w->size(1), out = w->size(2), si = w->stride(1), so = w->stride(2);
  if (!((out == 1 || so == 1) && (in == 1 || si >= out)) && !((in == 1 || si == 1) && (out == 1 || so >= in)))
    return fail(PyExc_ValueError, "an expert's rows or its columns must lie next to each other");
  if (!same_device(o, {x, w})) return nullptr;
  const ar_expert_rows_t rows = rows_of(o, *x, stride, gather, out);
  const at::Tensor y = empty({o.pairs, out}, at::kBFloat16);
  const ar_status_t status = ar_expert_matmul(&rows, w->const_data_ptr(), static_cast<size_t>(w->stride(0)),
                                              static_cast<size_t>(si), static_cast<size_t>(so), y.data_ptr(),
                                              stream);
  return checked(status, "expert_matmul", y);
  END_HANDLE_TH_ERRORS
}

// expert_weight_grad(x, dy, order, gather, wide, out) -> dw
PyObject* expert_weight_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arguments(n, 6)) return nullptr;
  Order o;
  hipStream_t stream;
  if (!check_order(a[2], &o)) return nullptr;
  if (!on_current(a[0], "x", &stream)) return elsewhere();
  const int gather = PyObject_IsTrue(a[3]), wide = PyObject_IsTrue(a[4]);
  if (gather < 0 || wide < 0) return nullptr;
  size_t stride, dy_stride;
  const at::Tensor* x = matrix(a[0], "x", gather ? o.tokens : o.pairs, -1, &stride);
  const at::Tensor* dy = x == nullptr ? nullptr : matrix(a[1], "dy", o.pairs, -1, &dy_stride);
  if (dy == nullptr || !same_device(o, {x, dy})) return nullptr;
  at::Tensor dw;
  if (a[5] != Py_None) {
    const at::Tensor* out = gpu_tensor(a[5], "out");
    if (out == nullptr) return nullptr;
    if (out->scalar_type() != at::kFloat && out->scalar_type() != at::kBFloat16)
      return fail(PyExc_TypeError, "out must be float32 or bfloat16, not %s", c10::toString(out->scalar_type()));
    if (out->dim() != 3 || out->size(0) != o.experts || out->size(1) != x->size(1) || out->size(2) != dy->size(1) ||
        !out->is_contiguous())
      return fail(PyExc_ValueError, "out must be contiguous, [%d, %lld, %lld]", o.experts,
                  static_cast<long long>(x->size(1)), static_cast<long long>(dy->size(1)));
    if (!same_device(o, {out})) return nullptr;
    dw = *out;
  } else {
    dw = empty({o.experts, x->size(1), dy->size(1)}, wide ? at::kFloat : at::kBFloat16);
  }
  const ar_expert_rows_t rows = rows_of(o, *x, stride, gather, dy->size(1));
  const size_t bytes = ar_expert_weight_grad_workspace(rows.pairs, rows.experts, rows.in, rows.out);
  at::Tensor workspace;
  if (bytes != 0) workspace = empty({static_cast<int64_t>(bytes)}, at::kByte);
  const ar_status_t status = ar_expert_weight_grad(&rows, dy->const_data_ptr(), dy_stride, dw.data_ptr(),
                                                   dw.scalar_type() == at::kFloat ? AR_FLOAT32 : AR_BFLOAT16,
                                                   bytes != 0 ? workspace.data_ptr() : nullptr, stream);
  if (a[5] != Py_None && status == AR_SUCCESS && !dw.is_inference()) dw.unsafeGetTensorImpl()->bump_version();
  return checked(status, "expert_weight_grad", dw);
  END_HANDLE_TH_ERRORS
}

// The weights of a token's choices, contiguous float32; false on an error.
bool check_weights(PyObject* p, const Order& o, const float** at) {
  const at::Tensor* t = gpu_tensor(p, "weights");
  if (t == nullptr) return false;
  if (t->scalar_type() != at::kFloat) {
    fail(PyExc_TypeError, "weights must be float32, not %s", c10::toString(t->scalar_type()));
    return false;
  }
  if (t->numel() != o.pairs || !t->is_contiguous()) {
    fail(PyExc_ValueError, "weights must be contiguous, one for each of the %lld pairs", static_cast<long long>(o.pairs));
    return false;
  }
  *at = static_cast<const float*>(t->const_data_ptr());
  return same_device(o, {t});
}

// expert_combine(y, order, weights) -> out
PyObject* expert_combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arguments(n, 3)) return nullptr;
  Order o;
  hipStream_t stream;
  if (!check_order(a[1], &o)) return nullptr;
  if (!on_current(a[0], "y", &stream)) return elsewhere();
  size_t stride;
  const at::Tensor* y = matrix(a[0], "y", o.pairs, -1, &stride);
  if (y == nullptr || !same_device(o, {y})) return nullptr;
  const float* weights = nullptr;
  if (a[2] != Py_None && !check_weights(a[2], o, &weights)) return nullptr;
  const at::Tensor out = empty({o.tokens, y->size(1)}, at::kBFloat16);
  const ar_status_t status = ar_expert_combine(
      y->const_data_ptr(), stride, static_cast<size_t>(o.pairs), static_cast<size_t>(y->size(1)), AR_BFLOAT16,
      static_cast<const int32_t*>(o.position.const_data_ptr()), weights, static_cast<size_t>(o.tokens), o.top_k,
      out.data_ptr(), stream);
  return checked(status, "expert_combine", out);
  END_HANDLE_TH_ERRORS
}

// expert_combine_grad(dout, y, order, weights) -> (dy, dweights)
PyObject* expert_combine_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arguments(n, 4)) return nullptr;
  Order o;
  hipStream_t stream;
  if (!check_order(a[2], &o)) return nullptr;
  if (!on_current(a[0], "dout", &stream)) return elsewhere();
  size_t dout_stride, y_stride;
  const at::Tensor* y = matrix(a[1], "y", o.pairs, -1, &y_stride);
  const at::Tensor* dout = y == nullptr ? nullptr : matrix(a[0], "dout", o.tokens, y->size(1), &dout_stride);
  if (dout == nullptr || !same_device(o, {y, dout})) return nullptr;
  const float* weights = nullptr;
  if (!check_weights(a[3], o, &weights)) return nullptr;
  const at::Tensor dy = empty({o.pairs, y->size(1)}, at::kBFloat16);
  const at::Tensor dweights = empty({o.tokens, o.top_k}, at::kFloat);
  const ar_status_t status = ar_expert_combine_grad(
      dout->const_data_ptr(), dout_stride, y->const_data_ptr(), y_stride, static_cast<size_t>(o.pairs),
      static_cast<size_t>(y->size(1)), AR_BFLOAT16, static_cast<const int32_t*>(o.position.const_data_ptr()),
      static_cast<const int32_t*>(o.offsets.const_data_ptr()), o.experts, weights, static_cast<size_t>(o.tokens),
      o.top_k, dy.data_ptr(), static_cast<float*>(dweights.data_ptr()), stream);
  return checked(status, "expert_combine_grad", {&dy, &dweights});
  END_HANDLE_TH_ERRORS
}

// written(list): tells autograd that these tensors were written in place (their
// version counters; tensors made in inference mode have none).
PyObject* written(PyObject*, PyObject* list) {
  HANDLE_TH_ERRORS
  const Py_ssize_t n = list_size(list, "tensors");
  if (n < 0) return nullptr;
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* o = PyList_GET_ITEM(list, i);
    if (!THPVariable_Check(o)) return fail(PyExc_TypeError, "tensors must be tensors");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  }
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

template <class F> PyCFunction as_function(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)); }

PyMethodDef methods[] = {
    {"device", device, METH_O, nullptr},
    {"route", as_function(route), METH_FASTCALL, nullptr},
    {"route_grad", as_function(route_grad), METH_FASTCALL, nullptr},
    {"dequantize", as_function(dequantize), METH_FASTCALL, nullptr},
    {"hooks", as_function(set_hooks), METH_FASTCALL, nullptr},
    {"expert_order", as_function(expert_order), METH_FASTCALL, nullptr},
    {"expert_matmul", as_function(expert_matmul), METH_FASTCALL, nullptr},
    {"expert_weight_grad", as_function(expert_weight_grad), METH_FASTCALL, nullptr},
    {"expert_combine", as_function(expert_combine), METH_FASTCALL, nullptr},
    {"expert_combine_grad", as_function(expert_combine_grad), METH_FASTCALL, nullptr},
    {"written", written, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_training", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__training() { return PyModule_Create(&module); }
