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
    {"written", written, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_training", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__training() { return PyModule_Create(&module); }
