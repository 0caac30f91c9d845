// The Python binding's way from tensors to the library's calls: addresses, sizes, strides and types
// are checked and gathered, outputs and workspaces allocated, and the call made, on the current
// stream of the tensors' device.  From Python each tensor of a list costs 0.35 us, here 0.02 (146
// tensors 51 and 3 us), and a call through ctypes, with its outputs' allocation, 5 us.  No
// arithmetic happens here.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <vector>

#include "../../include/flce_train.h"

namespace {

constexpr int32_t kF32 = FLCE_DTYPE_F32, kBf16 = FLCE_DTYPE_BF16;

// The library's entry points, given by `bind`.
struct Library {
  decltype(&flce_qk_norm_rope_forward) forward;
  decltype(&flce_qk_norm_rope_backward) backward;
  decltype(&flce_qk_norm_rope_workspace_bytes) qk_workspace;
  decltype(&flce_grad_norm) norm;
  decltype(&flce_grad_norm_workspace_bytes) norm_workspace;
} library{};

// bind(five addresses, in the order of `Library`)
PyObject* bind(PyObject* const* args, Py_ssize_t count) {
  if (count != 5) {
    PyErr_SetString(PyExc_TypeError, "bind takes 5 addresses");
    return nullptr;
  }
  void* address[5];
  for (int i = 0; i < 5; ++i) {
    address[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  library.forward = reinterpret_cast<decltype(library.forward)>(address[0]);
  library.backward = reinterpret_cast<decltype(library.backward)>(address[1]);
  library.qk_workspace = reinterpret_cast<decltype(library.qk_workspace)>(address[2]);
  library.norm = reinterpret_cast<decltype(library.norm)>(address[3]);
  library.norm_workspace = reinterpret_cast<decltype(library.norm_workspace)>(address[4]);
  Py_RETURN_NONE;
}

// Runs a call of the library with the tensors' device current and without the interpreter's lock, as
// torch launches its own operators.
template <typename F>
int on_device(int device, F&& call) {
  const int before = c10::cuda::current_device();
  if (before != device) c10::cuda::set_device(static_cast<c10::DeviceIndex>(device));
  void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = call(stream);
  Py_END_ALLOW_THREADS;
  if (before != device) c10::cuda::set_device(static_cast<c10::DeviceIndex>(before));
  return rc;
}
// A new dense tensor on another's device, from torch's allocator without its dispatcher (1.1 us each).
at::Tensor dense(const at::Tensor& like, at::IntArrayRef size, at::ScalarType type) {
  return at::Tensor(at::detail::empty_cuda(size, type, like.device(), std::nullopt));
}
at::Tensor bytes_on(const at::Tensor& like, size_t n) {
  return dense(like, {static_cast<int64_t>(n)}, at::kByte);
}

// The tensor of a Python object; nullptr with an exception set when it is none.
const at::Tensor* tensor_of(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor, got %s", what, Py_TYPE(o)->tp_name);
    return nullptr;
  }
  return &THPVariable_Unpack(o);
}

// Elements without an address: a wrapper around tensors that lie elsewhere (a sharded one, say).  The
// library takes NULL for an argument that is not given, so these must not reach it.
bool lies_elsewhere(const at::Tensor& t) { return t.numel() > 0 && t.const_data_ptr() == nullptr; }

// Its FLCE_DTYPE_*; -1 with an exception set when the library cannot read it.
int32_t code_of(const at::Tensor& t, int device, const char* what) {
  if (!t.is_cuda() || (device >= 0 && t.get_device() != device)) {
    PyErr_Format(PyExc_ValueError, "every %s must be on one CUDA device", what);
    return -1;
  }
  const auto type = t.scalar_type();
  if (type != at::kFloat && type != at::kBFloat16) {
    PyErr_Format(PyExc_TypeError, "every %s must be float32 or bfloat16, got %s", what,
                 c10::toString(type));
    return -1;
  }
  if (t.layout() != at::kStrided || !t.is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "every %s must be contiguous", what);
    return -1;
  }
  if (lies_elsewhere(t)) {
    PyErr_Format(PyExc_ValueError, "every %s must have memory of its own (a sharded tensor's local "
                 "part has)", what);
    return -1;
  }
  return type == at::kBFloat16 ? kBf16 : kF32;
}

// An owned reference that goes with the scope.
struct Held {
  PyObject* o;
  explicit Held(PyObject* p) : o(p) {}
  ~Held() { Py_XDECREF(o); }
  Held(const Held&) = delete;
  Held& operator=(const Held&) = delete;
  explicit operator bool() const { return o != nullptr; }
};
template <typename T>
T* data_of(const Held& bytes) {
  return reinterpret_cast<T*>(PyBytes_AS_STRING(bytes.o));
}

// A tensor that a call changes in place: a graph that saved it raises instead of using the
// new values.
void changes(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// gradients(gradients, parameters, device, types) -> (addresses, types, parameters' places): each
// gradient, where it is not None, checked against its parameter's shape.  An entry without one has
// address 0 and keeps its type of `types` (bytes of int32).  A place, three words, changes when the
// parameter is given other memory, another size, type, layout or device.
PyObject* gradients(PyObject* const* args, Py_ssize_t count) {
  if (count != 4 || !PyBytes_Check(args[3])) {
    PyErr_SetString(PyExc_TypeError, "gradients(gradients, parameters, device, types)");
    return nullptr;
  }
  Held grads(PySequence_Fast(args[0], "a list of gradients is wanted"));
  Held params(PySequence_Fast(args[1], "a list of parameters is wanted"));
  if (!grads || !params) return nullptr;
  const long device = PyLong_AsLong(args[2]);
  if (device == -1 && PyErr_Occurred()) return nullptr;
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(params.o);
  if (PySequence_Fast_GET_SIZE(grads.o) != n || PyBytes_GET_SIZE(args[3]) != 4 * n) {
    PyErr_Format(PyExc_ValueError, "%zd gradients wanted, got %zd", n,
                 PySequence_Fast_GET_SIZE(grads.o));
    return nullptr;
  }
  Held addresses(PyBytes_FromStringAndSize(nullptr, 8 * n));
  Held types(PyBytes_FromStringAndSize(PyBytes_AS_STRING(args[3]), 4 * n));
  Held places(PyBytes_FromStringAndSize(nullptr, 24 * n));
  if (!addresses || !types || !places) return nullptr;
  if (n == 0) return Py_BuildValue("OOO", addresses.o, types.o, places.o);
  for (Py_ssize_t i = 0; i < n; ++i) {
    const at::Tensor* p = tensor_of(PySequence_Fast_GET_ITEM(params.o, i), "a parameter");
    if (p == nullptr) return nullptr;
    uint64_t* place = data_of<uint64_t>(places) + 3 * i;
    place[0] = reinterpret_cast<uint64_t>(p->data_ptr());
    place[1] = static_cast<uint64_t>(p->numel());
    place[2] = static_cast<uint64_t>(p->scalar_type()) | (p->is_contiguous() ? 256u : 0u) |
               (p->is_cuda() ? static_cast<uint64_t>(p->get_device() + 1) << 16 : 0u);
    uint64_t address = 0;
    PyObject* o = PySequence_Fast_GET_ITEM(grads.o, i);
    if (o != Py_None) {
      const at::Tensor* g = tensor_of(o, "a gradient");
      if (g == nullptr) return nullptr;
      const int32_t code = code_of(*g, static_cast<int>(device), "gradient");
      if (code < 0) return nullptr;
      if (!g->sizes().equals(p->sizes())) {
        PyErr_Format(PyExc_ValueError, "gradient %zd has another shape than its parameter", i);
        return nullptr;
      }
      address = reinterpret_cast<uint64_t>(g->data_ptr());
      data_of<int32_t>(types)[i] = code;
    }
    data_of<uint64_t>(addresses)[i] = address;
  }
  return Py_BuildValue("OOO", addresses.o, types.o, places.o);
}
// stepped(gradients, parameters): the parameters with a gradient have been changed.
PyObject* stepped(PyObject* const* args, Py_ssize_t count) {
  if (count != 2) {
    PyErr_SetString(PyExc_TypeError, "stepped(gradients, parameters)");
    return nullptr;
  }
  Held grads(PySequence_Fast(args[0], "a list of gradients is wanted"));
  Held params(PySequence_Fast(args[1], "a list of parameters is wanted"));
  if (!grads || !params) return nullptr;
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(params.o);
  if (PySequence_Fast_GET_SIZE(grads.o) != n) {
    PyErr_Format(PyExc_ValueError, "%zd gradients wanted, got %zd", n,
                 PySequence_Fast_GET_SIZE(grads.o));
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (PySequence_Fast_GET_ITEM(grads.o, i) == Py_None) continue;
    const at::Tensor* p = tensor_of(PySequence_Fast_GET_ITEM(params.o, i), "a parameter");
    if (p == nullptr) return nullptr;
    changes(*p);
  }
  Py_RETURN_NONE;
}

// ------------------------------------------------------------------------------ gradient norm
// grad_norm(list, max_norm or None) -> (status, norm, factor or None), or None when the list has no
// gradient.
PyObject* grad_norm(PyObject* const* args, Py_ssize_t count) {
  if (count != 2) {
    PyErr_SetString(PyExc_TypeError, "grad_norm(list, max_norm)");
    return nullptr;
  }
  Held seq(PySequence_Fast(args[0], "a list of gradients is wanted"));
  if (!seq) return nullptr;
  const bool clip = args[1] != Py_None;
  const float max_norm = clip ? static_cast<float>(PyFloat_AsDouble(args[1])) : 0.f;
  if (PyErr_Occurred()) return nullptr;
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq.o);
  std::vector<const void*> addresses(n);
  std::vector<int64_t> sizes(n);
  std::vector<int32_t> types(n);
  at::Tensor some;
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* o = PySequence_Fast_GET_ITEM(seq.o, i);
    if (o == Py_None) continue;
    const at::Tensor* t = tensor_of(o, "a gradient");
    if (t == nullptr || (types[i] = code_of(*t, some.defined() ? some.get_device() : -1,
                                            "gradient")) < 0)
      return nullptr;
    if (!some.defined()) some = *t;
    addresses[i] = t->data_ptr();
    sizes[i] = t->numel();
  }
  if (!some.defined()) Py_RETURN_NONE;
  const at::Tensor norm = dense(some, {}, at::kFloat);
  const at::Tensor factor = clip ? dense(some, {}, at::kFloat) : at::Tensor();
  const size_t bytes = library.norm_workspace(n);
  const at::Tensor ws = bytes_on(some, bytes);
  float *to = static_cast<float*>(norm.data_ptr()),
        *factor_to = clip ? static_cast<float*>(factor.data_ptr()) : nullptr;
  void* workspace = ws.data_ptr();
  const int rc = on_device(some.get_device(), [&](void* stream) {
    return library.norm(addresses.data(), sizes.data(), types.data(), n, max_norm, to, factor_to,
                        workspace, bytes, stream);
  });
  return Py_BuildValue("iNN", rc, THPVariable_Wrap(norm),
                       clip ? THPVariable_Wrap(factor) : Py_NewRef(Py_None));
}

// ------------------------------------------------------------------------------ queries and keys
// These take what is right and answer None for anything else: the binding's own checks then say what
// is wrong.
const at::Tensor* cuda_tensor(PyObject* o) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.is_cuda() && t.layout() == at::kStrided && !lies_elsewhere(t) ? &t : nullptr;
}
bool element_type(const at::Tensor& t, int32_t* code) {
  const auto type = t.scalar_type();
  *code = type == at::kBFloat16 ? kBf16 : kF32;
  return type == at::kFloat || type == at::kBFloat16;
}
// Rows [T, H, D] or [B, T, H, D] with a dense last dimension, as a view of the library.
bool view_of(const at::Tensor& t, flce_qk_view* v, int64_t (&shape)[4]) {
  const int64_t n = t.dim();
  if (n != 3 && n != 4) return false;
  const auto sizes = t.sizes(), strides = t.strides();
  if (strides[n - 1] != 1 && sizes[n - 1] > 1) return false;
  shape[0] = n == 4 ? sizes[0] : 1;
  for (int i = 1; i < 4; ++i) shape[i] = sizes[n - 4 + i];
  *v = flce_qk_view{t.data_ptr(), n == 4 ? strides[0] : 0, strides[n - 3], strides[n - 2]};
  return true;
}
// A dense vector of n elements on q's device; its address, nullptr for None.
bool vector_of(PyObject* o, const at::Tensor& q, at::ScalarType type, int64_t n, void** address) {
  *address = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = cuda_tensor(o);
  if (t == nullptr || t->get_device() != q.get_device() || t->scalar_type() != type ||
      t->dim() != 1 || t->size(0) != n || !t->is_contiguous())
    return false;
  *address = t->data_ptr();
  return true;
}
// The arguments that forward and backward share: q, k, gamma_q, gamma_k, inv_freq, positions, eps,
// interleaved.
struct QkInputs {
  const at::Tensor *q, *k;             // k: nullptr without keys
  flce_qk_shape shape;
  flce_qk_view q_view, k_view;
  void *gamma[2], *inv_freq;
  const int64_t* positions;
  int64_t positions_batch;
  at::ScalarType gamma_type;
  const flce_qk_view* keys(const flce_qk_view& v) const { return k != nullptr ? &v : nullptr; }
};
bool qk_inputs(PyObject* const* args, QkInputs* in) {
  const at::Tensor* q = in->q = cuda_tensor(args[0]);
  flce_qk_shape& s = in->shape;
  int64_t shape[4], k_shape[4];
  if (q == nullptr || !element_type(*q, &s.dtype) || !view_of(*q, &in->q_view, shape)) return false;
  s.B = shape[0], s.T = shape[1], s.Hq = shape[2], s.D = shape[3];
  if (args[1] != Py_None) {
    const at::Tensor* k = in->k = cuda_tensor(args[1]);
    if (k == nullptr || k->get_device() != q->get_device() ||
        k->scalar_type() != q->scalar_type() || k->dim() != q->dim() ||
        !view_of(*k, &in->k_view, k_shape) || k_shape[0] != s.B || k_shape[1] != s.T ||
        k_shape[3] != s.D)
      return false;
    s.Hk = k_shape[2];
  } else if (args[3] != Py_None) {
    return false;
  }
  s.gamma_dtype = kF32;
  in->gamma_type = at::kFloat;
  if (PyObject* o = args[2] != Py_None ? args[2] : args[3]; o != Py_None) {
    const at::Tensor* g = cuda_tensor(o);
    if (g == nullptr || !element_type(*g, &s.gamma_dtype)) return false;
    in->gamma_type = g->scalar_type();
  }
  for (int i = 0; i < 2; ++i)
    if (!vector_of(args[2 + i], *q, in->gamma_type, s.D, &in->gamma[i])) return false;
  if (args[4] != Py_None) {
    const at::Tensor* f = cuda_tensor(args[4]);
    if (f == nullptr || !vector_of(args[4], *q, at::kFloat, f->numel(), &in->inv_freq)) return false;
    s.rot = 2 * f->numel();
  }
  if (args[5] != Py_None) {
    const at::Tensor* p = cuda_tensor(args[5]);
    if (p == nullptr || p->get_device() != q->get_device() || p->scalar_type() != at::kLong)
      return false;
    const int64_t n = p->dim();
    if ((n != 1 && n != 2) || p->size(n - 1) != s.T || (n == 2 && p->size(0) != s.B) ||
        (s.T > 1 && p->stride(n - 1) != 1))
      return false;
    if (n == 2 && s.B > 1) in->positions_batch = p->stride(0);
    in->positions = static_cast<const int64_t*>(p->data_ptr());
  }
  s.eps = static_cast<float>(PyFloat_AsDouble(args[6]));
  s.interleaved = PyObject_IsTrue(args[7]);
  return !PyErr_Occurred();
}
// Rows of the shape, type and device of an input.
const at::Tensor* rows_like(PyObject* o, const at::Tensor& like, flce_qk_view* v) {
  const at::Tensor* t = cuda_tensor(o);
  int64_t shape[4];
  return t != nullptr && t->get_device() == like.get_device() &&
                 t->scalar_type() == like.scalar_type() && t->sizes().equals(like.sizes()) &&
                 view_of(*t, v, shape)
             ? t
             : nullptr;
}
// A result: the caller's tensor, checked, or a new dense one once all checks have passed.
struct Result {
  PyObject* given = nullptr;
  const at::Tensor* like = nullptr;    // nullptr: there is no such result
  at::Tensor t;
  // Rows like an input.
  bool rows(PyObject* o, const at::Tensor* input, flce_qk_view* v) {
    like = input;
    if (o == Py_None) return true;
    given = o;
    return input != nullptr && rows_like(o, *input, v) != nullptr;
  }
  // fp32 [D], when there is a gamma.
  bool vector(PyObject* o, PyObject* gamma, const QkInputs& in) {
    if (gamma != Py_None) like = in.q;
    if (o == Py_None) return true;
    given = o;
    void* unused;
    return gamma != Py_None && vector_of(o, *in.q, at::kFloat, in.shape.D, &unused);
  }
  void make() {
    if (given != nullptr) t = THPVariable_Unpack(given);
  }
  // The call has been made, and has not refused.
  void written() const {
    if (given != nullptr) changes(t);
  }
  void make_rows(flce_qk_view* v) {
    make();
    if (given != nullptr || like == nullptr) return;
    t = dense(*like, like->sizes(), like->scalar_type());
    int64_t shape[4];
    view_of(t, v, shape);
  }
  void make_vector(int64_t n) {
    make();
    if (given == nullptr && like != nullptr)
      t = dense(*like, {n}, at::kFloat);
  }
  float* floats() const { return t.defined() ? static_cast<float*>(t.data_ptr()) : nullptr; }
  PyObject* object() const {
    if (given != nullptr) return Py_NewRef(given);
    return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
  }
};
// What is not right: an exception of Python's own, else None.
PyObject* not_right() {
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

// qk_forward(the inputs, q_out, k_out) -> (status, q_out, k_out), or None
PyObject* qk_forward(PyObject* const* args, Py_ssize_t count) {
  if (count != 10) {
    PyErr_SetString(PyExc_TypeError, "qk_forward takes 10 arguments");
    return nullptr;
  }
  QkInputs in{};
  Result q, k;
  flce_qk_view qv{}, kv{};
  if (!qk_inputs(args, &in) || !q.rows(args[8], in.q, &qv) || !k.rows(args[9], in.k, &kv))
    return not_right();
  q.make_rows(&qv);
  k.make_rows(&kv);
  const int rc = on_device(in.q->get_device(), [&](void* stream) {
    return library.forward(&in.shape, &in.q_view, in.keys(in.k_view), in.gamma[0], in.gamma[1],
                           static_cast<const float*>(in.inv_freq), in.positions,
                           in.positions_batch, &qv, in.keys(kv), stream);
  });
  if (rc == FLCE_OK) q.written(), k.written();
  return Py_BuildValue("iNN", rc, q.object(), k.object());
}

// qk_backward(the inputs, dq_out, dk_out, dq, dk, dgamma_q, dgamma_k, accumulate) ->
// (status, dq, dk, dgamma_q, dgamma_k), or None
PyObject* qk_backward(PyObject* const* args, Py_ssize_t count) {
  if (count != 15) {
    PyErr_SetString(PyExc_TypeError, "qk_backward takes 15 arguments");
    return nullptr;
  }
  QkInputs in{};
  Result q, k, gamma_q, gamma_k;
  flce_qk_view q_grad{}, k_grad{}, qv{}, kv{};
  const int accumulate = PyObject_IsTrue(args[14]);
  if (accumulate < 0 || !qk_inputs(args, &in) || rows_like(args[8], *in.q, &q_grad) == nullptr ||
      (in.k != nullptr ? rows_like(args[9], *in.k, &k_grad) == nullptr : args[9] != Py_None) ||
      !q.rows(args[10], in.q, &qv) || !k.rows(args[11], in.k, &kv) ||
      !gamma_q.vector(args[12], args[2], in) || !gamma_k.vector(args[13], args[3], in) ||
      (accumulate && ((gamma_q.like != nullptr && gamma_q.given == nullptr) ||
                      (gamma_k.like != nullptr && gamma_k.given == nullptr))))
    return not_right();
  q.make_rows(&qv);
  k.make_rows(&kv);
  gamma_q.make_vector(in.shape.D);
  gamma_k.make_vector(in.shape.D);
  const size_t bytes = library.qk_workspace(&in.shape);
  const at::Tensor ws = bytes_on(*in.q, bytes < 256 ? 256 : bytes);
  void* workspace = ws.data_ptr();
  float *to_q = gamma_q.floats(), *to_k = gamma_k.floats();
  const int rc = on_device(in.q->get_device(), [&](void* stream) {
    return library.backward(&in.shape, &q_grad, in.keys(k_grad), &in.q_view, in.keys(in.k_view),
                            in.gamma[0], in.gamma[1], static_cast<const float*>(in.inv_freq),
                            in.positions, in.positions_batch, &qv, in.keys(kv), to_q, to_k,
                            accumulate, workspace, bytes, stream);
  });
  if (rc == FLCE_OK) q.written(), k.written(), gamma_q.written(), gamma_k.written();
  return Py_BuildValue("iNNNN", rc, q.object(), k.object(), gamma_q.object(), gamma_k.object());
}

// torch reports errors by C++ exceptions; none may pass into the interpreter.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t count) {
  try {
    return F(args, count);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name, const char* doc) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(guarded<F>)),
          METH_FASTCALL, doc};
}

PyMethodDef methods[] = {
    method<bind>("bind", "the library's entry points"),
    method<gradients>("gradients", "(addresses, types, parameters' places) of gradients"),
    method<stepped>("stepped", "the parameters with a gradient have been changed"),
    method<grad_norm>("grad_norm", "(status, norm, factor) of a list of gradients, or None"),
    method<qk_forward>("qk_forward", "(status, q, k), or None"),
    method<qk_backward>("qk_backward", "(status, dq, dk, dgamma_q, dgamma_k), or None"),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal",
                      "From tensors to the library's calls", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
  PyObject* m = PyModule_Create(&module);
  // the torch and the Python that it was built for: the build looks whether they are still there
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", FLCE_MARSHAL_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
