// Native part of the Python binding: argument checks, allocation of outputs and the
// call, for the calls of speculative decoding and of the state cache.
//
// These run once per layer and round, and for a small batch their time is what the host
// spends before the launch: checking eight tensors through Python attributes and ctypes
// took 6 to 13 us of a call whose kernel takes 3 to 8; reading the tensors' own fields
// takes about one.  Every function returns (status, outputs ...); kda.py raises on a
// status that is not KDA_OK.  Checks of values, alignment and overlap are the C ABI's.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "kda.h"

namespace {

using at::ScalarType;
using at::Tensor;
using Shape = c10::SmallVector<int64_t, 4>;

struct Refused {};   // a Python error is set

[[noreturn]] void refuse(PyObject *type, const std::string &what) {
  PyErr_SetString(type, what.c_str());
  throw Refused{};
}

const Tensor &tensor(const char *name, PyObject *o) {
  if (!THPVariable_Check(o))
    refuse(PyExc_TypeError, std::string(name) + " must be a tensor, got " + Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

// A tensor with this many dimensions: the one whose sizes the others have to match.
const Tensor &first(const char *name, PyObject *o, int64_t dims) {
  const Tensor &t = tensor(name, o);
  if (t.dim() != dims)
    refuse(PyExc_ValueError,
           std::string(name) + " must have " + std::to_string(dims) + " dimensions, got " + std::to_string(t.dim()));
  return t;
}

std::string text(c10::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

// A dense CUDA tensor of this shape and type on this device.
const Tensor &want(const char *name, PyObject *o, c10::IntArrayRef shape, ScalarType dtype, c10::Device device) {
  const Tensor &t = tensor(name, o);
  if (t.scalar_type() != dtype)
    refuse(PyExc_TypeError, std::string(name) + " must be " + c10::toString(dtype) + ", got " +
                                c10::toString(t.scalar_type()));
  if (t.sizes() != shape)
    refuse(PyExc_ValueError, std::string(name) + " must have shape " + text(shape) + ", got " + text(t.sizes()));
  if (!t.is_cuda() || t.device() != device)
    refuse(PyExc_ValueError, std::string(name) + " must be on one CUDA device with the other arguments, got " +
                                 t.device().str());
  if (t.layout() != c10::kStrided || !t.is_contiguous())
    refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
  return t;
}

Tensor want_or_new(const char *name, PyObject *o, c10::IntArrayRef shape, ScalarType dtype, c10::Device device) {
  if (o == Py_None) return at::empty(shape, at::TensorOptions().dtype(dtype).device(device));
  return want(name, o, shape, dtype, device);
}

template <typename T> T *address(const Tensor &t) { return static_cast<T *>(t.data_ptr()); }

int float_code(const char *name, const Tensor &t) {
  if (t.scalar_type() == at::kBFloat16) return KDA_DTYPE_BF16;
  if (t.scalar_type() == at::kFloat) return KDA_DTYPE_F32;
  refuse(PyExc_TypeError, std::string(name) + " must be float32 or bfloat16, got " + c10::toString(t.scalar_type()));
}

int32_t to_int32(const char *name, int64_t x) {
  if (x > INT32_MAX) refuse(PyExc_ValueError, std::string(name) + " is too large: " + std::to_string(x));
  return (int32_t)x;
}

kda_shape make_shape(int64_t n, int64_t tokens, int64_t h, int64_t dk, int64_t dv, int dtype) {
  kda_shape s = {};
  s.num_seqs = to_int32("the number of sequences", n);
  s.total_tokens = tokens;
  s.num_heads = to_int32("the number of heads", h);
  s.head_dim_k = to_int32("the key size", dk);
  s.head_dim_v = to_int32("the value size", dv);
  s.qkv_dtype = dtype;
  return s;
}

// The arguments' device made current, and the stream: an address, or None for that
// device's current one.  A stream that is given is current while outputs are made, so
// that their memory is that stream's and is not handed on while it is still written.
struct Where {
  c10::cuda::CUDAGuard guard;
  c10::cuda::OptionalCUDAStreamGuard on;
  kda_stream_t stream;
  Where(c10::Device device, PyObject *s) : guard(device) {
    if (s == Py_None) {
      stream = reinterpret_cast<kda_stream_t>(c10::cuda::getCurrentCUDAStream(device.index()).stream());
      return;
    }
    stream = static_cast<kda_stream_t>(PyLong_AsVoidPtr(s));
    if (PyErr_Occurred()) throw Refused{};
    on.reset_stream(stream ? c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(stream), device.index())
                           : c10::cuda::getDefaultCUDAStream(device.index()));
  }
};

template <typename F> int call(F f) {
  int st;
  Py_BEGIN_ALLOW_THREADS st = f();
  Py_END_ALLOW_THREADS return st;
}

PyObject *wrap(const Tensor &t, PyObject *given) {
  if (given != Py_None) {
    Py_INCREF(given);
    return given;
  }
  return THPVariable_Wrap(t);
}

void arguments(Py_ssize_t n, Py_ssize_t wanted) {
  if (n != wanted)
    refuse(PyExc_TypeError, "expected " + std::to_string(wanted) + " arguments, got " + std::to_string(n));
}

struct Tree {
  int64_t N, T, H, Dk, Dv;
  ScalarType dtype;
  c10::Device device;
  const Tensor &k, &v, &g, &beta, &state;
  const int32_t *parents;
};

Tree tree(PyObject *ok, PyObject *ov, PyObject *og, PyObject *ob, PyObject *os, PyObject *op) {
  const Tensor &k = first("k", ok, 4), &v = first("v", ov, 4);
  const int64_t N = k.size(0), T = k.size(1), H = k.size(2), Dk = k.size(3), Dv = v.size(3);
  const ScalarType dt = k.scalar_type();
  const c10::Device dev = k.device();
  float_code("q/k/v", k);
  want("k", ok, {N, T, H, Dk}, dt, dev);
  want("v", ov, {N, T, H, Dv}, dt, dev);
  const Tensor &g = want("g", og, {N, T, H, Dk}, at::kFloat, dev);
  const Tensor &b = want("beta", ob, {N, T, H}, at::kFloat, dev);
  const Tensor &s = want("state", os, {N, H, Dk, Dv}, at::kFloat, dev);
  const int32_t *p = op == Py_None ? nullptr : address<int32_t>(want("parents", op, {N, T}, at::kInt, dev));
  return {N, T, H, Dk, Dv, dt, dev, k, v, g, b, s, p};
}

// (q, k, v, g, beta, state, parents, out, stream, dev_status) -> (status, out)
PyObject *decode_tree(PyObject *const *a, Py_ssize_t n) {
  arguments(n, 10);
  const Tree t = tree(a[1], a[2], a[3], a[4], a[5], a[6]);
  const Tensor &q = want("q", a[0], t.k.sizes(), t.dtype, t.device);
  const Where at(t.device, a[8]);
  const Tensor out = want_or_new("out", a[7], t.v.sizes(), t.dtype, t.device);
  kda_shape s = make_shape(t.N, t.N * t.T, t.H, t.Dk, t.Dv, float_code("q/k/v", t.k));
  if (a[9] != Py_None) s.dev_status = address<int32_t>(want("dev_status", a[9], {1}, at::kInt, t.device));
  const int32_t nodes = to_int32("the number of places", t.T);
  const int st = call([&] {
    return kda_decode_tree(q.data_ptr(), t.k.data_ptr(), t.v.data_ptr(), address<float>(t.g),
                           address<float>(t.beta), address<float>(t.state), t.parents, out.data_ptr(), nodes, &s,
                           at.stream);
  });
  return Py_BuildValue("(iN)", st, wrap(out, a[7]));
}

// (k, v, g, beta, state, accept_node, parents, state_out, stream) -> status
PyObject *tree_commit(PyObject *const *a, Py_ssize_t n) {
  arguments(n, 9);
  const Tree t = tree(a[0], a[1], a[2], a[3], a[4], a[6]);
  const Tensor &node = want("accept_node", a[5], {t.N}, at::kInt, t.device);
  const Tensor &out = want("state_out", a[7], t.state.sizes(), at::kFloat, t.device);
  const Where at(t.device, a[8]);
  const kda_shape s = make_shape(t.N, t.N * t.T, t.H, t.Dk, t.Dv, float_code("q/k/v", t.k));
  const int32_t nodes = to_int32("the number of places", t.T);
  return PyLong_FromLong(call([&] {
    return kda_tree_commit(t.k.data_ptr(), t.v.data_ptr(), address<float>(t.g), address<float>(t.beta),
                           address<float>(t.state), address<float>(out), t.parents, address<int32_t>(node), nodes,
                           &s, at.stream);
  }));
}

// (target, draft, tokens, parents, uniforms, accept_node, accept_len, out_tokens, stream)
// -> (status, accept_node, accept_len, out_tokens)
PyObject *verify_tree(PyObject *const *a, Py_ssize_t n) {
  arguments(n, 9);
  const Tensor &target = first("target_probs", a[0], 3);
  const int64_t N = target.size(0), T1 = target.size(1), T = T1 - 1, V = target.size(2);
  const ScalarType dt = target.scalar_type();
  const c10::Device dev = target.device();
  const int code = float_code("target_probs", target);
  if (T < 1) refuse(PyExc_ValueError, "target_probs must have a row for the prefix and one for every place");
  want("target_probs", a[0], {N, T1, V}, dt, dev);
  const void *draft = a[1] == Py_None ? nullptr : want("draft_probs", a[1], {N, T, V}, dt, dev).data_ptr();
  const Tensor &tokens = want("tokens", a[2], {N, T}, at::kInt, dev);
  const int32_t *parents = a[3] == Py_None ? nullptr : address<int32_t>(want("parents", a[3], {N, T}, at::kInt, dev));
  const Tensor &uniforms = want("uniforms", a[4], {N, T1}, at::kFloat, dev);
  const Where at(dev, a[8]);
  const Tensor node = want_or_new("accept_node", a[5], {N}, at::kInt, dev);
  const Tensor len = want_or_new("accept_len", a[6], {N}, at::kInt, dev);
  const Tensor out = want_or_new("out_tokens", a[7], {N, T1}, at::kInt, dev);
  const int32_t seqs = to_int32("the number of sequences", N), nodes = to_int32("the number of places", T);
  const int st = call([&] {
    return kda_verify_tree(target.data_ptr(), draft, address<int32_t>(tokens), parents, address<float>(uniforms),
                           address<int32_t>(node), address<int32_t>(len), address<int32_t>(out), seqs, nodes, V,
                           code, at.stream);
  });
  return Py_BuildValue("(iNNN)", st, wrap(node, a[5]), wrap(len, a[6]), wrap(out, a[7]));
}

struct Cache {
  int64_t slots, n, H, Dk, Dv;
  int code;
  c10::Device device;
};

Cache cache(PyObject *oc, PyObject *osc, PyObject *osl) {
  const Tensor &c = first("cache", oc, 4), &slots = first("slots", osl, 1);
  const int64_t S = c.size(0), n = slots.size(0), H = c.size(1), Dk = c.size(2), Dv = c.size(3);
  const ScalarType dt = c.scalar_type();
  if (dt != at::kFloat8_e4m3fn && dt != at::kChar)
    refuse(PyExc_TypeError, std::string("cache must be float8_e4m3fn or int8, got ") + c10::toString(dt));
  const c10::Device dev = c.device();
  want("cache", oc, {S, H, Dk, Dv}, dt, dev);
  want("scales", osc, {S, H, Dk}, at::kFloat, dev);
  want("slots", osl, {n}, at::kInt, dev);
  return {S, n, H, Dk, Dv, dt == at::kChar ? KDA_CACHE_INT8 : KDA_CACHE_E4M3, dev};
}

// (states, slots, cache, scales, stream) -> status
PyObject *state_store(PyObject *const *a, Py_ssize_t n) {
  arguments(n, 5);
  const Cache c = cache(a[2], a[3], a[1]);
  const Tensor &states = want("states", a[0], {c.n, c.H, c.Dk, c.Dv}, at::kFloat, c.device);
  const Where at(c.device, a[4]);
  const kda_shape s = make_shape(c.n, c.n, c.H, c.Dk, c.Dv, KDA_DTYPE_F32);
  const Tensor &slots = tensor("slots", a[1]), &codes = tensor("cache", a[2]), &scales = tensor("scales", a[3]);
  return PyLong_FromLong(call([&] {
    return kda_state_store(address<float>(states), address<int32_t>(slots), codes.data_ptr(),
                           address<float>(scales), c.slots, c.code, &s, at.stream);
  }));
}

// (cache, scales, slots, states, stream) -> (status, states)
PyObject *state_load(PyObject *const *a, Py_ssize_t n) {
  arguments(n, 5);
  const Cache c = cache(a[0], a[1], a[2]);
  const Where at(c.device, a[4]);
  const Tensor states = want_or_new("states", a[3], {c.n, c.H, c.Dk, c.Dv}, at::kFloat, c.device);
  const kda_shape s = make_shape(c.n, c.n, c.H, c.Dk, c.Dv, KDA_DTYPE_F32);
  const Tensor &codes = tensor("cache", a[0]), &scales = tensor("scales", a[1]), &slots = tensor("slots", a[2]);
  const int st = call([&] {
    return kda_state_load(codes.data_ptr(), address<float>(scales), address<int32_t>(slots),
                          address<float>(states), c.slots, c.code, &s, at.stream);
  });
  return Py_BuildValue("(iN)", st, wrap(states, a[3]));
}

// No C++ exception leaves a function.
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t n) {
  try {
    return F(a, n);
  } catch (const Refused &) {
  } catch (...) {          // as PyTorch's own functions raise it (memory that is not there, ...)
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

#define KDA_ENTRY(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KDA_ENTRY(decode_tree), KDA_ENTRY(tree_commit), KDA_ENTRY(verify_tree),
                         KDA_ENTRY(state_store), KDA_ENTRY(state_load), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject *m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", KDA_TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
