// Python marshalling of the operators of an attention layer (binding.py): checks tensors, allocates outputs and calls the
// C-ABI entry points with device pointers and the current CUDA stream.  A step of such a layer for a few tokens takes
// some five microseconds on the device, half of what the same checks and allocations take in Python.
//
// The entry points' addresses and the exception to raise are handed over by bind(), so that this module depends on
// torch alone.  Every function takes positional arguments; None stands for what is not given.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/SmallVector.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <cmath>
#include <sstream>
#include <string>

#include "../../include/kda.h"

namespace {

struct {
  decltype(&kda_block_tables) block_tables = nullptr;
  decltype(&kda_rope_append) rope_append = nullptr;
  decltype(&kda_window_attention_fwd) fwd = nullptr;
  decltype(&kda_window_attention_decode_step) step = nullptr;
  decltype(&kda_tree_attention) tree = nullptr;
  PyObject* error = nullptr;  // KdaError
} g;

struct PyError {};  // a Python exception has been set

[[noreturn]] void refuse(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw PyError();
}

std::string text(at::IntArrayRef shape) {
  std::ostringstream s;
  s << "(";
  for (size_t i = 0; i < shape.size(); ++i) s << (i ? ", " : "") << shape[i];
  s << (shape.size() == 1 ? ",)" : ")");
  return s.str();
}

const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyError();
  return v;
}
// an int argument of the C interface
int small(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v != (int)v) refuse(PyExc_ValueError, std::string(name) + " does not fit 32 bits");
  return (int)v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyError();
  return v;
}

void on_device(const at::Tensor& t, const char* name, int index) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
  if (t.get_device() != index)
    refuse(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", expected cuda:" + std::to_string(index));
}
void typed(const at::Tensor& t, const char* name, at::ScalarType dtype) {
  if (t.scalar_type() != dtype)
    refuse(PyExc_TypeError, std::string(name) + " must be " + c10::toString(dtype) + ", got " + c10::toString(t.scalar_type()));
}
void shaped(const at::Tensor& t, const char* name, at::IntArrayRef shape) {
  if (t.sizes() != shape) refuse(PyExc_ValueError, std::string(name) + " has shape " + text(t.sizes()) + ", expected " + text(shape));
}
// The index of the tensor's device, which has to be the current one.
int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
  const int index = t.get_device(), current = c10::cuda::current_device();
  if (index != current)
    refuse(PyExc_ValueError, std::string(name) + " is on cuda:" + std::to_string(index) + ", the current device is cuda:" +
                                 std::to_string(current));
  return index;
}
// Lets other Python threads run while it lives: allocations and launches may wait for the device, and what the device waits
// for may need the interpreter.  (The caller's frame keeps the arguments' tensors.)
struct Released {
  PyThreadState* const state = PyEval_SaveThread();
  Released() = default;
  Released(const Released&) = delete;
  ~Released() { PyEval_RestoreThread(state); }
};
// The address of a dense tensor of that type, shape and device.
template <class T>
T* data(const at::Tensor* t, const char* name, at::ScalarType dtype, at::IntArrayRef shape, int index) {
  if (t == nullptr) return nullptr;
  on_device(*t, name, index);
  if (!t->is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
  typed(*t, name, dtype);
  shaped(*t, name, shape);
  return static_cast<T*>(t->data_ptr());
}
// Outputs: dense tensors of that type, shape and device that are given, or new ones.
struct Wanted {
  PyObject* given;
  const char* name;
  c10::SmallVector<int64_t, 3> shape;
};
template <size_t N>
std::array<at::Tensor, N> outputs(const Wanted (&wanted)[N], at::ScalarType dtype, int index) {
  std::array<at::Tensor, N> r;
  bool all = true;
  for (size_t i = 0; i < N; ++i) {
    const at::Tensor* t = tensor(wanted[i].given, wanted[i].name, true);
    data<void>(t, wanted[i].name, dtype, wanted[i].shape, index);
    if (t) r[i] = *t; else all = false;
  }
  if (all) return r;
  const Released other_threads;
  const auto options = at::TensorOptions().dtype(dtype).device(at::kCUDA, (c10::DeviceIndex)index);
  for (size_t i = 0; i < N; ++i)
    if (!r[i].defined()) r[i] = at::empty(wanted[i].shape, options);
  return r;
}
// [tokens, heads, d] whose heads are dense and whose tokens may lie further apart: the distance of two tokens.
int64_t token_rows(const at::Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape, int index) {
  on_device(t, name, index);
  typed(t, name, dtype);
  shaped(t, name, shape);
  if (t.stride(2) != 1 || (shape[1] > 1 && t.stride(1) != shape[2]))
    refuse(PyExc_ValueError, std::string(name) + ": the heads of a token must be contiguous");
  return shape[0] > 1 ? t.stride(0) : shape[1] * shape[2];
}
void rank(const at::Tensor& t, const char* name, int64_t n) {
  if (t.dim() != n) refuse(PyExc_ValueError, std::string(name) + " must have " + std::to_string(n) + " dimensions");
}
int narrow(int64_t n, const char* name) {
  if (n > 0x7fffffff) refuse(PyExc_ValueError, std::string(name) + " has too many elements in a dimension");
  return (int)n;
}

// The two caches [num_blocks, block_size, Hkv, d], which have to be alike.
struct Caches {
  int blocks, size, heads, d;
  int64_t strides[3];
  Caches(const at::Tensor& k, const at::Tensor& v, int index) {
    if (k.dim() != 4 || v.sizes() != k.sizes())
      refuse(PyExc_ValueError, "k_cache and v_cache must both be [num_blocks, block_size, Hkv, d]");
    typed(k, "k_cache", at::kBFloat16);
    typed(v, "v_cache", at::kBFloat16);
    on_device(k, "k_cache", index);
    on_device(v, "v_cache", index);
    if (k.stride(3) != 1 || v.strides() != k.strides())
      refuse(PyExc_ValueError, "k_cache and v_cache must have the same strides, and dense heads");
    blocks = narrow(k.size(0), "k_cache"); size = narrow(k.size(1), "k_cache"); heads = narrow(k.size(2), "k_cache");
    d = narrow(k.size(3), "k_cache");
    for (int i = 0; i < 3; ++i) strides[i] = k.size(i) != 1 ? k.stride(i) : d;  // (of a dimension of one it says nothing)
  }
};

void* stream_of(int index) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream(); }

// Calls an entry point, whose arguments have been formed, and raises what it answers.
template <class F, class... A>
void call(const char* fn, F entry, A... args) {
  int status;
  {
    const Released other_threads;
    status = entry(args...);
  }
  if (status == 0) return;
  if (PyObject* e = PyObject_CallFunction(g.error, "si", fn, status)) {
    PyErr_SetObject(g.error, e);
    Py_DECREF(e);
  }
  throw PyError();
}

void want(Py_ssize_t n, Py_ssize_t expected) {
  if (n != expected) refuse(PyExc_TypeError, "wrong number of arguments");
}

template <class F>
PyObject* guarded(F&& f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const PyError&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// bind({name: address}, exception)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want(n, 2);
    auto address = [&](const char* name) {
      PyObject* o = PyDict_GetItemString(a[0], name);
      if (!o) refuse(PyExc_KeyError, name);
      return reinterpret_cast<void*>(integer(o));
    };
    g.block_tables = reinterpret_cast<decltype(g.block_tables)>(address("kda_block_tables"));
    g.rope_append = reinterpret_cast<decltype(g.rope_append)>(address("kda_rope_append"));
    g.fwd = reinterpret_cast<decltype(g.fwd)>(address("kda_window_attention_fwd"));
    g.step = reinterpret_cast<decltype(g.step)>(address("kda_window_attention_decode_step"));
    g.tree = reinterpret_cast<decltype(g.tree)>(address("kda_tree_attention"));
    Py_INCREF(a[1]);
    Py_XDECREF(g.error);
    g.error = a[1];
    Py_RETURN_NONE;
  });
}

// counts, lengths, block_tables, free_ring, free_state, block_size, max_tokens, new_lengths, new_free_state, slot_map,
// positions, cu_seqlens
PyObject* block_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want(n, 12);
    const at::Tensor &counts = *tensor(a[0], "counts"), &lengths = *tensor(a[1], "lengths"), &table = *tensor(a[2], "block_tables"),
                     &ring = *tensor(a[3], "free_ring"), &state = *tensor(a[4], "free_state");
    const int dev = device_of(table, "block_tables");
    rank(table, "block_tables", 2);
    rank(ring, "free_ring", 1);
    const int64_t N = table.size(0), width = table.size(1), blocks = ring.size(0), T = integer(a[6]);
    if (T < 0) refuse(PyExc_ValueError, "max_tokens must not be negative");
    const at::ScalarType i32 = at::kInt;
    const int32_t* pc = data<int32_t>(&counts, "counts", i32, {N}, dev);
    const int32_t* pl = data<int32_t>(&lengths, "lengths", i32, {N}, dev);
    int32_t* pt = data<int32_t>(&table, "block_tables", i32, {N, width}, dev);
    int32_t* pr = data<int32_t>(&ring, "free_ring", i32, {blocks}, dev);
    const int32_t* ps = data<int32_t>(&state, "free_state", i32, {2}, dev);
    const auto [now, left, slot, pos, cu] = outputs({{a[7], "new_lengths", {N}}, {a[8], "new_free_state", {2}}, {a[9], "slot_map", {T}},
                                                     {a[10], "positions", {T}}, {a[11], "cu_seqlens", {N + 1}}}, i32, dev);
    call("kda_block_tables", g.block_tables, pc, pl, pt, pr, ps, now.data_ptr<int32_t>(), left.data_ptr<int32_t>(),
         slot.data_ptr<int32_t>(), pos.data_ptr<int32_t>(), cu.data_ptr<int32_t>(), narrow(N, "block_tables"),
         narrow(width, "block_tables"), narrow(blocks, "free_ring"), small(a[5], "block_size"), T, stream_of(dev));
    PyObject* r = PyTuple_New(5);
    if (!r) return nullptr;
    const at::Tensor* all[5] = {&slot, &pos, &cu, &now, &left};
    for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(*all[i]));
    return r;
  });
}

// q, k, v, inv_freq, positions, slot_map, k_cache, v_cache, axis, interleaved, q_out
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want(n, 11);
    const at::Tensor &q = *tensor(a[0], "q"), &k = *tensor(a[1], "k"), &v = *tensor(a[2], "v"), &freq = *tensor(a[3], "inv_freq"),
                     &pos = *tensor(a[4], "positions"), &slot = *tensor(a[5], "slot_map"), &kc = *tensor(a[6], "k_cache"),
                     &vc = *tensor(a[7], "v_cache");
    const at::Tensor* axis = tensor(a[8], "axis", true);
    const at::ScalarType dt = q.scalar_type();
    if (dt != at::kBFloat16 && dt != at::kFloat)
      refuse(PyExc_TypeError, std::string("unsupported dtype ") + c10::toString(dt) + " (bf16 or fp32)");
    const int dev = device_of(q, "q");
    rank(q, "q", 3);
    const int64_t T = q.size(0), H = q.size(1), d = q.size(2), pairs = freq.numel();
    const Caches c(kc, vc, dev);
    if (c.d != d) refuse(PyExc_ValueError, "the cache's heads have " + std::to_string(c.d) + " values, q's " + std::to_string(d));
    const int64_t qs = token_rows(q, "q", dt, {T, H, d}, dev), ks = token_rows(k, "k", dt, {T, c.heads, d}, dev),
                  vs = token_rows(v, "v", dt, {T, c.heads, d}, dev);
    const double* pf = data<double>(&freq, "inv_freq", at::kDouble, {pairs}, dev);
    const int32_t* pa = data<int32_t>(axis, "axis", at::kInt, {pairs}, dev);
    const int64_t axes = pos.dim() == 2 ? pos.size(0) : 1;
    const int32_t* pp = pos.dim() == 2 ? data<int32_t>(&pos, "positions", at::kInt, {axes, T}, dev)
                                       : data<int32_t>(&pos, "positions", at::kInt, {T}, dev);
    const int32_t* ps = data<int32_t>(&slot, "slot_map", at::kInt, {T}, dev);
    const int turned = PyObject_IsTrue(a[9]);
    if (turned < 0) throw PyError();
    const auto [out] = outputs({{a[10], "q_out", {T, H, d}}}, at::kBFloat16, dev);
    call("kda_rope_append", g.rope_append, q.data_ptr(), k.data_ptr(), v.data_ptr(), pf, pa, pp, ps, out.data_ptr(), kc.data_ptr(),
         vc.data_ptr(), T, narrow(H, "q"), c.heads, c.d, narrow(2 * pairs, "inv_freq"), narrow(axes, "positions"), turned, qs, ks,
         vs, c.blocks, c.size, c.strides, dt == at::kBFloat16 ? KDA_DTYPE_BF16 : KDA_DTYPE_FP32, stream_of(dev));
    return THPVariable_Wrap(out);
  });
}

// What the three attentions have in common: q, k_cache, v_cache, block_tables, lengths, .. out, window, sinks, scale, max_length
struct Attention {
  const at::Tensor &q, &kc, &vc, &table, &lengths;
  int dev;
  int64_t T, H, N, width, q_stride;
  Caches c;
  const int32_t *tables, *len;
  at::Tensor out;
  int window, sinks;
  int64_t most;
  float scale;
  Attention(PyObject* const* a, PyObject* const* rest)
      : q(*tensor(a[0], "q")), kc(*tensor(a[1], "k_cache")), vc(*tensor(a[2], "v_cache")), table(*tensor(a[3], "block_tables")),
        lengths(*tensor(a[4], "lengths")), dev(device_of(q, "q")), c(kc, vc, dev) {
    rank(q, "q", 3);
    rank(table, "block_tables", 2);
    T = q.size(0); H = q.size(1); N = table.size(0); width = table.size(1);
    if (c.d != q.size(2))
      refuse(PyExc_ValueError, "the cache's heads have " + std::to_string(c.d) + " values, q's " + std::to_string(q.size(2)));
    q_stride = token_rows(q, "q", at::kBFloat16, {T, H, c.d}, dev);
    tables = data<int32_t>(&table, "block_tables", at::kInt, {N, width}, dev);
    len = data<int32_t>(&lengths, "lengths", at::kInt, {N}, dev);
    out = outputs({{rest[0], "out", {T, H, c.d}}}, at::kBFloat16, dev)[0];
    window = small(rest[1], "window"); sinks = small(rest[2], "sinks");
    scale = rest[3] == Py_None ? (float)(1.0 / std::sqrt((double)c.d)) : (float)number(rest[3]);
    most = integer(rest[4]);
    narrow(N, "block_tables"); narrow(width, "block_tables"); narrow(H, "q");
  }
};

// .., cu_seqlens, out, window, sinks, scale, max_length
PyObject* window_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want(n, 11);
    const Attention t(a, a + 6);
    const int32_t* cu = data<int32_t>(tensor(a[5], "cu_seqlens"), "cu_seqlens", at::kInt, {t.N + 1}, t.dev);
    call("kda_window_attention_fwd", g.fwd, t.q.data_ptr(), t.kc.data_ptr(), t.vc.data_ptr(), t.tables, t.len, cu, t.out.data_ptr(),
         (int)t.N, t.T, (int)t.H, t.c.heads, t.c.d, t.q_stride, t.c.blocks, t.c.size, (int)t.width, t.c.strides, t.window, t.sinks,
         t.most, t.scale, stream_of(t.dev));
    return THPVariable_Wrap(t.out);
  });
}

// .., out, window, sinks, scale, max_length
PyObject* window_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want(n, 10);
    const Attention t(a, a + 5);
    if (t.T != t.N)
      refuse(PyExc_ValueError, "q has " + std::to_string(t.T) + " tokens for " + std::to_string(t.N) + " requests");
    call("kda_window_attention_decode_step", g.step, t.q.data_ptr(), t.kc.data_ptr(), t.vc.data_ptr(), t.tables, t.len,
         t.out.data_ptr(), (int)t.N, (int)t.H, t.c.heads, t.c.d, t.q_stride, t.c.blocks, t.c.size, (int)t.width, t.c.strides,
         t.window, t.sinks, t.most, t.scale, stream_of(t.dev));
    return THPVariable_Wrap(t.out);
  });
}

// .., cu_seqlens, tree_mask, out, window, sinks, scale, max_length
PyObject* tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want(n, 12);
    const Attention t(a, a + 7);
    const int32_t* cu = data<int32_t>(tensor(a[5], "cu_seqlens"), "cu_seqlens", at::kInt, {t.N + 1}, t.dev);
    const at::Tensor& mask = *tensor(a[6], "tree_mask");
    rank(mask, "tree_mask", 2);
    const int64_t words = mask.size(1);
    const uint64_t* pm = data<uint64_t>(&mask, "tree_mask", at::kLong, {t.T, words}, t.dev);
    call("kda_tree_attention", g.tree, t.q.data_ptr(), t.kc.data_ptr(), t.vc.data_ptr(), t.tables, t.len, cu, pm,
         narrow(words, "tree_mask"), t.out.data_ptr(), (int)t.N, t.T, (int)t.H, t.c.heads, t.c.d, t.q_stride, t.c.blocks, t.c.size,
         (int)t.width, t.c.strides, t.window, t.sinks, t.most, t.scale, stream_of(t.dev));
    return THPVariable_Wrap(t.out);
  });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"bind", FAST(bind)},
                         {"block_tables", FAST(block_tables)},
                         {"rope_append", FAST(rope_append)},
                         {"window_fwd", FAST(window_fwd)},
                         {"window_step", FAST(window_step)},
                         {"tree", FAST(tree)},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kda_marshal() { return PyModule_Create(&module); }
