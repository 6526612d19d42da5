// attn_torch.cpp -- the attention-side operators' calls from Python: checks of
// torch tensors, output allocation on the current stream, and the C entry
// points of svdq_attn.h.
//
// A CPython extension module rather than ctypes calls: at single tokens a kernel
// takes 2 to 8 us, and the same checks and descriptions in Python took 7 to 9 us
// a call (norms 14 us a call, of which 4 are the launch; here 6).
// attention.py documents the arguments; everything here is positional, and a
// `stream` argument has been made current by then.
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>

#include <cmath>
#include <cstdarg>
#include <string>
#include <utility>

#include "head_overlap.h"
#include "svdq_attn.h"

namespace {

// Thrown once a Python exception is set.
struct PythonError {};

[[noreturn]] void raise(PyObject* type, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw PythonError();
}

std::string shape_text(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + (t.dim() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s: expected a tensor, got %s", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
// A tensor on the call's device; -1: this one says which.
const at::Tensor& on_device(PyObject* o, const char* name, int* device) {
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda()) raise(PyExc_ValueError, "%s: must be a CUDA tensor", name);
  const int d = t.get_device();
  if (*device < 0) *device = d;
  if (d != *device) raise(PyExc_ValueError, "%s: on cuda:%d, the other tensors on cuda:%d", name, d, *device);
  return t;
}
bool given(PyObject* o) { return o != Py_None; }

int type_code(const at::Tensor& t, const char* name) {
  const auto s = t.scalar_type();
  if (s == at::kBFloat16) return 0;
  if (s == at::kHalf) return 1;
  raise(PyExc_TypeError, "%s: must be bf16 or fp16, got %s", name, at::toString(s));
}
void need_type(const at::Tensor& t, const char* name, at::ScalarType type) {
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, "%s: expected %s, got %s", name, at::toString(type), at::toString(t.scalar_type()));
}

int count(int64_t n, const char* name) {
  if (n > 0x7FFFFFFF) raise(PyExc_ValueError, "%s: too large", name);
  return (int)n;
}

// A tensor of heads: (tokens, heads, head_dim), head_dim contiguous.
svdq_heads heads_of(const at::Tensor& t, const char* name) {
  if (t.dim() != 3)
    raise(PyExc_ValueError, "%s: expected (tokens, heads, head_dim), got shape %s", name, shape_text(t).c_str());
  if (t.numel() == 0) return {nullptr, 0, 0};
  if (t.size(2) > 1 && t.stride(2) != 1) raise(PyExc_ValueError, "%s: head_dim must be contiguous", name);
  const svdq_heads h = {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : 0, t.size(1) > 1 ? t.stride(1) : 0};
  if (((h.token_stride | h.head_stride) & 7) || (reinterpret_cast<uintptr_t>(h.data) & 15))
    raise(PyExc_ValueError,
          "%s: needs 16-byte alignment and token and head strides that are multiples of 8 elements", name);
  return h;
}
svdq_heads contiguous_heads(const at::Tensor& t) {
  if (t.numel() == 0) return {nullptr, 0, 0};
  return {t.data_ptr(), t.size(1) * t.size(2), t.size(2)};
}
void need_shape(const at::Tensor& t, const char* name, int64_t a, int64_t b, int64_t c) {
  if (t.dim() != 3 || t.size(0) != a || t.size(1) != b || t.size(2) != c)
    raise(PyExc_ValueError, "%s: expected shape (%lld, %lld, %lld), got %s", name, (long long)a, (long long)b,
          (long long)c, shape_text(t).c_str());
}
// Refuses an output whose elements share memory (expanded or overlapping views).
void distinct(const at::Tensor& t, const char* name) {
  if (t.numel() == 0) return;
  int order[3] = {0, 1, 2};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (t.stride(order[j]) < t.stride(order[i])) std::swap(order[i], order[j]);
  int64_t extent = 1;
  for (int i : order) {
    if (t.size(i) == 1) continue;
    if (t.stride(i) < extent) raise(PyExc_ValueError, "%s: its elements overlap in memory", name);
    extent += t.stride(i) * (t.size(i) - 1);
  }
}
// The memory of an argument: a tensor of heads, a block table (rows of contiguous numbers), or a contiguous tensor.
struct Memory {
  svdq::HeadRuns runs;
  long long end;                                // past its last byte; runs.at if it has none
  const char* name;
  at::Tensor tensor;
  Memory() = default;
  Memory(const at::Tensor& t, const char* n) : name(n), tensor(t) {
    const long long size = (long long)t.element_size(), at = (long long)reinterpret_cast<uintptr_t>(t.data_ptr());
    const auto size_of = t.sizes(), stride = t.strides();
    if (t.numel() == 0)
      runs = {at, 0, 0, 1, 1, 0};
    else if (size_of.size() == 3)
      runs = {at, stride[0] * size, stride[1] * size, size_of[0], size_of[1], size_of[2] * size};
    else if (size_of.size() == 2)
      runs = {at, stride[0] * size, 0, size_of[0], 1, size_of[1] * size};
    else
      runs = {at, 0, 0, 1, 1, (long long)t.numel() * size};
    end = svdq::end_of(runs);
  }
};
// Refuses an output that lies over another argument (views of one buffer side by side are fine).
void apart(const Memory& t, const Memory& other) {
  if (t.runs.at >= other.end || other.runs.at >= t.end || t.runs.bytes == 0 || other.runs.bytes == 0) return;
  if (!svdq::runs_overlap(t.runs, other.runs)) return;
  raise(PyExc_ValueError, "%s and %s overlap in memory", t.name, other.name);
}
// What torch's own in-place operations do: who saved the tensor for a backward pass learns that it changed.
void changed(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
bool tracked(const at::Tensor& t) { return t.requires_grad() && at::GradMode::is_enabled(); }
// An output that is given, or an input written over, cannot be part of a graph.
void not_tracked(const at::Tensor& t, const char* name) {
  if (tracked(t))
    raise(PyExc_RuntimeError, "%s: requires grad, and this operator has no backward pass (call it under torch.no_grad())", name);
}
// A new output of inputs that require grad is part of their graph; a backward pass through it raises.
void no_backward(at::Tensor& y, const char* name, const torch::autograd::variable_list& inputs) {
  if (!y.defined()) return;
  torch::autograd::set_history(
      y, std::shared_ptr<torch::autograd::Node>(
             new torch::autograd::NotImplemented(name, torch::autograd::collect_next_edges(inputs)),
             torch::autograd::deleteNode));
}

// A contiguous vector of n elements (n < 0: any number).
const at::Tensor& vector(PyObject* o, const char* name, at::ScalarType type, int64_t n, int* device) {
  const at::Tensor& t = on_device(o, name, device);
  need_type(t, name, type);
  if (t.dim() != 1 || (n >= 0 && t.size(0) != n))
    raise(PyExc_ValueError, "%s: expected shape (%lld,), got %s", name, (long long)n, shape_text(t).c_str());
  if (!t.is_contiguous()) raise(PyExc_ValueError, "%s: must be contiguous", name);
  return t;
}

// `memory`: that of the four, if wanted.
svdq_kv4_cache cache_of(PyObject* o, int* device, Memory* memory = nullptr) {
  static const char* names[4] = {"k_codes", "k_scales", "v_codes", "v_scales"};
  PyObject* seq = PySequence_Fast(o, "cache: expected (k_codes, k_scales, v_codes, v_scales)");
  if (!seq) throw PythonError();
  struct Release {
    PyObject* o;
    ~Release() { Py_DECREF(o); }
  } release{seq};
  if (PySequence_Fast_GET_SIZE(seq) != 4)
    raise(PyExc_ValueError, "cache: expected (k_codes, k_scales, v_codes, v_scales)");
  svdq_kv4_cache c = {};
  void* data[4];
  for (int i = 0; i < 4; ++i) {
    const at::Tensor& t = on_device(PySequence_Fast_GET_ITEM(seq, i), names[i], device);
    const bool scales = i & 1;
    if (t.scalar_type() != at::kByte && !(scales && t.scalar_type() == at::kFloat8_e4m3fn))
      raise(PyExc_TypeError, scales ? "%s: must be uint8 or float8_e4m3fn" : "%s: must be uint8", names[i]);
    if (i == 0) {
      if (t.dim() != 4)
        raise(PyExc_ValueError, "%s: expected (pages, heads, page_size, head_dim / 2), got %s", names[i],
              shape_text(t).c_str());
      c.pages = t.size(0);
      c.heads = count(t.size(1), names[i]);
      c.page_size = count(t.size(2), names[i]);
      c.head_dim = count(2 * t.size(3), names[i]);
    }
    if (t.dim() != 4 || t.size(0) != c.pages || t.size(1) != c.heads || t.size(2) != c.page_size ||
        t.size(3) != c.head_dim / (scales ? 16 : 2))
      raise(PyExc_ValueError, "%s: expected shape (%lld, %d, %d, %d), got %s", names[i], c.pages, c.heads, c.page_size,
            c.head_dim / (scales ? 16 : 2), shape_text(t).c_str());
    if (!t.is_contiguous()) raise(PyExc_ValueError, "%s: must be contiguous", names[i]);
    data[i] = t.data_ptr();
    if (memory) memory[i] = Memory(t, names[i]);
  }
  c.k_codes = data[0];
  c.k_scales = data[1];
  c.v_codes = data[2];
  c.v_scales = data[3];
  return c;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError();
  return v;
}
void* current_stream(int device) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }
at::Tensor empty(at::IntArrayRef shape, const at::Tensor& like, at::ScalarType type) {
  return at::empty(shape, like.options().dtype(type).requires_grad(false));
}

PyObject* g_out_of_memory = nullptr;             // torch.OutOfMemoryError

// Runs a call's body; C++ exceptions become Python ones.
template <typename Body>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, Body body) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return body();
  } catch (const PythonError&) {
    return nullptr;
  } catch (const std::bad_alloc&) {
    return PyErr_NoMemory();
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_out_of_memory, e.what_without_backtrace());
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}
// (status, result): a status other than 0 is raised by the caller.
PyObject* answer(svdq_status status, PyObject* result) {
  if (!result) return nullptr;
  return Py_BuildValue("iN", (int)status, result);
}

// q, k, q_weight, k_weight, eps, positions, inv_freq, pair_axis, interleaved, hadamard, inplace
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    int device = -1;
    svdq_qk_norm_rope_desc d = {};
    const at::Tensor& q = on_device(a[0], "q", &device);
    d.dtype = type_code(q, "q");
    d.q = heads_of(q, "q");
    d.tokens = count(q.size(0), "q");
    d.q_heads = count(q.size(1), "q");
    d.head_dim = count(q.size(2), "q");
    const at::Tensor* k = nullptr;
    if (given(a[1])) {
      k = &on_device(a[1], "k", &device);
      need_type(*k, "k", q.scalar_type());
      d.k = heads_of(*k, "k");
      if (k->size(0) != q.size(0) || k->size(2) != q.size(2))
        raise(PyExc_ValueError, "k: expected (%d, heads, %d), got %s", d.tokens, d.head_dim, shape_text(*k).c_str());
      d.k_heads = count(k->size(1), "k");
    } else if (given(a[3])) {
      raise(PyExc_ValueError, "k_weight without k");
    }
    bool in_graph = tracked(q) || (k && tracked(*k));
    if (given(a[2])) {
      const at::Tensor& w = vector(a[2], "q_weight", q.scalar_type(), d.head_dim, &device);
      d.q_weight = w.data_ptr();
      in_graph |= tracked(w);
    }
    if (given(a[3])) {
      const at::Tensor& w = vector(a[3], "k_weight", q.scalar_type(), d.head_dim, &device);
      d.k_weight = w.data_ptr();
      in_graph |= tracked(w);
    }
    d.eps = (float)number(a[4]);
    d.axes = 1;
    if (given(a[6])) {
      if (!given(a[5])) raise(PyExc_ValueError, "inv_freq without positions");
      const at::Tensor& pos = on_device(a[5], "positions", &device);
      need_type(pos, "positions", at::kInt);
      if (pos.dim() < 1 || pos.dim() > 2 || pos.size(0) != q.size(0) || (pos.dim() == 2 && pos.size(1) == 0))
        raise(PyExc_ValueError, "positions: expected (tokens,) or (tokens, axes), got %s", shape_text(pos).c_str());
      d.axes = pos.dim() == 2 ? count(pos.size(1), "positions") : 1;
      if (d.axes > 1 && pos.stride(1) != 1)
        raise(PyExc_ValueError, "positions: the axes of a token must be contiguous");
      d.positions = static_cast<const int*>(pos.data_ptr());
      d.position_stride = pos.stride(0);
      const at::Tensor& f = vector(a[6], "inv_freq", at::kFloat, -1, &device);
      d.pairs = count(f.size(0), "inv_freq");
      d.inv_freq = static_cast<const float*>(f.data_ptr());
      in_graph |= tracked(f);
      if (given(a[7]))
        d.pair_axis = static_cast<const unsigned char*>(vector(a[7], "pair_axis", at::kByte, d.pairs, &device).data_ptr());
    } else if (given(a[5]) || given(a[7])) {
      raise(PyExc_ValueError, "positions or pair_axis without inv_freq");
    }
    d.interleaved = truth(a[8]);
    d.hadamard = truth(a[9]);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    if (truth(a[10])) {
      distinct(q, "q");
      if (k) {
        distinct(*k, "k");
        apart(Memory(q, "q"), Memory(*k, "k"));
      }
      for (const int i : {0, 1, 2, 3, 6})
        if (given(a[i])) not_tracked(tensor(a[i], ""), "inplace");
      d.q_out = d.q;
      d.k_out = d.k;
      const svdq_status status = svdq_qk_norm_rope(&d, current_stream(device));
      if (status == SVDQ_OK) {
        changed(q);
        if (k) changed(*k);
      }
      return answer(status, PyTuple_Pack(2, a[0], a[1]));
    }
    at::Tensor q_out = empty(q.sizes(), q, q.scalar_type());
    d.q_out = contiguous_heads(q_out);
    at::Tensor k_out;
    if (k) {
      k_out = empty(k->sizes(), q, q.scalar_type());
      d.k_out = contiguous_heads(k_out);
    }
    const svdq_status status = svdq_qk_norm_rope(&d, current_stream(device));
    if (in_graph) {
      torch::autograd::variable_list inputs;
      for (const int i : {0, 1, 2, 3, 6})
        if (given(a[i])) inputs.push_back(tensor(a[i], ""));
      no_backward(q_out, "qk_norm_rope", inputs);
      no_backward(k_out, "qk_norm_rope", inputs);
    }
    return answer(status, Py_BuildValue("NN", THPVariable_Wrap(q_out), k ? THPVariable_Wrap(k_out) : Py_NewRef(Py_None)));
  });
}

// cache, k, v, slots
PyObject* kv4_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* {
    int device = -1;
    const at::Tensor& k = on_device(a[1], "k", &device);
    const int dtype = type_code(k, "k");
    Memory cache[4];
    const svdq_kv4_cache c = cache_of(a[0], &device, cache);
    const at::Tensor& slots = vector(a[3], "slots", at::kLong, -1, &device);
    const at::Tensor& v = on_device(a[2], "v", &device);
    need_type(v, "v", k.scalar_type());
    need_shape(k, "k", slots.size(0), c.heads, c.head_dim);
    need_shape(v, "v", slots.size(0), c.heads, c.head_dim);
    const svdq_heads ka = heads_of(k, "k"), va = heads_of(v, "v");
    const Memory inputs[3] = {Memory(k, "k"), Memory(v, "v"), Memory(slots, "slots")};
    for (int i = 0; i < 4; ++i) {
      for (const Memory& m : inputs) apart(cache[i], m);
      for (int j = 0; j < i; ++j) apart(cache[i], cache[j]);
    }
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    const svdq_status status = svdq_kv4_append(&c, &ka, &va, count(slots.size(0), "slots"), dtype,
                                               static_cast<const long long*>(slots.data_ptr()), current_stream(device));
    if (status == SVDQ_OK)
      for (const Memory& m : cache) changed(m.tensor);
    return answer(status, Py_NewRef(Py_None));
  });
}

// cache, slots, whether fp16
PyObject* kv4_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    int device = -1;
    const at::Tensor& slots = vector(a[1], "slots", at::kLong, -1, &device);
    const svdq_kv4_cache c = cache_of(a[0], &device);
    const bool half = truth(a[2]);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    const int64_t shape[3] = {slots.size(0), c.heads, c.head_dim};
    const at::Tensor k = empty(shape, slots, half ? at::kHalf : at::kBFloat16), v = empty(shape, slots, k.scalar_type());
    const svdq_heads ka = contiguous_heads(k), va = contiguous_heads(v);
    const svdq_status status = svdq_kv4_read(&c, &ka, &va, count(slots.size(0), "slots"), half ? 1 : 0,
                                             static_cast<const long long*>(slots.data_ptr()), current_stream(device));
    return answer(status, Py_BuildValue("NN", THPVariable_Wrap(k), THPVariable_Wrap(v)));
  });
}

// q, cache, kv_len, block_table, q_start, causal, softmax_scale, max_kv_len, out, return_lse
PyObject* kv4_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    int device = -1;
    svdq_kv4_attention_desc d = {};
    const at::Tensor& q = on_device(a[0], "q", &device);
    d.dtype = type_code(q, "q");
    Memory cache[4];
    d.cache = cache_of(a[1], &device, given(a[8]) ? cache : nullptr);
    d.q = heads_of(q, "q");
    d.tokens = count(q.size(0), "q");
    d.q_heads = count(q.size(1), "q");
    if (q.size(2) != d.cache.head_dim)
      raise(PyExc_ValueError, "q: head_dim %lld, the cache's is %d", (long long)q.size(2), d.cache.head_dim);
    const at::Tensor& lens = vector(a[2], "kv_len", at::kInt, -1, &device);
    d.requests = count(lens.size(0), "kv_len");
    d.kv_len = static_cast<const int*>(lens.data_ptr());
    const at::Tensor& table = on_device(a[3], "block_table", &device);
    need_type(table, "block_table", at::kInt);
    if (table.dim() != 2 || table.size(0) != d.requests)
      raise(PyExc_ValueError, "block_table: expected (%d, max_pages), got %s", d.requests, shape_text(table).c_str());
    if (table.size(1) > 1 && table.stride(1) != 1)
      raise(PyExc_ValueError, "block_table: a request's row must be contiguous");
    d.block_table = static_cast<const int*>(table.data_ptr());
    d.table_stride = table.stride(0);
    d.max_pages = count(table.size(1), "block_table");
    if (given(a[4])) {
      const at::Tensor& start = vector(a[4], "q_start", at::kInt, (int64_t)d.requests + 1, &device);
      d.q_start = static_cast<const int*>(start.data_ptr());
    }
    d.causal = truth(a[5]);
    d.softmax_scale = (float)(given(a[6]) ? number(a[6]) : 1.0 / std::sqrt((double)d.cache.head_dim));
    if (given(a[7])) {
      const long long most = PyLong_AsLongLong(a[7]);
      if (most == -1 && PyErr_Occurred()) throw PythonError();
      d.max_kv_len = most > 0x7FFFFFFF ? 0x7FFFFFFF : most < -1 ? -1 : (int)most;
    }
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    at::Tensor out, lse, work;
    if (given(a[8])) {
      out = on_device(a[8], "out", &device);
      need_type(out, "out", q.scalar_type());
      need_shape(out, "out", q.size(0), q.size(1), q.size(2));
      d.out = heads_of(out, "out");
      distinct(out, "out");
      not_tracked(out, "out");
      not_tracked(q, "q");
      const Memory written(out, "out");
      apart(written, Memory(q, "q"));
      for (const Memory& m : cache) apart(written, m);
      apart(written, Memory(lens, "kv_len"));
      apart(written, Memory(table, "block_table"));
      if (given(a[4])) apart(written, Memory(tensor(a[4], "q_start"), "q_start"));
    } else {
      out = empty(q.sizes(), q, q.scalar_type());
      d.out = contiguous_heads(out);
    }
    const bool want_lse = truth(a[9]);
    if (want_lse) {
      lse = empty({q.size(0), q.size(1)}, q, at::kFloat);
      d.lse = static_cast<float*>(lse.data_ptr());
    }
    // The workspace comes from the caching allocator, on the stream in use: calls on other streams and captured graphs
    // have their own.
    const size_t size = svdq_kv4_attention_workspace_bytes(&d);
    if (size) work = empty({(int64_t)size}, q, at::kByte);
    const svdq_status status = svdq_kv4_attention(&d, size ? work.data_ptr() : nullptr, size, current_stream(device));
    if (given(a[8])) {
      if (status == SVDQ_OK) changed(out);
    } else if (tracked(q)) {
      no_backward(out, "kv4_attention", {q});
    }
    if (want_lse && tracked(q)) no_backward(lse, "kv4_attention", {q});
    PyObject* first = given(a[8]) ? Py_NewRef(a[8]) : THPVariable_Wrap(out);
    return answer(status, want_lse ? Py_BuildValue("NN", first, THPVariable_Wrap(lse)) : first);
  });
}

#define CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(qk_norm_rope), CALL(kv4_append), CALL(kv4_read), CALL(kv4_attention),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_torch(void) {
  PyObject* torch = PyImport_ImportModule("torch");
  if (!torch) return nullptr;
  g_out_of_memory = PyObject_GetAttrString(torch, "OutOfMemoryError");
  Py_DECREF(torch);
  return g_out_of_memory ? PyModule_Create(&module) : nullptr;
}
