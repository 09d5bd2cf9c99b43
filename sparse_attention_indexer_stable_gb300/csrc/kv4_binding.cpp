// kv4_binding.cpp -- the torch side of the 4-bit cache's functions: checks the
// tensors, allocates what is not given, calls the C ABI (include/dcp_kv4.h).
//
// In C++ because the smallest calls are bound by the host: on the GB300's CPU
// the same checks and allocations took 18 us in Python beside 7 us of GPU time
// (attention of one row of 2048 tokens); here they take about a third.
//
// The library is loaded by the package, which hands its entry points over
// (connect), so that this module needs nothing but torch to be built.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>
#include <string>

#include "dcp_kv4.h"

namespace {

decltype(&dcp_kv4_append) g_append = nullptr;
decltype(&dcp_kv4_read) g_read = nullptr;
decltype(&dcp_kv4_attention_workspace_size) g_workspace_size = nullptr;
decltype(&dcp_kv4_attention) g_attention = nullptr;
decltype(&dcp_kv4_evict) g_evict = nullptr;

// A Python exception on its way out: `type` with `text`.
struct Refused {
  PyObject* type;
  std::string text;
};
[[noreturn]] void type_error(const std::string& text) { throw Refused{PyExc_TypeError, text}; }
[[noreturn]] void value_error(const std::string& text) { throw Refused{PyExc_ValueError, text}; }

const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
  return &THPVariable_Unpack(o);
}

const at::Tensor& needed(PyObject* o, const char* name) {
  const at::Tensor* t = tensor(o, name);
  if (!t) type_error(std::string(name) + " must be a torch.Tensor");
  return *t;
}

void check_type(const at::Tensor& t, const char* name, c10::ScalarType type) {
  if (t.scalar_type() != type)
    type_error(std::string(name) + " must be " + c10::toString(type) + ", got " +
               c10::toString(t.scalar_type()));
}

void check_device(const at::Tensor& t, const char* name, int dev) {
  if (!t.is_cuda() || t.get_device() != dev)
    value_error(std::string(name) + " must be on cuda:" + std::to_string(dev));
}

// A contiguous tensor of this type and shape.
void check(const at::Tensor& t, const char* name, c10::ScalarType type, int dev,
           at::IntArrayRef shape) {
  check_type(t, name, type);
  check_device(t, name, dev);
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  if (t.sizes() != shape) {
    std::string s;
    for (const int64_t n : shape) s += (s.empty() ? "" : ", ") + std::to_string(n);
    value_error(std::string(name) + " must be (" + s + ")");
  }
}

// A 2-D tensor whose rows are contiguous, at any stride.
void check_rows(const at::Tensor& t, const char* name, c10::ScalarType type, int dev,
                const char* what) {
  check_type(t, name, type);
  check_device(t, name, dev);
  if (t.dim() != 2 || (t.size(0) > 0 && t.size(1) > 1 && t.stride(1) != 1))
    value_error(std::string(name) + " must be " + what + ", its rows contiguous");
}

int value_type(const at::Tensor& t, const char* name, bool wide) {
  switch (t.scalar_type()) {
    case at::kHalf: return DCP_F16;
    case at::kBFloat16: return DCP_BF16;
    case at::kFloat:
      if (wide) return DCP_F32;
      break;
    default: break;
  }
  type_error(std::string(name) + " must be a torch.Tensor of float16" +
             (wide ? ", bfloat16 or float32" : " or bfloat16"));
}

// (n, heads, dim) values with unit stride along dim.
void check_values(const at::Tensor& t, const char* name, int dev, int dim) {
  check_device(t, name, dev);
  if (t.dim() != 3 || t.size(2) != dim || t.stride(2) != 1)
    value_error(std::string(name) +
                " must be 3-D, its last dimension dim = " + std::to_string(dim) + " contiguous");
}

int to_int(int64_t n, const char* name) {
  if (n > INT32_MAX) value_error(std::string(name) + " is too large");
  return (int)n;
}

// The device, and the stream that a call runs on: `stream` (a raw handle), or
// the device's current one.  What is allocated meanwhile belongs to it, so it
// may be freed as soon as the call returns.
struct Place {
  c10::cuda::OptionalCUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard other;
  dcp_stream_t stream;

  Place(int dev, PyObject* handle) {
    if (c10::cuda::current_device() != dev) device.set_index((c10::DeviceIndex)dev);
    if (handle == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    } else {
      void* p = PyLong_AsVoidPtr(handle);
      if (!p && PyErr_Occurred()) throw python_error();
      stream = static_cast<dcp_stream_t>(p);
      if (p)
        other.reset_stream(c10::cuda::getStreamFromExternal(stream, (c10::DeviceIndex)dev));
      else
        other.reset_stream(c10::cuda::getDefaultCUDAStream((c10::DeviceIndex)dev));
    }
  }
};

at::Tensor allocate(at::IntArrayRef shape, c10::ScalarType type, int dev) {
  return at::empty(shape, at::TensorOptions(type).device(at::kCUDA, (c10::DeviceIndex)dev));
}

const dcp_kv4_cache* cache_of(PyObject* raw) {
  if (!PyBytes_Check(raw) || PyBytes_GET_SIZE(raw) != (Py_ssize_t)sizeof(dcp_kv4_cache))
    type_error("cache must be a Kv4Cache");
  return reinterpret_cast<const dcp_kv4_cache*>(PyBytes_AS_STRING(raw));
}

int int_of(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  if (v > INT32_MAX || v < INT32_MIN) value_error("a size is out of range");
  return (int)v;
}

float float_of(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)v;
}

template <typename T>
T* ptr(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

// Runs a function body: its result, or the exception that it left with.
template <typename F>
PyObject* guarded(F body) {
  HANDLE_TH_ERRORS
  try {
    return body();
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

bool takes(Py_ssize_t given, Py_ssize_t wanted) {
  if (given == wanted) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", wanted, given);
  return false;
}

// The library's functions neither touch Python nor throw.
template <typename F>
dcp_status call(F f) {
  PyThreadState* state = PyEval_SaveThread();
  const dcp_status st = f();
  PyEval_RestoreThread(state);
  return st;
}

// append(cache, device, k, v, slots, stream) -> status
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!takes(n, 6)) return nullptr;
  return guarded([&]() -> PyObject* {
    const dcp_kv4_cache* c = cache_of(a[0]);
    const int dev = int_of(a[1]);
    const at::Tensor &k = needed(a[2], "k"), &v = needed(a[3], "v"), &s = needed(a[4], "slots");
    const int type = value_type(k, "k", true);
    if (value_type(v, "v", true) != type || k.sizes() != v.sizes())
      value_error("k and v must both be (N, heads, dim) of one dtype");
    check_values(k, "k", dev, c->dim);
    check_values(v, "v", dev, c->dim);
    if (k.size(1) != c->heads) value_error("k and v must have the cache's heads");
    check(s, "slots", at::kLong, dev, {k.size(0)});
    const Place place(dev, a[5]);
    return PyLong_FromLong(call([&] {
      return g_append(c, k.data_ptr(), v.data_ptr(), type, k.size(0), k.stride(0), k.stride(1),
                      v.stride(0), v.stride(1), static_cast<const int64_t*>(s.data_ptr()),
                      place.stream);
    }));
  });
}

// read(cache, device, slots, dtype code, k, v, stream) -> (k, v) or status
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!takes(n, 7)) return nullptr;
  return guarded([&]() -> PyObject* {
    const dcp_kv4_cache* c = cache_of(a[0]);
    const int dev = int_of(a[1]), type = int_of(a[3]);
    const at::Tensor& s = needed(a[2], "slots");
    const at::Tensor *gk = tensor(a[4], "k"), *gv = tensor(a[5], "v");
    if (s.dim() != 1) value_error("slots must be (N,)");
    check(s, "slots", at::kLong, dev, s.sizes());
    const c10::ScalarType kind = type == DCP_F16 ? at::kHalf
                                 : type == DCP_BF16 ? at::kBFloat16 : at::kFloat;
    const int64_t shape[3] = {s.size(0), c->heads, c->dim};
    const Place place(dev, a[6]);
    if (gk) check(*gk, "k", kind, dev, shape);
    if (gv) check(*gv, "v", kind, dev, shape);
    const at::Tensor k = gk ? *gk : allocate(shape, kind, dev);
    const at::Tensor v = gv ? *gv : allocate(shape, kind, dev);
    const dcp_status st = call([&] {
      return g_read(c, k.data_ptr(), v.data_ptr(), type, shape[0],
                    static_cast<const int64_t*>(s.data_ptr()), place.stream);
    });
    if (st != DCP_OK) return PyLong_FromLong(st);
    return Py_BuildValue("(NN)", THPVariable_Wrap(k), THPVariable_Wrap(v));
  });
}

// attention(cache, device, q, table, lens, ids, owner, starts, row_starts,
//           scale, softcap, weights, max_len, out, lse, workspace, stream)
//   -> (out, lse) or status
PyObject* attention(PyObject*, PyObject* const* p, Py_ssize_t n) {
  if (!takes(n, 17)) return nullptr;
  return guarded([&]() -> PyObject* {
    const dcp_kv4_cache* c = cache_of(p[0]);
    const int dev = int_of(p[1]);
    const at::Tensor &q = needed(p[2], "q"), &table = needed(p[3], "table"),
                     &lens = needed(p[4], "lens");
    const at::Tensor *ids = tensor(p[5], "ids"), *owner = tensor(p[6], "owner"),
                     *starts = tensor(p[7], "starts"), *row_starts = tensor(p[8], "row_starts"),
                     *weights = tensor(p[11], "weights"), *given_out = tensor(p[13], "out"),
                     *given_lse = tensor(p[14], "lse"), *given_ws = tensor(p[15], "workspace");
    dcp_kv4_attention_args a{};
    a.dtype = value_type(q, "q", false);
    check_values(q, "q", dev, c->dim);
    const int64_t T = q.size(0), heads = q.size(1);
    if (heads < 1 || heads % c->heads)
      value_error("q's heads must be a multiple of the cache's heads");
    check_rows(table, "table", at::kInt, dev, "(sequences, pages)");
    check(lens, "lens", at::kInt, dev, {T});
    if (starts) check(*starts, "starts", at::kInt, dev, {T});
    if (owner) check(*owner, "owner", at::kInt, dev, {T});
    if (row_starts) check(*row_starts, "row_starts", at::kInt, dev, {T});
    if (!owner && table.size(0) < T)
      value_error("table must have a row for each row of q (or give owner)");
    a.softcap = float_of(p[10]);
    if (!std::isfinite(a.softcap) || a.softcap < 0.0f)
      value_error("softcap must be finite and not negative");
    a.scale = p[9] == Py_None ? 0.0f : float_of(p[9]);
    if (!std::isfinite(a.scale)) value_error("scale must be finite");
    a.q = q.data_ptr();
    a.q_row_stride = q.stride(0);
    a.q_head_stride = q.stride(1);
    a.table = static_cast<const int32_t*>(table.data_ptr());
    a.table_stride = table.stride(0);
    a.lens = static_cast<const int32_t*>(lens.data_ptr());
    a.starts = ptr<const int32_t>(starts);
    a.owner = ptr<const int32_t>(owner);
    a.row_starts = ptr<const int32_t>(row_starts);
    if (ids) {
      check_rows(*ids, "ids", at::kInt, dev, "(T, K)");
      if (ids->size(0) != T) value_error("ids must be (T, K)");
      // No ids at all (K = 0) have no address, and a null one means every
      // position; nothing is read from this one.
      a.ids = ids->data_ptr() ? ptr<const int32_t>(ids) : a.lens;
      a.num_ids = to_int(ids->size(1), "K");
      a.ids_stride = ids->stride(0);
    }
    if (weights) {
      check_rows(*weights, "weights", at::kFloat, dev, "(T, positions)");
      if (owner) value_error("weights need one row per sequence: not with owner");
      if (weights->size(0) != T) value_error("weights must be (T, positions)");
      if (T > 1 && weights->stride(0) < weights->size(1))
        value_error("the rows of weights must not overlap");
      a.weights = ptr<float>(weights);
      a.weights_stride = weights->stride(0);
      a.weights_width = weights->size(1);
    }
    a.rows = to_int(T, "T");
    a.q_heads = to_int(heads, "q's heads");
    a.num_seqs = to_int(table.size(0), "sequences");
    a.table_width = to_int(table.size(1), "pages");
    a.max_len = int_of(p[12]);
    const int64_t out_shape[3] = {T, heads, c->dim}, lse_shape[2] = {T, heads};
    const Place place(dev, p[16]);
    if (given_out) check(*given_out, "out", q.scalar_type(), dev, out_shape);
    if (given_lse) check(*given_lse, "lse", at::kFloat, dev, lse_shape);
    size_t need = 0;
    dcp_status st = g_workspace_size(c, &a, &need);
    if (st != DCP_OK) return PyLong_FromLong(st);
    const at::Tensor out = given_out ? *given_out : allocate(out_shape, q.scalar_type(), dev);
    const at::Tensor lse = given_lse ? *given_lse : allocate(lse_shape, at::kFloat, dev);
    std::optional<at::Tensor> workspace;
    if (given_ws) {
      check(*given_ws, "workspace", at::kByte, dev, given_ws->sizes());
      if ((size_t)given_ws->numel() < need)
        value_error("workspace must hold " + std::to_string(need) + " bytes");
      workspace = *given_ws;
    } else if (need) {
      workspace = allocate({(int64_t)need}, at::kByte, dev);
    }
    a.out = out.data_ptr();
    a.lse = static_cast<float*>(lse.data_ptr());
    if (workspace) {
      a.workspace = workspace->data_ptr();
      a.workspace_bytes = (size_t)workspace->numel();
    }
    st = call([&] { return g_attention(c, &a, place.stream); });
    if (st != DCP_OK) return PyLong_FromLong(st);
    return Py_BuildValue("(NN)", THPVariable_Wrap(out), THPVariable_Wrap(lse));
  });
}

// evict(cache, device, table, lens, weights, out_table, budget, sinks, recent,
//       kept, out_lens, out_weights, stream)
//   -> (kept, out_lens, out_weights) or status
PyObject* evict(PyObject*, PyObject* const* p, Py_ssize_t n) {
  if (!takes(n, 13)) return nullptr;
  return guarded([&]() -> PyObject* {
    const dcp_kv4_cache* c = cache_of(p[0]);
    const int dev = int_of(p[1]);
    const at::Tensor &table = needed(p[2], "table"), &lens = needed(p[3], "lens"),
                     &weights = needed(p[4], "weights"), &out_table = needed(p[5], "out_table");
    const at::Tensor *given_kept = tensor(p[9], "kept"), *given_lens = tensor(p[10], "out_lens"),
                     *given_weights = tensor(p[11], "out_weights");
    dcp_kv4_evict_args a{};
    a.budget = int_of(p[6]);
    a.sinks = int_of(p[7]);
    a.recent = int_of(p[8]);
    if (a.budget < 1 || a.sinks < 0 || a.recent < 0 ||
        (int64_t)a.sinks + a.recent > a.budget)
      value_error("need budget >= 1, sinks >= 0, recent >= 0, sinks + recent <= budget");
    check_rows(table, "table", at::kInt, dev, "(sequences, pages)");
    check_rows(out_table, "out_table", at::kInt, dev, "(sequences, pages)");
    check_rows(weights, "weights", at::kFloat, dev, "(sequences, positions)");
    const int64_t B = table.size(0);
    if (weights.size(0) != B || out_table.size(0) != B)
      value_error("table, weights and out_table must have a row for each sequence");
    if (out_table.size(1) * c->page_size < a.budget)
      value_error("out_table must have ceil(budget / page_size) pages for each sequence");
    check(lens, "lens", at::kInt, dev, {B});
    const int64_t shape[2] = {B, a.budget};
    const Place place(dev, p[12]);
    if (given_kept) check(*given_kept, "kept", at::kInt, dev, shape);
    if (given_lens) check(*given_lens, "out_lens", at::kInt, dev, {B});
    if (given_weights) check(*given_weights, "out_weights", at::kFloat, dev, shape);
    const at::Tensor kept = given_kept ? *given_kept : allocate(shape, at::kInt, dev);
    const at::Tensor out_lens = given_lens ? *given_lens : allocate({B}, at::kInt, dev);
    const at::Tensor out_weights =
        given_weights ? *given_weights : allocate(shape, at::kFloat, dev);
    a.table = static_cast<const int32_t*>(table.data_ptr());
    a.table_stride = table.stride(0);
    a.lens = static_cast<const int32_t*>(lens.data_ptr());
    a.weights = static_cast<const float*>(weights.data_ptr());
    a.weights_stride = weights.stride(0);
    a.out_table = static_cast<const int32_t*>(out_table.data_ptr());
    a.out_table_stride = out_table.stride(0);
    a.kept = static_cast<int32_t*>(kept.data_ptr());
    a.out_lens = static_cast<int32_t*>(out_lens.data_ptr());
    a.out_weights = static_cast<float*>(out_weights.data_ptr());
    a.num_seqs = to_int(B, "sequences");
    a.table_width = to_int(table.size(1), "pages");
    a.weights_width = to_int(weights.size(1), "positions");
    const dcp_status st = call([&] { return g_evict(c, &a, place.stream); });
    if (st != DCP_OK) return PyLong_FromLong(st);
    return Py_BuildValue("(NNN)", THPVariable_Wrap(kept), THPVariable_Wrap(out_lens),
                         THPVariable_Wrap(out_weights));
  });
}

// connect(append, read, workspace size, attention, evict): their addresses
PyObject* connect(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!takes(n, 5)) return nullptr;
  void* f[5];
  for (int i = 0; i < 5; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (!f[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null entry point");
      return nullptr;
    }
  }
  g_append = reinterpret_cast<decltype(g_append)>(f[0]);
  g_read = reinterpret_cast<decltype(g_read)>(f[1]);
  g_workspace_size = reinterpret_cast<decltype(g_workspace_size)>(f[2]);
  g_attention = reinterpret_cast<decltype(g_attention)>(f[3]);
  g_evict = reinterpret_cast<decltype(g_evict)>(f[4]);
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef g_methods[] = {
    {"connect", fast(connect), METH_FASTCALL, nullptr},
    {"append", fast(append), METH_FASTCALL, nullptr},
    {"read", fast(read), METH_FASTCALL, nullptr},
    {"attention", fast(attention), METH_FASTCALL, nullptr},
    {"evict", fast(evict), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_kv4_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv4_binding(void) { return PyModule_Create(&g_module); }
