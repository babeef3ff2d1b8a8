// Python binding of the cache and attention entry points: argument checks,
// allocation and the call in one step. A decode step makes these calls once a
// layer with kernels of a few microseconds, and the same checks made in Python
// took three to four times as long as the launch.
//
// Argument rules and messages are those that attention.py documents; every
// function runs on torch's current stream of the cache's device.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <stdexcept>
#include <string>

#include "../../include/sai.h"

namespace {

struct Refused : std::invalid_argument {  // becomes a ValueError
  using std::invalid_argument::invalid_argument;
};
struct Failed {  // becomes a SaiError
  int status;
  const char* where;
};
struct Raised {};  // a Python error is set

[[noreturn]] void refuse(const std::string& s) { throw Refused(s); }

// The KVCache object's descriptor and device, kept by the Python object.
struct Cache {
  const sai_kv_cache* d;
  int device;
};

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
int32_t int32_of(PyObject* o, const char* name) {
  const long long v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " does not fit 32 bits");
  return static_cast<int32_t>(v);
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v == 1;
}

const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}

const char* type_name(at::ScalarType t) {
  return t == at::kBFloat16 ? "torch.bfloat16" : t == at::kInt ? "torch.int32" : t == at::kFloat ? "torch.float32" : "torch.uint8";
}

// Required tensor on the device, of this type and number of dims.
const at::Tensor& need(PyObject* o, const char* name, at::ScalarType type, int64_t dims, int device) {
  const at::Tensor* t = tensor(o, name);
  if (!t) refuse(std::string(name) + " is required");
  if (!t->is_cuda() || t->get_device() != device)
    refuse(std::string(name) + " must be on cuda:" + std::to_string(device));
  if (t->scalar_type() != type) refuse(std::string(name) + " must be " + type_name(type));
  if (t->dim() != dims) refuse(std::string(name) + " must have " + std::to_string(dims) + " dims");
  return *t;
}

// int32 [rows], contiguous.
const int32_t* row_index(PyObject* o, const char* name, int64_t rows, int device) {
  const at::Tensor& t = need(o, name, at::kInt, 1, device);
  if (t.size(0) != rows || !t.is_contiguous()) refuse(std::string(name) + " must be contiguous [" + std::to_string(rows) + "]");
  return static_cast<const int32_t*>(t.data_ptr());
}

struct Rows {
  const uint16_t* p;
  int64_t stride;
  int32_t heads;
};
// bf16 [rows, heads, dim], heads and dims contiguous, any row stride.
Rows rows_of(PyObject* o, const char* name, int64_t rows, int64_t heads, const Cache& c) {
  const at::Tensor& t = need(o, name, at::kBFloat16, 3, c.device);
  if (t.size(0) != rows || t.size(2) != c.d->dim || (heads && t.size(1) != heads))
    refuse(std::string(name) + " must be [" + std::to_string(rows) + ", " + (heads ? std::to_string(heads) : "heads") + ", " +
           std::to_string(c.d->dim) + "]");
  if (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != c.d->dim))
    refuse(std::string(name) + " needs contiguous heads");
  return Rows{static_cast<const uint16_t*>(t.data_ptr()), rows > 1 ? t.stride(0) : t.size(1) * c.d->dim,
              static_cast<int32_t>(t.size(1))};
}

struct Table {
  const int32_t* p;
  int64_t rows, stride;
  int64_t cells;  // tokens that a row of it names, if rows are more than that apart; else no bound of its own
};
// int32 [requests, blocks], perhaps columns of a wider table: the library
// bounds lengths by the stride, so the bound by columns is passed beside it.
Table table_of(PyObject* o, const Cache& c) {
  const at::Tensor& t = need(o, "block_table", at::kInt, 2, c.device);
  const int64_t rows = t.size(0), cols = t.size(1), stride = rows > 1 && cols > 0 ? t.stride(0) : cols;
  if ((cols > 1 && t.stride(1) != 1) || stride < cols)
    refuse("block_table needs unit column stride and rows that do not overlap");
  return Table{static_cast<const int32_t*>(t.data_ptr()), rows, stride,
               stride > cols ? cols * c.d->block_size : INT64_MAX};
}

Cache cache_of(PyObject* ref, PyObject* device) {
  Cache c{static_cast<const sai_kv_cache*>(PyLong_AsVoidPtr(ref)), int32_of(device, "device")};
  if (PyErr_Occurred()) throw Raised{};
  const int now = c10::cuda::current_device();
  if (now != c.device)
    refuse("the current device is cuda:" + std::to_string(now) + ", the cache is on cuda:" + std::to_string(c.device));
  return c;
}

sai_stream_t stream_of(const Cache& c) {
  return reinterpret_cast<sai_stream_t>(c10::cuda::getCurrentCUDAStream(c.device).stream());
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const Cache& c) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, c.device)));
}

// A given output, or a new one: contiguous, of this type and shape.
at::Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, const Cache& c) {
  const at::Tensor* t = tensor(o, name);
  if (!t) return fresh(shape, type, c);
  if (!t->is_cuda() || t->get_device() != c.device || t->scalar_type() != type || t->sizes() != shape || !t->is_contiguous()) {
    std::string s;
    for (int64_t x : shape) s += (s.empty() ? "" : ", ") + std::to_string(x);
    refuse(std::string(name) + " must be contiguous " + type_name(type) + " [" + s + "]");
  }
  return *t;
}

struct Space {
  at::Tensor hold;
  void* p = nullptr;
  size_t bytes = 0;
};
Space workspace_of(PyObject* o, size_t bytes, const Cache& c) {
  Space w;
  if (const at::Tensor* t = tensor(o, "workspace")) {
    if (!t->is_cuda() || t->get_device() != c.device || !t->is_contiguous())
      refuse("workspace must be contiguous on cuda:" + std::to_string(c.device));
    w.p = t->data_ptr();
    w.bytes = t->nbytes();
  } else if (bytes) {
    w.hold = fresh({static_cast<int64_t>(bytes)}, at::kByte, c);
    w.p = w.hold.data_ptr();
    w.bytes = bytes;
  }
  return w;
}

void check(int status, const char* where) {
  if (status != SAI_OK) throw Failed{status, where};
}

// (cache, device, k, v, block_table, seq_lens, cos_sin, q, out_q, row_to_batch, interleaved)
PyObject* append_kv(PyObject* const* a) {
  const Cache c = cache_of(a[0], a[1]);
  const at::Tensor* kt = tensor(a[2], "k");
  if (!kt || kt->dim() != 3) refuse("k must have 3 dims");
  const int64_t rows = kt->size(0);
  const Rows k = rows_of(a[2], "k", rows, c.d->heads, c), v = rows_of(a[3], "v", rows, c.d->heads, c);
  const Table bt = table_of(a[4], c);
  const int32_t* lens = row_index(a[5], "seq_lens", rows, c.device);
  const int32_t* r2b = a[9] == Py_None ? nullptr : row_index(a[9], "row_to_batch", rows, c.device);
  const float* cs = nullptr;
  int64_t max_pos = bt.cells, rot = 0;
  if (a[6] != Py_None) {
    const at::Tensor& t = need(a[6], "cos_sin", at::kFloat, 2, c.device);
    if (!t.is_contiguous()) refuse("cos_sin must be contiguous");
    cs = static_cast<const float*>(t.data_ptr());
    rot = std::min<int64_t>(t.size(1), INT32_MAX);
    if (rot) max_pos = std::min(max_pos, t.size(0));  // angles of no dims bound nothing
  }
  const bool interleaved = truth(a[10]);
  Rows q{nullptr, 0, 0};
  at::Tensor out;
  if (a[7] != Py_None) {
    q = rows_of(a[7], "q", rows, 0, c);
    out = output(a[8], "out_q", {rows, q.heads, c.d->dim}, at::kBFloat16, c);
  } else if (a[8] != Py_None) {
    refuse("out_q goes with q");
  }
  check(sai_append_kv(c.d, k.p, k.stride, v.p, v.stride, q.p, q.stride, q.heads,
                      out.defined() ? static_cast<uint16_t*>(out.data_ptr()) : nullptr, cs, max_pos,
                      static_cast<int32_t>(rot), interleaved, bt.p, bt.rows, bt.stride, r2b, lens, rows,
                      stream_of(c)),
        "sai_append_kv");
  if (!out.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(out);
}

double scale_of(PyObject* o, const Cache& c) {
  if (o == Py_None) return 1.0 / std::sqrt(static_cast<double>(c.d->dim));
  const double s = PyFloat_AsDouble(o);
  if (s == -1.0 && PyErr_Occurred()) throw Raised{};
  return s;
}

PyObject* attention_result(const at::Tensor& out, const at::Tensor& lse) {
  PyObject* o = THPVariable_Wrap(out);
  if (!o || !lse.defined()) return o;
  PyObject* l = THPVariable_Wrap(lse);
  PyObject* r = l ? PyTuple_Pack(2, o, l) : nullptr;
  Py_DECREF(o);
  Py_XDECREF(l);
  return r;
}

// (cache, device, q, block_table, seq_lens, max_seq_len, row_to_batch, packed, window, sinks, sm_scale, out, want_lse,
//  out_lse, workspace)
PyObject* paged_attention(PyObject* const* a) {
  const Cache c = cache_of(a[0], a[1]);
  const at::Tensor* qt = tensor(a[2], "q");
  if (!qt || qt->dim() != 3) refuse("q must have 3 dims");
  const int64_t rows = qt->size(0);
  const Rows q = rows_of(a[2], "q", rows, 0, c);
  const Table bt = table_of(a[3], c);
  const int32_t* lens = row_index(a[4], "seq_lens", rows, c.device);
  const int32_t most = static_cast<int32_t>(std::min<int64_t>(int32_of(a[5], "max_seq_len"), bt.cells)), window = int32_of(a[8], "window"), sinks = int32_of(a[9], "sinks");
  const int32_t* r2b = a[6] == Py_None ? nullptr : row_index(a[6], "row_to_batch", rows, c.device);
  const int32_t packed = int32_of(a[7], "packed");  // False, True, PACKED_TILES
  if (packed && !r2b) refuse("packed rows need row_to_batch");
  const double scale = scale_of(a[10], c);
  const at::Tensor out = output(a[11], "out", {rows, q.heads, c.d->dim}, at::kBFloat16, c);
  at::Tensor lse;
  if (truth(a[12]) || a[13] != Py_None) lse = output(a[13], "out_lse", {rows, q.heads}, at::kFloat, c);
  const Space w = workspace_of(a[14], a[14] == Py_None ? sai_paged_attention_workspace(rows, q.heads, c.d->heads, c.d->dim,
                                                                                       c.d->dtype, most, window, sinks, packed)
                                                       : 0, c);
  check(sai_paged_attention(q.p, q.stride, q.heads, c.d, bt.p, bt.rows, bt.stride, r2b, lens, rows, most, window, sinks,
                            static_cast<float>(scale), packed, static_cast<uint16_t*>(out.data_ptr()),
                            lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr, w.p, w.bytes, stream_of(c)),
        "sai_paged_attention");
  return attention_result(out, lse);
}

// (cache, device, q, slots, sm_scale, out, want_lse, out_lse, workspace)
PyObject* sparse_attention(PyObject* const* a) {
  const Cache c = cache_of(a[0], a[1]);
  const at::Tensor* qt = tensor(a[2], "q");
  if (!qt || qt->dim() != 3) refuse("q must have 3 dims");
  const int64_t rows = qt->size(0);
  const Rows q = rows_of(a[2], "q", rows, 0, c);
  const at::Tensor& slots = need(a[3], "slots", at::kInt, 2, c.device);
  const int64_t k = slots.size(1);
  if (slots.size(0) != rows || (k > 1 && slots.stride(1) != 1))
    refuse("slots must be [" + std::to_string(rows) + ", k] with unit column stride");
  if (k > INT32_MAX) refuse("slots does not fit 32 bits");
  const double scale = scale_of(a[4], c);
  const at::Tensor out = output(a[5], "out", {rows, q.heads, c.d->dim}, at::kBFloat16, c);
  at::Tensor lse;
  if (truth(a[6]) || a[7] != Py_None) lse = output(a[7], "out_lse", {rows, q.heads}, at::kFloat, c);
  const int32_t k32 = static_cast<int32_t>(k);
  const Space w = workspace_of(
      a[8], a[8] == Py_None ? sai_sparse_attention_workspace(rows, q.heads, c.d->heads, c.d->dim, c.d->dtype, k32) : 0, c);
  check(sai_sparse_attention(q.p, q.stride, q.heads, c.d, static_cast<const int32_t*>(slots.data_ptr()),
                             rows > 1 ? slots.stride(0) : std::max<int64_t>(k, 1), k32, rows, static_cast<float>(scale),
                             static_cast<uint16_t*>(out.data_ptr()),
                             lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr, w.p, w.bytes, stream_of(c)),
        "sai_sparse_attention");
  return attention_result(out, lse);
}

// Runs one of the above; C++ exceptions become Python errors.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const Failed& f) {
    // SaiError(status, where) of _lib.py
    PyObject* m = PyImport_ImportModule("sparse_attention_indexer_top_gb300._lib");
    PyObject* type = m ? PyObject_GetAttrString(m, "SaiError") : nullptr;
    PyObject* err = type ? PyObject_CallFunction(type, "is", f.status, f.where) : nullptr;
    if (err) PyErr_SetObject(type, err);
    Py_XDECREF(err);
    Py_XDECREF(type);
    Py_XDECREF(m);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyMethodDef methods[] = {
    {"append_kv", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&guarded<append_kv, 11>)), METH_FASTCALL, nullptr},
    {"paged_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&guarded<paged_attention, 15>)), METH_FASTCALL,
     nullptr},
    {"sparse_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&guarded<sparse_attention, 9>)), METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
