// The calls of ops.py whose smallest uses wait for the host: checks of the tensors and the call of the C ABI's function, in
// place of ctypes (about 16 us a call on a GB300's host, of which the function itself takes 3 to 5).  Same checks, same
// errors; every computation runs in libadp.so, whose functions' addresses the package hands over once.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <exception>
#include <optional>
#include <string>

#include "../../include/adp.h"

namespace {

// What the package hands over: its exception type, and addresses in the order of the names below.
PyObject* error_type = nullptr;
struct {
  decltype(&adp_paged_kv_append) append;
  decltype(&adp_paged_attention) attention;
  decltype(&adp_paged_attention_workspace) attention_workspace;
  decltype(&adp_paged_window_attention) window;
  decltype(&adp_paged_window_attention_workspace) window_workspace;
  decltype(&adp_paged_chunk_attention) chunk;
  decltype(&adp_paged_chunk_attention_workspace) chunk_workspace;
} lib;

// A call that was refused, or that failed (`where` is all of the message's beginning).
struct Refused {
  int code;
  std::string where;
};
[[noreturn]] void refuse(const char* where, const std::string& what) { throw Refused{ADP_ERR_INVALID_ARG, std::string(where) + ": " + what}; }
void check(int rc, const char* name) {
  if (rc != ADP_OK) throw Refused{rc, name};
}
struct PythonError {};

using at::Tensor;

const Tensor& tensor(const char* where, const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) refuse(where, std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
std::optional<Tensor> maybe(const char* where, const char* name, PyObject* o) {
  if (o == Py_None) return std::nullopt;
  return tensor(where, name, o);
}
int cuda_index(const Tensor& t) { return t.is_cuda() ? t.get_device() : -1; }
std::string on(int device) { return " on device " + std::to_string(device); }

int rows_type(at::ScalarType t) { return t == at::kHalf ? ADP_F16 : t == at::kBFloat16 ? ADP_BF16 : t == at::kFloat ? ADP_F32 : -1; }
int half_type(at::ScalarType t) { return t == at::kHalf ? ADP_F16 : t == at::kBFloat16 ? ADP_BF16 : -1; }

// Address of a contiguous int32 [n] tensor on the device.
const int32_t* indices(const char* where, const char* name, const Tensor& t, int64_t n, int device) {
  if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous() || cuda_index(t) != device)
    refuse(where, std::string(name) + " must be a contiguous int32 tensor [" + std::to_string(n) + "]" + on(device));
  return static_cast<const int32_t*>(t.data_ptr());
}
// Elements from one row to the next of a [rows, heads, head_dim] tensor whose rows may lie apart.
int64_t rows(const char* where, const char* name, const Tensor& t, int64_t n, int64_t heads, int64_t hd, at::ScalarType dtype, int device) {
  if (t.dim() != 3 || t.size(0) != n || t.size(1) != heads || t.size(2) != hd || t.scalar_type() != dtype || cuda_index(t) != device)
    refuse(where, std::string(name) + " must be (" + std::to_string(n) + ", " + std::to_string(heads) + ", " + std::to_string(hd) + ") of " +
                      c10::toString(dtype) + on(device));
  if (t.is_contiguous() || n == 0) return heads * hd;
  if (t.stride(2) != 1 || (t.stride(1) != hd && heads > 1)) refuse(where, std::string(name) + " must have contiguous heads");
  return n > 1 ? t.stride(0) : heads * hd;  // (the stride of a single row says nothing)
}
int32_t* status_of(const char* where, PyObject* o, int device) {
  if (o == Py_None) return nullptr;
  const Tensor& t = tensor(where, "status", o);
  if (t.scalar_type() != at::kInt || t.numel() != 1 || cuda_index(t) != device) refuse(where, "status must be one int32" + on(device));
  return static_cast<int32_t*>(t.data_ptr());
}

adp_paged_kv paged(const char* where, PyObject* const* o, PyObject* k_scale_o, PyObject* v_scale_o, int* device) {
  const Tensor &k = tensor(where, "k_pages", o[0]), &v = tensor(where, "v_pages", o[1]), &table = tensor(where, "table", o[2]),
               &lens = tensor(where, "lens", o[3]);
  if (!k.is_cuda()) refuse(where, "the tensors must be on a CUDA device");
  const int d = *device = k.get_device();
  const auto type = k.scalar_type();
  const int dt = type == at::kFloat8_e4m3fn ? ADP_E4M3 : half_type(type);
  if (dt < 0 || k.dim() != 4 || v.scalar_type() != type || v.sizes() != k.sizes() || cuda_index(v) != d)
    refuse(where, "k_pages and v_pages must be alike: [pages, kv_heads, page_size, head_dim], f16, bf16 or e4m3");
  const int64_t n = k.size(0), heads = k.size(1), ps = k.size(2), hd = k.size(3);
  int64_t page = heads * ps * hd, scales = heads * ps;
  if (!k.is_contiguous() || !v.is_contiguous()) {
    if (v.strides() != k.strides()) refuse(where, "k_pages and v_pages must have the same strides");
    if (page && (k.stride(3) != 1 || (k.stride(2) != hd && ps > 1) || (k.stride(1) != ps * hd && heads > 1)))
      refuse(where, "a page must be contiguous");
    if (n > 1) page = k.stride(0);  // (the stride of a single page says nothing)
  }
  if (table.scalar_type() != at::kInt || table.dim() != 2 || !table.is_contiguous() || cuda_index(table) != d)
    refuse(where, "table must be a contiguous int32 tensor [seqs, width]" + on(d));
  const int64_t seqs = table.size(0), width = table.size(1), most = 0x7FFFFFFF;
  if (n > most || heads > most || ps > most || hd > most || seqs > most || width > most) refuse(where, "a size is beyond 32 bits");
  adp_paged_kv kv{};
  kv.lens = indices(where, "lens", lens, seqs, d);
  if (dt == ADP_E4M3) {
    const auto ks = maybe(where, "k_scale", k_scale_o), vs = maybe(where, "v_scale", v_scale_o);
    const bool alike = ks && vs && ks->scalar_type() == at::kFloat && vs->scalar_type() == at::kFloat && ks->sizes() == k.sizes().slice(0, 3) &&
                       vs->sizes() == k.sizes().slice(0, 3) && cuda_index(*ks) == d && cuda_index(*vs) == d;
    if (!alike) refuse(where, "e4m3 pages need k_scale and v_scale: fp32 [pages, kv_heads, page_size]");
    if (!ks->is_contiguous() || !vs->is_contiguous()) {
      if (vs->strides() != ks->strides() || (ks->stride(2) != 1 && ps > 1) || (ks->stride(1) != ps && heads > 1))
        refuse(where, "k_scale and v_scale must have the same strides, and contiguous pages");
      if (n > 1) scales = ks->stride(0);
    }
    kv.k_scale = static_cast<float*>(ks->data_ptr());
    kv.v_scale = static_cast<float*>(vs->data_ptr());
  }
  kv.k = k.data_ptr();
  kv.v = v.data_ptr();
  kv.table = static_cast<const int32_t*>(table.data_ptr());
  kv.page_stride = page;
  kv.scale_stride = scales;
  kv.n_pages = (int32_t)n;
  kv.page_size = (int32_t)ps;
  kv.n_kv_heads = (int32_t)heads;
  kv.head_dim = (int32_t)hd;
  kv.dtype = dt;
  kv.n_seqs = (int32_t)seqs;
  kv.table_width = (int32_t)width;
  return kv;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError();
  return v;
}
// A whole number, cut to what 32 bits hold.
int64_t whole(PyObject* o) {
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &over);
  if (v == -1 && PyErr_Occurred()) throw PythonError();
  const long long top = 0x7FFFFFFF;
  return over ? (over > 0 ? top : -top) : v > top ? top : v < -top ? -top : v;
}
// 0: no window.
void window_of(const char* where, PyObject* window, PyObject* sinks, int32_t* w, int32_t* s) {
  const int64_t first = whole(sinks);
  if (window == Py_None) {
    if (first != 0) refuse(where, "sinks go with a window");
    *w = *s = 0;
    return;
  }
  const int64_t last = whole(window);
  if (last < 1 || first < 0) refuse(where, "window must be at least 1, sinks at least 0");
  *w = (int32_t)last;
  *s = (int32_t)first;
}
float scale_of(PyObject* scale, int64_t hd) { return scale == Py_None ? (float)std::pow((double)hd, -0.5) : (float)number(scale); }

// The result: the tensor that was given, or a new one like q.
struct Out {
  PyObject* given;
  Tensor made;
  void* p;
  int64_t stride;
  Out(const char* where, PyObject* o, const Tensor& q, int device) : given(o) {
    const int64_t n = q.size(0), heads = q.size(1), hd = q.size(2);
    if (o == Py_None) {
      made = at::empty(q.sizes(), q.options());
      p = made.data_ptr();
      stride = heads * hd;
    } else {
      const Tensor& t = tensor(where, "out", o);
      stride = rows(where, "out", t, n, heads, hd, q.scalar_type(), device);
      p = t.data_ptr();
    }
  }
  PyObject* result() { return given == Py_None ? THPVariable_Wrap(made) : Py_NewRef(given); }
};
struct Workspace {
  Tensor held;
  void* p = nullptr;
  uint64_t bytes = 0;
  template <class Ask>
  Workspace(const char* where, PyObject* o, const Tensor& like, int device, Ask ask) {
    if (o != Py_None) {
      held = tensor(where, "workspace", o);
      if (held.scalar_type() != at::kByte || !held.is_contiguous() || cuda_index(held) != device)
        refuse(where, "workspace must be a contiguous uint8 tensor on the tensors' device");
      p = held.data_ptr();
      bytes = (uint64_t)held.numel();
      return;
    }
    ask(&bytes);
    if (bytes == 0) return;
    held = at::empty({(int64_t)bytes}, like.options().dtype(at::kByte));
    p = held.data_ptr();
  }
};
// The library's call, without the interpreter's lock: a launch may wait for room in its stream's queue.
template <class Call>
void launch(const char* name, Call call) {
  PyThreadState* const state = PyEval_SaveThread();
  const int rc = call();
  PyEval_RestoreThread(state);
  check(rc, name);
}
void* stream_of(int device) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }

// k_pages, v_pages, table, lens, cu_rows, q, k, v, cos, sin, q_gain, k_gain, eps, k_scale, v_scale, out, status
PyObject* append(PyObject* const* o) {
  const char* where = "paged_kv_append";
  int d;
  const adp_paged_kv kv = paged(where, o, o[13], o[14], &d);
  const int32_t* cu = indices(where, "cu_rows", tensor(where, "cu_rows", o[4]), (int64_t)kv.n_seqs + 1, d);
  const Tensor &k = tensor(where, "k", o[6]), &v = tensor(where, "v", o[7]);
  const auto type = k.scalar_type();
  const int dt = rows_type(type);
  if (dt < 0 || k.dim() != 3) refuse(where, "k and v rows must be [rows, kv_heads, head_dim] of f16, bf16 or f32");
  const int64_t n = k.size(0), hd = kv.head_dim;
  if (n > 0x7FFFFFFF) refuse(where, "a size is beyond 32 bits");
  const int64_t ks = rows(where, "k", k, n, kv.n_kv_heads, hd, type, d), vs = rows(where, "v", v, n, kv.n_kv_heads, hd, type, d);
  const auto q = maybe(where, "q", o[5]);
  const void* qp = nullptr;
  void* op = nullptr;
  int64_t heads = 0, qs = 0, os = 0;
  int odt = 0;
  Tensor made;
  if (q) {
    if (q->dim() != 3 || q->size(1) < 1 || q->size(1) > 0x7FFFFFFF) refuse(where, "q must be [rows, heads, head_dim]");
    heads = q->size(1);
    qs = rows(where, "q", *q, n, heads, hd, type, d);
    qp = q->data_ptr();
    if (o[15] == Py_None) {
      made = at::empty(q->sizes(), q->options());
      op = made.data_ptr();
      os = heads * hd;
      odt = dt;
    } else {
      const Tensor& out = tensor(where, "out", o[15]);
      odt = rows_type(out.scalar_type());
      if (odt < 0) refuse(where, "out must be of f16, bf16 or f32");
      os = rows(where, "out", out, n, heads, hd, out.scalar_type(), d);
      op = out.data_ptr();
    }
  } else if (o[15] != Py_None) {
    refuse(where, "out goes with q");
  }
  const Tensor &cos = tensor(where, "cos", o[8]), &sin = tensor(where, "sin", o[9]);
  if (cos.scalar_type() != at::kFloat || sin.scalar_type() != at::kFloat || cos.dim() != 2 || sin.sizes() != cos.sizes() || !cos.is_contiguous() ||
      !sin.is_contiguous() || cuda_index(cos) != d || cuda_index(sin) != d || cos.size(0) > 0x7FFFFFFF || cos.size(1) > 0x3FFFFFFF)
    refuse(where, "cos and sin must be alike: contiguous fp32 [positions, rotated / 2]" + on(d));
  adp_rope rope{};
  std::optional<at::ScalarType> gain_type;
  for (int i = 0; i < 2; ++i) {
    if (o[10 + i] == Py_None) continue;
    const Tensor& g = tensor(where, i ? "k_gain" : "q_gain", o[10 + i]);
    rope.gain_dtype = rows_type(g.scalar_type());
    if (rope.gain_dtype < 0 || g.dim() != 1 || g.size(0) != hd || !g.is_contiguous() || cuda_index(g) != d)
      refuse(where, "q_gain and k_gain must be contiguous [" + std::to_string(hd) + "] of f16, bf16 or f32" + on(d));
    if (gain_type && *gain_type != g.scalar_type()) refuse(where, "q_gain and k_gain must be of one type");
    gain_type = g.scalar_type();
    (i ? rope.k_gain : rope.q_gain) = g.data_ptr();
  }
  rope.cos = static_cast<const float*>(cos.data_ptr());
  rope.sin = static_cast<const float*>(sin.data_ptr());
  rope.n_positions = (int32_t)cos.size(0);
  rope.rotated = (int32_t)(2 * cos.size(1));
  rope.eps = (float)number(o[12]);
  int32_t* status = status_of(where, o[16], d);
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)d);
  const void *kp = k.data_ptr(), *vp = v.data_ptr();
  void* const stream = stream_of(d);
  launch("adp_paged_kv_append", [&] {
    return lib.append(&kv, &rope, qp, kp, vp, dt, (int32_t)heads, qs, ks, vs, cu, (int32_t)n, op, odt, os, status, stream);
  });
  if (!q) Py_RETURN_NONE;
  return o[15] == Py_None ? THPVariable_Wrap(made) : Py_NewRef(o[15]);
}

// k_pages, v_pages, table, lens, q, window, sinks, scale, k_scale, v_scale, out, workspace, status
PyObject* attention(PyObject* const* o) {
  const char* where = "paged_attention";
  int d;
  int32_t window, sinks;
  window_of(where, o[5], o[6], &window, &sinks);
  const adp_paged_kv kv = paged(where, o, o[8], o[9], &d);
  const Tensor& q = tensor(where, "q", o[4]);
  const int dt = half_type(q.scalar_type());
  if (dt < 0 || q.dim() != 3 || q.size(0) != kv.n_seqs || q.size(2) != kv.head_dim || q.size(2) < 1 || q.size(1) > 0x7FFFFFFF)
    refuse(where, "q must be [seqs, heads, head_dim] of f16 or bf16");
  const int64_t heads = q.size(1), hd = q.size(2), qs = rows(where, "q", q, q.size(0), heads, hd, q.scalar_type(), d);
  Out out(where, o[10], q, d);
  const float scale = scale_of(o[7], hd);
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)d);
  const void* const qp = q.data_ptr();
  void* const stream = stream_of(d);
  if (window) {
    Workspace w(where, o[11], q, d, [&](uint64_t* b) {
      check(lib.window_workspace(&kv, (int32_t)heads, window, sinks, b), "adp_paged_window_attention_workspace");
    });
    int32_t* status = status_of(where, o[12], d);
    launch("adp_paged_window_attention", [&] {
      return lib.window(&kv, qp, dt, (int32_t)heads, qs, scale, window, sinks, out.p, out.stride, w.p, w.bytes, status, stream);
    });
  } else {
    Workspace w(where, o[11], q, d,
                [&](uint64_t* b) { check(lib.attention_workspace(&kv, (int32_t)heads, b), "adp_paged_attention_workspace"); });
    int32_t* status = status_of(where, o[12], d);
    launch("adp_paged_attention", [&] {
      return lib.attention(&kv, qp, dt, (int32_t)heads, qs, scale, out.p, out.stride, w.p, w.bytes, status, stream);
    });
  }
  return out.result();
}

// k_pages, v_pages, table, lens, q, cu_rows, window, sinks, scale, k_scale, v_scale, out, workspace, status
PyObject* chunk(PyObject* const* o) {
  const char* where = "paged_chunk_attention";
  int d;
  int32_t window, sinks;
  window_of(where, o[6], o[7], &window, &sinks);
  const adp_paged_kv kv = paged(where, o, o[9], o[10], &d);
  const Tensor& q = tensor(where, "q", o[4]);
  const int dt = half_type(q.scalar_type());
  if (dt < 0 || q.dim() != 3 || q.size(2) != kv.head_dim || q.size(2) < 1 || q.size(0) > 0x7FFFFFFF || q.size(1) > 0x7FFFFFFF)
    refuse(where, "q must be [rows, heads, head_dim] of f16 or bf16");
  const int64_t n = q.size(0), heads = q.size(1), hd = q.size(2), qs = rows(where, "q", q, n, heads, hd, q.scalar_type(), d);
  const int32_t* cu = indices(where, "cu_rows", tensor(where, "cu_rows", o[5]), (int64_t)kv.n_seqs + 1, d);
  Out out(where, o[11], q, d);
  const float scale = scale_of(o[8], hd);
  const c10::cuda::CUDAGuard guard((c10::DeviceIndex)d);
  Workspace w(where, o[12], q, d, [&](uint64_t* b) {
    check(lib.chunk_workspace(&kv, (int32_t)heads, (int32_t)n, window, sinks, b), "adp_paged_chunk_attention_workspace");
  });
  int32_t* status = status_of(where, o[13], d);
  const void* const qp = q.data_ptr();
  void* const stream = stream_of(d);
  launch("adp_paged_chunk_attention", [&] {
    return lib.chunk(&kv, qp, dt, (int32_t)heads, qs, cu, (int32_t)n, scale, window, sinks, out.p, out.stride, w.p, w.bytes, status, stream);
  });
  return out.result();
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N || !error_type) {
    PyErr_SetString(PyExc_TypeError, error_type ? "wrong number of arguments" : "the binding has not been set up");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& r) {
    PyObject* e = PyObject_CallFunction(error_type, "is", r.code, r.where.c_str());
    if (e) {
      PyErr_SetObject(error_type, e);
      Py_DECREF(e);
    }
  } catch (const PythonError&) {
  } catch (...) {  // PyTorch's own errors keep their types (OutOfMemoryError among them)
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// setup(exception type, the seven addresses)
PyObject* setup(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "setup(exception, 7 addresses)");
    return nullptr;
  }
  void* p[7];
  for (int i = 0; i < 7; ++i) {
    p[i] = PyLong_AsVoidPtr(args[1 + i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is 0");
      return nullptr;
    }
  }
  lib.append = reinterpret_cast<decltype(lib.append)>(p[0]);
  lib.attention = reinterpret_cast<decltype(lib.attention)>(p[1]);
  lib.attention_workspace = reinterpret_cast<decltype(lib.attention_workspace)>(p[2]);
  lib.window = reinterpret_cast<decltype(lib.window)>(p[3]);
  lib.window_workspace = reinterpret_cast<decltype(lib.window_workspace)>(p[4]);
  lib.chunk = reinterpret_cast<decltype(lib.chunk)>(p[5]);
  lib.chunk_workspace = reinterpret_cast<decltype(lib.chunk_workspace)>(p[6]);
  Py_XDECREF(error_type);
  error_type = Py_NewRef(args[0]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void (*)())setup, METH_FASTCALL, nullptr},
    {"paged_kv_append", (PyCFunction)(void (*)())guarded<append, 17>, METH_FASTCALL, nullptr},
    {"paged_attention", (PyCFunction)(void (*)())guarded<attention, 13>, METH_FASTCALL, nullptr},
    {"paged_chunk_attention", (PyCFunction)(void (*)())guarded<chunk, 14>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", ADP_TORCH_VERSION) != 0) Py_CLEAR(m);  // (the package compares it)
  return m;
}
