// CPython module _bind: the tensors' checks and addresses for the calls of
// include/moe_experts.h. A call of these operators lasts a few microseconds; checked and
// converted in Python, its seven to nine tensors took as long again and more.
// Computes nothing and keeps nothing but the entries' addresses, which moe.py hands over
// from the library that it has loaded.
#include <Python.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/moe_experts.h"

namespace {

decltype(&moe_route) route_entry;
decltype(&moe_route_backward) route_backward_entry;
decltype(&moe_mx_quantize) mx_quantize_entry;
decltype(&moe_expert_product) expert_product_entry;
decltype(&moe_int8_quantize) int8_quantize_entry;
decltype(&moe_expert_product_int8) expert_product_int8_entry;
decltype(&moe_combine_backward) combine_backward_entry;
decltype(&moe_dispatch_backward) dispatch_backward_entry;

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(const char* what, const char* why) {
  PyErr_Format(PyExc_ValueError, "%s: %s", what, why);
  throw Refused{};
}

// A ctypes structure's address, by the buffer protocol; released with the object.
template <typename T>
struct Config {
  Py_buffer view;
  explicit Config(PyObject* o) {
    if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE) != 0) throw Refused{};
    if (view.len != (Py_ssize_t)sizeof(T)) {
      PyBuffer_Release(&view);
      refuse("configuration", "not of this call's type");
    }
  }
  ~Config() { PyBuffer_Release(&view); }
  Config(const Config&) = delete;
  Config& operator=(const Config&) = delete;
  const T* get() const { return static_cast<const T*>(view.buf); }
};

const at::Tensor& tensor_of(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(what, "expected a tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse(what, "expected a CUDA tensor");
  return t;
}

// n contiguous elements of a type; None is no address.
void* typed(PyObject* o, at::ScalarType dtype, int64_t n, const char* what) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor_of(o, what);
  if (t.scalar_type() != dtype || t.numel() != n || !t.is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "%s: expected %lld contiguous elements of %s", what, (long long)n, c10::toString(dtype));
    throw Refused{};
  }
  return t.data_ptr();
}

// `rows` contiguous rows of `cols` elements, `stride` apart.
void* rows_of(PyObject* o, int dtype, int64_t rows, int64_t cols, int64_t stride, const char* what) {
  const at::Tensor& t = tensor_of(o, what);
  const at::ScalarType want = dtype == MOE_F32 ? at::kFloat : dtype == MOE_F16 ? at::kHalf : at::kBFloat16;
  const bool apart = t.is_contiguous() ? stride == cols || rows < 2
                                       : t.dim() == 2 && t.stride(1) == 1 && (t.stride(0) == stride || rows < 2);
  if (!apart || t.scalar_type() != want || t.numel() != rows * cols || (t.dim() ? t.size(-1) : 0) != cols) {
    PyErr_Format(PyExc_ValueError, "%s: expected %lld contiguous rows of %lld elements of %s, %lld apart", what,
                 (long long)rows, (long long)cols, c10::toString(want), (long long)stride);
    throw Refused{};
  }
  return t.data_ptr();
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}
int32_t integer32(PyObject* o, const char* what) {
  const int64_t v = integer(o);
  if (v != (int32_t)v) refuse(what, "beyond 32 bits");
  return (int32_t)v;
}
void* address(PyObject* o) {
  const unsigned long long v = PyLong_AsUnsignedLongLong(o);
  if (v == (unsigned long long)-1 && PyErr_Occurred()) throw Refused{};
  return reinterpret_cast<void*>(v);
}
// None is the current device's current stream; else a handle, or an object that has one as cuda_stream.
void* stream_of(PyObject* o) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
  if (PyLong_Check(o)) return address(o);
  PyObject* handle = PyObject_GetAttrString(o, "cuda_stream");
  if (!handle) throw Refused{};
  const unsigned long long v = PyLong_AsUnsignedLongLong(handle);
  Py_DECREF(handle);
  if (v == (unsigned long long)-1 && PyErr_Occurred()) throw Refused{};
  return reinterpret_cast<void*>(v);
}

// The entry, called without the interpreter's lock: its status as an int.
template <typename F, typename... Args>
PyObject* enqueue(F entry, Args... args) {
  if (!entry) refuse("_bind", "no library loaded");
  moe_status_t status;
  Py_BEGIN_ALLOW_THREADS
  status = entry(args...);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

template <int N, PyObject* (*F)(PyObject* const*)>
PyObject* method(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) return PyErr_Format(PyExc_TypeError, "expected %d arguments", N);
  try {
    return F(a);
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {  // a tensor without storage, ..
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
}

PyObject* entries(PyObject* const* a) {
  route_entry = reinterpret_cast<decltype(route_entry)>(address(a[0]));
  route_backward_entry = reinterpret_cast<decltype(route_backward_entry)>(address(a[1]));
  mx_quantize_entry = reinterpret_cast<decltype(mx_quantize_entry)>(address(a[2]));
  expert_product_entry = reinterpret_cast<decltype(expert_product_entry)>(address(a[3]));
  int8_quantize_entry = reinterpret_cast<decltype(int8_quantize_entry)>(address(a[4]));
  expert_product_int8_entry = reinterpret_cast<decltype(expert_product_int8_entry)>(address(a[5]));
  combine_backward_entry = reinterpret_cast<decltype(combine_backward_entry)>(address(a[6]));
  dispatch_backward_entry = reinterpret_cast<decltype(dispatch_backward_entry)>(address(a[7]));
  Py_RETURN_NONE;
}

// rc, logits, bias, expert_ids, expert_scales, stream
PyObject* route(PyObject* const* a) {
  const Config<moe_router_config_t> rc(a[0]);
  const moe_router_config_t* c = rc.get();
  const int64_t picks = (int64_t)c->tokens * c->topk;
  void* logits = rows_of(a[1], c->logits_dtype, c->tokens, c->expert_num, c->logits_stride, "logits");
  void* bias = typed(a[2], at::kFloat, c->expert_num, "bias");
  void* ids = typed(a[3], at::kInt, picks, "expert_ids");
  void* weights = typed(a[4], at::kFloat, picks, "expert_scales");
  return enqueue(route_entry, c, logits, static_cast<const float*>(bias), static_cast<int32_t*>(ids),
                 static_cast<float*>(weights), stream_of(a[5]));
}

// rc, logits, expert_ids, grad_scales, grad_logits, stream
PyObject* route_backward(PyObject* const* a) {
  const Config<moe_router_config_t> rc(a[0]);
  const moe_router_config_t* c = rc.get();
  const int64_t picks = (int64_t)c->tokens * c->topk;
  void* logits = rows_of(a[1], c->logits_dtype, c->tokens, c->expert_num, c->logits_stride, "logits");
  void* ids = typed(a[2], at::kInt, picks, "expert_ids");
  void* grad = typed(a[3], at::kFloat, picks, "grad_scales");
  const at::Tensor& g = tensor_of(a[4], "grad_logits");
  const int64_t stride = g.is_contiguous() || c->tokens < 2 || g.dim() < 1 ? c->expert_num : g.stride(0);
  void* out = rows_of(a[4], c->logits_dtype, c->tokens, c->expert_num, stride, "grad_logits");
  return enqueue(route_backward_entry, c, logits, static_cast<const int32_t*>(ids), static_cast<const float*>(grad), out,
                 stride, stream_of(a[5]));
}

// The element type of a quantiser's input, and its matrices, rows and columns.
struct Matrices {
  int dtype;
  int64_t mats, rows, cols, row_stride, mat_stride;
  const void* data;
  explicit Matrices(PyObject* o) {
    const at::Tensor& x = tensor_of(o, "x");
    dtype = x.scalar_type() == at::kFloat      ? (int)MOE_F32
            : x.scalar_type() == at::kHalf     ? (int)MOE_F16
            : x.scalar_type() == at::kBFloat16 ? (int)MOE_BF16
                                               : -1;
    if (x.dim() < 2 || x.dim() > 3 || dtype < 0)
      refuse("x", "expected a 2D or 3D CUDA tensor of float32, float16 or bfloat16");
    rows = x.size(-2), cols = x.size(-1), mats = x.dim() == 3 ? x.size(0) : 1;
    if (cols > 1 && x.stride(-1) != 1) refuse("x", "expected contiguous rows");
    if (cols != (int32_t)cols || mats != (int32_t)mats) refuse("x", "sizes beyond 32 bits");
    row_stride = rows > 1 ? x.stride(-2) : cols;
    mat_stride = x.dim() == 3 ? x.stride(0) : 0;
    data = x.data_ptr();
  }
};

// x, codes, scales, layout, stream
PyObject* mx_quantize(PyObject* const* a) {
  const Matrices x(a[0]);
  const int32_t layout = integer32(a[3], "layout");
  const int64_t blocks = (x.cols + 31) / 32;
  void* codes = typed(a[1], at::kByte, x.mats * x.rows * (x.cols / 2), "codes");
  void* scales = typed(a[2], at::kByte,
                       layout == MOE_SF_ROWS ? x.mats * x.rows * blocks : x.mats * ((x.rows + 127) / 128) * ((blocks + 3) / 4) * 512,
                       "scales");
  return enqueue(mx_quantize_entry, x.data, x.dtype, (int32_t)x.mats, x.rows, (int32_t)x.cols, x.row_stride, x.mat_stride,
                 layout, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), stream_of(a[4]));
}

// x, codes, scales, ep_recv_count, stream
PyObject* int8_quantize(PyObject* const* a) {
  const Matrices x(a[0]);
  void* codes = typed(a[1], at::kChar, x.mats * x.rows * x.cols, "codes");
  void* scales = typed(a[2], at::kFloat, x.mats * x.rows, "scales");
  void* counts = nullptr;
  int64_t each = 0;
  if (a[3] != Py_None) {
    const int64_t n = tensor_of(a[3], "ep_recv_count").numel();
    if (x.mats < 1 || n < 1 || n % x.mats || n > 0x7fffffff) refuse("ep_recv_count", "expected as many counts for each rank");
    counts = typed(a[3], at::kInt, n, "ep_recv_count");
    each = n / x.mats;
  }
  return enqueue(int8_quantize_entry, x.data, x.dtype, (int32_t)x.mats, x.rows, (int32_t)x.cols, x.row_stride, x.mat_stride,
                 static_cast<const int32_t*>(counts), (int32_t)each, static_cast<int8_t*>(codes), static_cast<float*>(scales),
                 stream_of(a[4]));
}

// Rows that all ranks together have room for, W * A.
int64_t capacity(const moe_config_t* c) {
  const int64_t W = c->ep_world_size;
  if (W < 1) refuse("cfg", "no ranks");
  const int64_t local = c->moe_expert_num / W;
  return W * c->bs * W * (local < c->topk ? local : c->topk);
}

struct Workspace {
  void* data;
  size_t bytes;
  explicit Workspace(PyObject* o) {
    const at::Tensor& ws = tensor_of(o, "ws");
    if (!ws.is_contiguous()) refuse("ws", "expected a contiguous tensor");
    data = ws.data_ptr();
    bytes = (size_t)ws.numel() * ws.element_size();
  }
};

// cfg, x, x_scales, ep_recv_count, w, w_scales, y, y_scales, epilogue, ws, stream
PyObject* expert_product(PyObject* const* a) {
  const Config<moe_config_t> config(a[0]);
  const moe_config_t* c = config.get();
  const int64_t W = c->ep_world_size, E = c->moe_expert_num, rows = capacity(c);
  const at::Tensor& w = tensor_of(a[4], "w");
  if (w.dim() < 2) refuse("w", "expected [experts, n, k / 2]");
  const int64_t n = w.size(-2), k = 2 * w.size(-1);
  if (n != (int32_t)n || k != (int32_t)k) refuse("w", "sizes beyond 32 bits");
  const int32_t epilogue = integer32(a[8], "epilogue");
  const int64_t columns = epilogue == MOE_EPI_SWIGLU ? n / 2 : n;
  const at::ScalarType yt = tensor_of(a[6], "y").scalar_type();
  const int32_t y_dtype = yt == at::kByte       ? (int)MOE_MXFP4
                          : yt == at::kBFloat16 ? (int)MOE_BF16
                          : yt == at::kHalf     ? (int)MOE_F16
                                                : -1;
  void* x = typed(a[1], at::kByte, rows * (k / 2), "x");
  void* x_scales = typed(a[2], at::kByte, rows * (k / 32), "x_scales");
  void* counts = typed(a[3], at::kInt, E * W, "ep_recv_count");
  void* codes = typed(a[4], at::kByte, E * n * (k / 2), "w");
  void* w_scales = typed(a[5], at::kByte, E * ((n + 127) / 128) * ((k + 127) / 128) * 512, "w_scales");
  void* y = typed(a[6], yt, rows * (yt == at::kByte ? columns / 2 : columns), "y");
  void* y_scales = typed(a[7], at::kByte, rows * ((columns + 31) / 32), "y_scales");
  const Workspace ws(a[9]);
  return enqueue(expert_product_entry, c, static_cast<const void*>(x), static_cast<const uint8_t*>(x_scales),
                 static_cast<const int32_t*>(counts), static_cast<const void*>(codes), static_cast<const uint8_t*>(w_scales),
                 (int32_t)n, (int32_t)k, epilogue, y_dtype, y, static_cast<uint8_t*>(y_scales), ws.data, ws.bytes,
                 stream_of(a[10]));
}

// cfg, x, x_scales, ep_recv_count, w, w_scales, y, epilogue, ws, stream
PyObject* expert_product_int8(PyObject* const* a) {
  const Config<moe_config_t> config(a[0]);
  const moe_config_t* c = config.get();
  const int64_t E = c->moe_expert_num, rows = capacity(c);
  const at::Tensor& wt = tensor_of(a[4], "w");
  if (wt.dim() < 2) refuse("w", "expected [experts, n, k]");
  const int64_t n = wt.size(-2), k = wt.size(-1);
  if (n != (int32_t)n || k != (int32_t)k) refuse("w", "sizes beyond 32 bits");
  const int32_t epilogue = integer32(a[7], "epilogue");
  const at::ScalarType yt = tensor_of(a[6], "y").scalar_type();
  const int32_t y_dtype = yt == at::kBFloat16 ? (int)MOE_BF16 : yt == at::kHalf ? (int)MOE_F16 : -1;
  void* x = typed(a[1], at::kChar, rows * k, "x");
  void* x_scales = typed(a[2], at::kFloat, rows, "x_scales");
  void* counts = typed(a[3], at::kInt, E * c->ep_world_size, "ep_recv_count");
  void* w = typed(a[4], at::kChar, E * n * k, "w");
  void* w_scales = typed(a[5], at::kFloat, E * n, "w_scales");
  void* y = typed(a[6], yt, rows * (epilogue == MOE_EPI_SWIGLU ? n / 2 : n), "y");
  const Workspace ws(a[8]);
  return enqueue(expert_product_int8_entry, c, static_cast<const int8_t*>(x), static_cast<const float*>(x_scales),
                 static_cast<const int32_t*>(counts), static_cast<const int8_t*>(w), static_cast<const float*>(w_scales),
                 (int32_t)n, (int32_t)k, epilogue, y_dtype, y, ws.data, ws.bytes, stream_of(a[9]));
}

// The arrays of both gradients: elements of cfg's type, and what the routing left.
struct Gradient {
  const moe_config_t* c;
  int64_t tokens, picks, rows, h;
  at::ScalarType type;
  explicit Gradient(const moe_config_t* c_) : c(c_) {
    rows = capacity(c);
    tokens = (int64_t)c->ep_world_size * c->bs;
    picks = tokens * c->topk;
    h = c->h;
    type = c->x_dtype == MOE_F16 ? at::kHalf : c->x_dtype == MOE_BF16 ? at::kBFloat16 : at::kInt;
  }
  void* token_rows(PyObject* o, const char* what) const { return typed(o, type, tokens * h, what); }
  void* expert_rows(PyObject* o, const char* what) const { return typed(o, type, rows * h, what); }
  int32_t* assist(PyObject* o) const { return static_cast<int32_t*>(typed(o, at::kInt, rows * 3, "assist_info")); }
  int32_t* counts(PyObject* o) const {
    return static_cast<int32_t*>(typed(o, at::kInt, (int64_t)c->moe_expert_num * c->ep_world_size, "ep_recv_count"));
  }
  int32_t* ids(PyObject* o) const { return static_cast<int32_t*>(typed(o, at::kInt, picks, "expert_ids")); }
  float* weights(PyObject* o, const char* what) const { return static_cast<float*>(typed(o, at::kFloat, picks, what)); }
  // bytes or truth values; not looked at where cfg says there is none
  uint8_t* mask(PyObject* o) const {
    if (o == Py_None || c->mask_kind == 0) return nullptr;
    const bool truth = tensor_of(o, "active_mask").scalar_type() == at::kBool;
    return static_cast<uint8_t*>(typed(o, truth ? at::kBool : at::kByte, c->mask_kind == 1 ? tokens : picks, "active_mask"));
  }
};

// cfg, grad_out, expert_out, assist_info, ep_recv_count, expert_ids, expert_scales, active_mask, x, grad_expert_out,
// grad_scales, grad_x, ws, stream
PyObject* combine_backward(PyObject* const* a) {
  const Config<moe_config_t> config(a[0]);
  const Gradient g(config.get());
  void* grad_out = g.token_rows(a[1], "grad_out");
  void* expert_out = g.expert_rows(a[2], "expert_out");
  const int32_t* assist = g.assist(a[3]);
  const int32_t* counts = g.counts(a[4]);
  const int32_t* ids = g.ids(a[5]);
  const float* weights = g.weights(a[6], "expert_scales");
  const uint8_t* mask = g.mask(a[7]);
  void* x = g.token_rows(a[8], "x");
  void* grad_rows = g.expert_rows(a[9], "grad_expert_out");
  float* grad_scales = g.weights(a[10], "grad_scales");
  void* grad_x = g.token_rows(a[11], "grad_x");
  const Workspace ws(a[12]);
  return enqueue(combine_backward_entry, g.c, static_cast<const void*>(grad_out), static_cast<const void*>(expert_out), assist,
                 counts, ids, weights, mask, static_cast<const void*>(x), grad_rows, grad_scales, grad_x, ws.data, ws.bytes,
                 stream_of(a[13]));
}

// cfg, grad_expand_x, assist_info, ep_recv_count, expert_ids, active_mask, grad_x, residual, grad_expand_scales,
// grad_scales, ws, stream
PyObject* dispatch_backward(PyObject* const* a) {
  const Config<moe_config_t> config(a[0]);
  const Gradient g(config.get());
  void* grad_rows = g.expert_rows(a[1], "grad_expand_x");
  const int32_t* assist = g.assist(a[2]);
  const int32_t* counts = g.counts(a[3]);
  const int32_t* ids = g.ids(a[4]);
  const uint8_t* mask = g.mask(a[5]);
  void* grad_x = g.token_rows(a[6], "grad_x");
  void* residual = g.token_rows(a[7], "residual");
  void* row_weights = typed(a[8], at::kFloat, g.rows, "grad_expand_scales");
  float* grad_scales = g.weights(a[9], "grad_scales");
  const Workspace ws(a[10]);
  return enqueue(dispatch_backward_entry, g.c, static_cast<const void*>(grad_rows), assist, counts, ids, mask,
                 static_cast<const void*>(residual), static_cast<const float*>(row_weights), grad_x, grad_scales, ws.data,
                 ws.bytes, stream_of(a[11]));
}

#define BIND(name, count) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&method<count, name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {BIND(entries, 8), BIND(route, 6), BIND(route_backward, 6), BIND(mx_quantize, 5),
                         BIND(expert_product, 11), BIND(int8_quantize, 5), BIND(expert_product_int8, 10),
                         BIND(combine_backward, 14), BIND(dispatch_backward, 12), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", "Calls of include/moe_experts.h on torch tensors.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
