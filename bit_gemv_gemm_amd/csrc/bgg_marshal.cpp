// Argument marshalling of the decoder-layer calls for the Python package:
// checks of the torch tensors, then the C entry points of libbgg.so, whose
// addresses bind() is given.  The same checks written in Python take longer
// than most of the kernels they launch (5 of a call's 8 us; here under 1).
// No arithmetic and no GPU work of its own.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <exception>

#include "../../include/bgg.h"

namespace {

// What a failed check leaves: a Python error is set.
struct Refused {};

[[noreturn]] void refuse(const char* what, const char* why) {
  PyErr_Format(PyExc_ValueError, "%s: %s", what, why);
  throw Refused{};
}

decltype(&bgg_paged_attention) p_attention;
decltype(&bgg_rotary_append) p_rotary;
decltype(&bgg_ternary_gemv_epilogue) p_gemv;
decltype(&bgg_gemv_run_epilogue) p_run;
decltype(&bgg_ternary_gemm_epilogue) p_gemm;

bool is_none(PyObject* o) { return o == Py_None; }

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_ValueError, "%s must be a tensor, not %s", what, Py_TYPE(o)->tp_name);
    throw Refused{};
  }
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}

// The device of a call's tensors: that of its first one.
int device_of(const at::Tensor& t, const char* what) {
  if (!t.is_cuda()) refuse(what, "must be a device tensor");
  return t.get_device();
}

// Contiguous, of `type`, on `dev`, at least n values (None: nullptr).
void* vector(PyObject* o, int64_t n, at::ScalarType type, int dev, const char* what) {
  if (is_none(o)) return nullptr;
  const at::Tensor& t = tensor(o, what);
  if (!t.is_cuda() || t.get_device() != dev) refuse(what, "must be on the device of the call's other tensors");
  if (t.scalar_type() != type) refuse(what, "has the wrong type");
  if (!t.is_contiguous()) refuse(what, "must be contiguous");
  if (t.numel() < n) refuse(what, "is too small");
  return t.data_ptr();
}

// A buffer of at least `bytes` bytes, contiguous, on `dev`.
void* bytes(PyObject* o, uint64_t n, int dev, const char* what, uint64_t* size = nullptr) {
  const at::Tensor& t = tensor(o, what);
  if (!t.is_cuda() || t.get_device() != dev) refuse(what, "must be on the device of the call's other tensors");
  if (!t.is_contiguous()) refuse(what, "must be contiguous");
  const uint64_t have = (uint64_t)t.numel() * t.element_size();
  if (have < n) refuse(what, "is too small");
  if (size) *size = have;
  return t.data_ptr();
}

struct Rows {
  void* data = nullptr;
  int64_t stride = 0, heads = 0;
};
// [rows, heads * dim] or [rows, heads, dim], the values of a row side by side.
Rows rows(PyObject* o, int64_t n, int64_t dim, at::ScalarType type, int dev, const char* what) {
  if (dim < 1) refuse("cache", "describes no valid cache");  // (a descriptor nobody filled; the library checks the rest)
  const at::Tensor& t = tensor(o, what);
  if (!t.is_cuda() || t.get_device() != dev) refuse(what, "must be on the device of the call's other tensors");
  if (t.scalar_type() != type) refuse(what, "has the wrong type");
  const int64_t d = t.dim();
  if ((d != 2 && d != 3) || t.size(0) != n) refuse(what, "must be [tokens, heads * head_dim] or [tokens, heads, head_dim]");
  int64_t width = t.size(1);
  bool side_by_side = t.stride(d - 1) == 1;
  if (d == 3) {
    if (t.size(2) != dim) refuse(what, "has the wrong head dimension");
    side_by_side = side_by_side && (t.size(1) == 1 || t.stride(1) == dim);
    width *= dim;
  }
  if (width % dim) refuse(what, "must have whole heads");
  if (!side_by_side) refuse(what, "must have contiguous rows");
  Rows r;
  r.data = t.data_ptr();
  r.stride = n > 1 ? t.stride(0) : width;
  r.heads = width / dim;
  return r;
}

at::ScalarType torch_type(int32_t type) {
  return type == BGG_TYPE_F16 ? at::kHalf : type == BGG_TYPE_BF16 ? at::kBFloat16 : at::kFloat8_e4m3fn;
}
int32_t type_of(const at::Tensor& t, const char* what) {
  if (t.scalar_type() == at::kHalf) return BGG_TYPE_F16;
  if (t.scalar_type() == at::kBFloat16) return BGG_TYPE_BF16;
  refuse(what, "must be float16 or bfloat16");
}

// The C struct inside a ctypes.Structure.
template <class S>
struct Struct {
  Py_buffer view{};
  Struct(PyObject* o, const char* what) {
    if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE)) throw Refused{};
    if (view.len != (Py_ssize_t)sizeof(S)) {
      PyBuffer_Release(&view);
      refuse(what, "is not a descriptor of this call");
    }
  }
  ~Struct() { PyBuffer_Release(&view); }
  const S* operator->() const { return (const S*)view.buf; }
  const S* get() const { return (const S*)view.buf; }
};
using Cache = Struct<bgg_cache_desc>;
using Weights = Struct<bgg_weights_desc>;

template <class F>
PyObject* status_of(F call) {
  bgg_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = call();
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong((long)st);
}

// Every entry: nothing thrown leaves it.
template <class F>
PyObject* guarded(const char* name, Py_ssize_t given, Py_ssize_t wanted, F body) {
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, not %zd", name, wanted, given);
    return nullptr;
  }
  try {
    return body();
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

void cache_buffers(const Cache& c, PyObject* k, PyObject* v, int dev, void** kp, void** vp) {
  const at::ScalarType t = torch_type(c->type);
  const int64_t n = (int64_t)(c->total_bytes / (c->type == BGG_TYPE_E4M3 ? 1 : 2));
  *kp = vector(k, n, t, dev, "k_cache");
  *vp = vector(v, n, t, dev, "v_cache");
}

// (cache, k_cache, v_cache, page_table, lengths, q, out, workspace, scale, window, lse, k_scale, v_scale, stream)
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("paged_attention", n, 14, [&]() -> PyObject* {
    Cache c(a[0], "cache");
    const at::Tensor& q = tensor(a[5], "q");
    const int dev = device_of(q, "q");
    bgg_attention_args g{};
    g.type = type_of(q, "q");
    g.batch = q.dim() ? q.size(0) : 0;
    const Rows rq = rows(a[5], g.batch, c->head_dim, q.scalar_type(), dev, "q");
    const Rows ro = rows(a[6], g.batch, c->head_dim, q.scalar_type(), dev, "out");
    if (ro.heads != rq.heads) refuse("out", "must have q's heads");
    g.q_heads = rq.heads;
    g.q_dev = rq.data, g.q_stride = rq.stride;
    g.out_dev = ro.data, g.out_stride = ro.stride;
    void *kc, *vc;
    cache_buffers(c, a[1], a[2], dev, &kc, &vc);
    g.k_cache_dev = kc, g.v_cache_dev = vc;
    const at::Tensor& t = tensor(a[3], "page_table");
    if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != at::kInt || t.dim() != 2 ||
        t.size(0) != g.batch || (t.size(1) > 1 && t.stride(1) != 1))
      refuse("page_table", "must be int32 [batch, pages] with contiguous rows on q's device");
    g.page_table_dev = (const int32_t*)t.data_ptr();
    g.table_width = t.size(1);
    g.table_stride = g.batch > 1 ? t.stride(0) : t.size(1);
    g.lengths_dev = (const int32_t*)vector(a[4], g.batch, at::kInt, dev, "lengths");
    uint64_t size;
    g.workspace = bytes(a[7], 0, dev, "workspace", &size);
    g.workspace_bytes = size;
    g.scale = (float)number(a[8]);
    g.window = integer(a[9]);
    g.lse_dev = (float*)vector(a[10], g.batch * g.q_heads, at::kFloat, dev, "lse");
    g.k_scale_dev = (const float*)vector(a[11], c->kv_heads, at::kFloat, dev, "k_scale");
    g.v_scale_dev = (const float*)vector(a[12], c->kv_heads, at::kFloat, dev, "v_scale");
    if (g.batch == 0) return PyLong_FromLong(0);  // (empty tensors have no pointers)
    void* stream = (void*)(uintptr_t)integer(a[13]);
    return status_of([&] { return p_attention(c.get(), &g, stream); });
  });
}

// (cache, k_cache, v_cache, positions, slots, freqs, q, q_out, k, v, layout, magnitude, k_scale, v_scale, stream)
PyObject* rotary_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("rotary_append", n, 15, [&]() -> PyObject* {
    Cache c(a[0], "cache");
    const at::Tensor& pos = tensor(a[3], "positions");
    const int dev = device_of(pos, "positions");
    const int64_t T = pos.numel(), D = c->head_dim;
    const bool with_q = !is_none(a[6]), with_k = !is_none(a[8]);
    if (!with_q && !with_k) refuse("q and k", "one of them is needed");
    if (with_k != !is_none(a[9])) refuse("k and v", "come together");
    const at::Tensor& ref = tensor(a[with_q ? 6 : 8], with_q ? "q" : "k");
    bgg_rotary_args g{};
    g.type = type_of(ref, with_q ? "q" : "k");
    const at::ScalarType st = ref.scalar_type();
    if (with_q) {
      const Rows rq = rows(a[6], T, D, st, dev, "q"), ro = rows(a[7], T, D, st, dev, "q_out");
      if (ro.heads != rq.heads) refuse("q_out", "must have q's heads");
      g.q_dev = rq.data, g.q_stride = rq.stride, g.q_heads = rq.heads;
      g.q_out_dev = ro.data, g.q_out_stride = ro.stride;
    }
    if (with_k) {
      const Rows rk = rows(a[8], T, D, st, dev, "k"), rv = rows(a[9], T, D, st, dev, "v");
      if (rk.heads != c->kv_heads || rv.heads != c->kv_heads) refuse("k and v", "must have the cache's heads");
      g.k_dev = rk.data, g.k_stride = rk.stride;
      g.v_dev = rv.data, g.v_stride = rv.stride;
      cache_buffers(c, a[1], a[2], dev, &g.k_cache_dev, &g.v_cache_dev);
      g.slots_dev = (const int64_t*)vector(a[4], T, at::kLong, dev, "slots");
    }
    g.layout = (int32_t)integer(a[10]);
    g.positions_dev = (const int32_t*)vector(a[3], T, at::kInt, dev, "positions");
    g.freqs_dev = (const float*)vector(a[5], 1, at::kFloat, dev, "freqs");
    g.rotary_dim = 2 * tensor(a[5], "freqs").numel();
    g.tokens = T;
    g.magnitude = (float)number(a[11]);
    g.k_scale_dev = (const float*)vector(a[12], c->kv_heads, at::kFloat, dev, "k_scale");
    g.v_scale_dev = (const float*)vector(a[13], c->kv_heads, at::kFloat, dev, "v_scale");
    if (T == 0) return PyLong_FromLong(0);  // (empty tensors have no pointers)
    void* stream = (void*)(uintptr_t)integer(a[14]);
    return status_of([&] { return p_rotary(c.get(), &g, stream); });
  });
}

// float16 [M, N], rows of any stride (None: nullptr, 0)
const void* operand(PyObject* o, int64_t M, int64_t N, int dev, const char* what, int64_t* stride) {
  *stride = 0;
  if (is_none(o)) return nullptr;
  const at::Tensor& t = tensor(o, what);
  if (!t.is_cuda() || t.get_device() != dev) refuse(what, "must be on the device of the call's other tensors");
  if (t.scalar_type() != at::kHalf || t.dim() != 2 || t.size(0) != M || t.size(1) != N || (N > 1 && t.stride(1) != 1))
    refuse(what, "must be float16 [M, N] with contiguous rows");
  *stride = M > 1 ? t.stride(0) : N;
  return t.data_ptr();
}

void* halves(PyObject* o, int64_t n, int dev, const char* what) {
  const at::Tensor& t = tensor(o, what);
  if (t.scalar_type() != at::kHalf) refuse(what, "must be float16");
  return bytes(o, (uint64_t)n * 2, dev, what);
}

// (which, desc, packed, x, y, M, flags, workspace, activation, bias, mul, residual, stream); which: 0 gemv, 1 run, 2 gemm
PyObject* product(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("product", n, 13, [&]() -> PyObject* {
    const int64_t which = integer(a[0]);
    Weights d(a[1], "desc");
    const int dev = device_of(tensor(a[4], "y"), "y");
    const int64_t M = integer(a[5]), N = d->N;
    const uint32_t flags = (uint32_t)integer(a[6]);
    if (M < 0 || M > (int64_t(1) << 31)) refuse("M", "is out of range");  // (M times a matrix size stays in 64 bits)
    const void* packed = bytes(a[2], d->total_bytes, dev, "packed");
    const void* x = which == 1 ? nullptr : halves(a[3], M * d->K, dev, "x");
    void* y = halves(a[4], M * N, dev, "y");
    uint64_t size = 0;
    void* ws = is_none(a[7]) ? nullptr : bytes(a[7], 0, dev, "workspace", &size);
    bgg_epilogue e{};
    e.activation = (int32_t)integer(a[8]);
    e.bias_dev = vector(a[9], N, at::kHalf, dev, "bias");
    e.mul_dev = operand(a[10], M, N, dev, "mul", &e.mul_stride);
    e.residual_dev = operand(a[11], M, N, dev, "residual", &e.residual_stride);
    void* stream = (void*)(uintptr_t)integer(a[12]);
    if (which == 0) return status_of([&] { return p_gemv(d.get(), packed, x, y, M, flags, &e, ws, size, stream); });
    if (which == 1) return status_of([&] { return p_run(d.get(), packed, y, M, &e, ws, size, stream); });
    return status_of([&] { return p_gemm(d.get(), packed, x, y, M, flags, &e, ws, size, stream); });
  });
}

// The addresses of bgg_paged_attention, bgg_rotary_append, bgg_ternary_gemv_epilogue,
// bgg_gemv_run_epilogue and bgg_ternary_gemm_epilogue.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("bind", n, 5, [&]() -> PyObject* {
    void* p[5];
    for (int i = 0; i < 5; ++i) p[i] = (void*)(uintptr_t)integer(a[i]);
    p_attention = (decltype(p_attention))p[0];
    p_rotary = (decltype(p_rotary))p[1];
    p_gemv = (decltype(p_gemv))p[2];
    p_run = (decltype(p_run))p[3];
    p_gemm = (decltype(p_gemm))p[4];
    Py_RETURN_NONE;
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction entry() {
  return (PyCFunction)(void (*)(void))F;
}
PyMethodDef methods[] = {{"bind", entry<bind>(), METH_FASTCALL, nullptr},
                         {"paged_attention", entry<paged_attention>(), METH_FASTCALL, nullptr},
                         {"rotary_append", entry<rotary_append>(), METH_FASTCALL, nullptr},
                         {"product", entry<product>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
  PyObject* m = PyModule_Create(&module);
  // the torch whose tensors this code can read
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION)) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
