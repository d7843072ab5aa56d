// binding.cpp — the attention-layer calls of tgdn.h for PyTorch tensors (module _calls).
//
// A decode step makes several of these calls per layer, and a call's kernels take 3-15 us;
// reading the tensors' types, shapes and addresses here instead of in Python takes ~0.5 us of
// host time per call instead of ~6 (rotation of 33 rows: 2.8 us a call after 9.6).  Every
// tensor is checked, so that no host pointer, no other device's and no wrong layout reaches a
// kernel; what is wrong is raised as TypeError or ValueError with the argument's name.  Each
// function returns the call's tgdn_status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <exception>

#include "tgdn.h"

namespace {

struct Raised {};  // a Python error is set

[[noreturn]] void raise(PyObject* type, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw Raised();
}

const char* name_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kHalf: return "torch.float16";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kByte: return "torch.uint8";
    default: return c10::toString(t);
  }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s: expected a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

// The current device, looked up once per call (under the interpreter's lock); 0 without any.
int g_device = -1;
int current_device() {
  if (g_device < 0) {
    c10::DeviceIndex d = 0;
    g_device = c10::cuda::GetDevice(&d) == cudaSuccess ? d : 0;
  }
  return g_device;
}

const at::Tensor& on_device(PyObject* o, at::ScalarType type, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda())
    raise(PyExc_ValueError, "%s: must be a CUDA tensor (the library takes device pointers)", name);
  if (t.get_device() != current_device())
    raise(PyExc_ValueError, "%s: on cuda:%d, the current device is cuda:%d (where the call runs)", name,
          (int)t.get_device(), current_device());
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, "%s: dtype %s, expected %s", name, name_of(t.scalar_type()), name_of(type));
  return t;
}

// Device pointer of a contiguous tensor of at least `numel` elements.
void* array(PyObject* o, at::ScalarType type, int64_t numel, const char* name) {
  const at::Tensor& t = on_device(o, type, name);
  if (!t.is_contiguous()) raise(PyExc_ValueError, "%s: must be contiguous", name);
  if (t.numel() < numel)
    raise(PyExc_ValueError, "%s: %lld elements, need %lld", name, (long long)t.numel(),
          (long long)numel);
  return t.data_ptr();
}
int32_t* ints(PyObject* o, int64_t numel, const char* name) {
  return static_cast<int32_t*>(array(o, at::kInt, numel, name));
}
int32_t* ints_or_null(PyObject* o, int64_t numel, const char* name) {
  return o == Py_None ? nullptr : ints(o, numel, name);
}

// Rows [T][heads][d] that may be views of longer ones.
struct Rows {
  void* at;
  int64_t stride;  // elements between rows
};
Rows rows(PyObject* o, at::ScalarType type, int64_t T, int64_t heads, int64_t d, const char* name) {
  const at::Tensor& t = on_device(o, type, name);
  const auto z = t.sizes(), s = t.strides();
  if (z.size() != 3 || z[0] != T || z[1] != heads || z[2] != d)
    raise(PyExc_ValueError, "%s: shape %zd dimensions of %lld elements, expected (%lld, %lld, %lld)",
          name, (Py_ssize_t)z.size(), (long long)t.numel(), (long long)T, (long long)heads, (long long)d);
  if ((s[2] != 1 && d > 1) || (s[1] != d && heads > 1))
    raise(PyExc_ValueError, "%s: the heads of a row must be contiguous", name);
  return {t.data_ptr(), T > 1 ? s[0] : heads * d};
}

struct Heads {  // a tensor [T][heads][d] of an io type
  int io;
  at::ScalarType type;
  int64_t T, heads, d;
};
Heads heads_of(PyObject* o, const char* name) {
  if (THPVariable_Check(o)) {
    const at::Tensor& t = THPVariable_Unpack(o);
    const at::ScalarType type = t.scalar_type();
    const int io = type == at::kBFloat16 ? TGDN_BF16 : type == at::kHalf ? TGDN_F16
                                                     : type == at::kFloat ? TGDN_F32 : -1;
    if (io >= 0 && t.dim() == 3) return {io, type, t.size(0), t.size(1), t.size(2)};
  }
  raise(PyExc_TypeError, "%s: expected a float32, bfloat16 or float16 tensor [T][heads][d]", name);
}

int64_t size_of(PyObject* o, int dim, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() <= dim) raise(PyExc_ValueError, "%s: shape of %d dimensions", name, (int)t.dim());
  return t.size(dim);
}
int64_t numel(PyObject* o, const char* name) { return tensor(o, name).numel(); }

// What the C call takes as int32.
int32_t i32(int64_t x, const char* name) {
  if (x < INT32_MIN || x > INT32_MAX) raise(PyExc_ValueError, "%s: %lld is out of range", name, (long long)x);
  return (int32_t)x;
}

// ------------------------------------------------------------------ Python values
struct Ref {
  PyObject* o;
  explicit Ref(PyObject* x) : o(x) {
    if (o == nullptr) throw Raised();
  }
  ~Ref() { Py_DECREF(o); }
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
};

PyObject* names[24];
enum Name {
  N_B, N_T, N_n_max, N_depth_max, N_words, N_cu_nodes, N_parent, N_depth, N_order, N_pos, N_anc,
  N_status, N_n_pages, N_page_size, N_max_pages, N_table, N_len, N_held, N_refs, N_cuda_stream, N_count
};
const char* const kNames[] = {"B", "T", "n_max", "depth_max", "words", "cu_nodes", "parent", "depth",
                              "order", "pos", "anc", "status", "n_pages", "page_size", "max_pages",
                              "table", "len", "held", "refs", "cuda_stream"};
static_assert(sizeof(kNames) / sizeof(kNames[0]) == N_count && N_count <= 24, "a string per name");

int64_t integer(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw Raised();
  return x;
}
double real(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Raised();
  return x;
}
int truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw Raised();
  return x;
}
int32_t attr_int(PyObject* o, Name n) {
  const Ref a(PyObject_GetAttr(o, names[n]));
  return i32(integer(a.o), kNames[n]);
}
void* attr_array(PyObject* o, Name n, at::ScalarType type, int64_t numel) {
  const Ref a(PyObject_GetAttr(o, names[n]));  // (the object keeps the tensor alive)
  return array(a.o, type, numel, kNames[n]);
}
int32_t* attr_ints(PyObject* o, Name n, int64_t numel) {
  return static_cast<int32_t*>(attr_array(o, n, at::kInt, numel));
}

// None: the current stream; else a torch stream or a handle.
tgdn_stream_t stream_of(PyObject* o) {
  if (o == Py_None) return reinterpret_cast<tgdn_stream_t>(c10::cuda::getCurrentCUDAStream().stream());
  if (PyLong_Check(o)) return reinterpret_cast<tgdn_stream_t>((uintptr_t)integer(o));
  const Ref a(PyObject_GetAttr(o, names[N_cuda_stream]));
  return reinterpret_cast<tgdn_stream_t>((uintptr_t)integer(a.o));
}

tgdn_tree tree_of(PyObject* o) {
  tgdn_tree t{};
  t.B = attr_int(o, N_B);
  t.T = attr_int(o, N_T);
  t.n_max = attr_int(o, N_n_max);
  t.depth_max = attr_int(o, N_depth_max);
  t.words = attr_int(o, N_words);
  t.cu_nodes = attr_ints(o, N_cu_nodes, (int64_t)t.B + 1);
  t.parent = attr_ints(o, N_parent, t.T);
  t.depth = attr_ints(o, N_depth, t.T);
  t.order = attr_ints(o, N_order, t.T);
  t.pos = attr_ints(o, N_pos, t.T);
  t.anc = static_cast<uint64_t*>(attr_array(o, N_anc, at::kLong, (int64_t)t.T * t.words));
  t.status = attr_ints(o, N_status, t.B);
  return t;
}

tgdn_pages pages_of(PyObject* o) {
  tgdn_pages p{};
  p.B = attr_int(o, N_B);
  p.n_pages = attr_int(o, N_n_pages);
  p.page_size = attr_int(o, N_page_size);
  p.max_pages = attr_int(o, N_max_pages);
  p.table = attr_ints(o, N_table, (int64_t)p.B * p.max_pages);
  p.len = attr_ints(o, N_len, p.B);
  p.held = attr_ints(o, N_held, p.B);
  p.refs = attr_ints(o, N_refs, p.n_pages);
  p.status = attr_ints(o, N_status, p.B);
  return p;
}

struct Pool {
  tgdn_pool c;
  at::ScalarType type;
};
Pool pool_of(PyObject* o, const tgdn_pages& p) {
  if (!THPVariable_Check(o) || (THPVariable_Unpack(o).scalar_type() != at::kBFloat16 &&
                                THPVariable_Unpack(o).scalar_type() != at::kHalf))
    raise(PyExc_TypeError, "pool: expected a bfloat16 or float16 tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  const auto z = t.sizes();
  if (z.size() != 6 || z[1] != 2 || z[2] != p.n_pages || z[4] != p.page_size)
    raise(PyExc_ValueError, "pool: shape of %lld elements, expected (layers, 2, n_pages, H_kv, page_size, d)",
          (long long)t.numel());
  Pool pool{{}, t.scalar_type()};
  pool.c.layers = i32(z[0], "pool");
  pool.c.H_kv = i32(z[3], "pool");
  pool.c.d = i32(z[5], "pool");
  pool.c.data = array(o, pool.type, 0, "pool");
  return pool;
}

struct Space {
  void* at;
  size_t bytes;
};
Space space(PyObject* o) {
  if (o == Py_None || numel(o, "ws") == 0) return {nullptr, 0};
  const at::Tensor& t = THPVariable_Unpack(o);
  return {array(o, t.scalar_type(), 0, "ws"), (size_t)t.numel() * t.element_size()};
}
void* pages_space(PyObject* o, const tgdn_pages& p) {
  return array(o, at::kByte, (int64_t)tgdn_pages_workspace_bytes(&p), "ws");
}

// ------------------------------------------------------------------ the calls
// The C call without the interpreter's lock (a full launch queue makes it wait).
template <typename F>
int unlocked(F&& call) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = call();
  Py_END_ALLOW_THREADS
  return rc;
}

int rope(PyObject* const* a) {
  PyObject *q = a[0], *k = a[1], *q_out = a[2], *k_out = a[3], *freq = a[4], *cu = a[5], *base = a[6],
           *off = a[7];
  const Heads h = heads_of(q, "q");
  const int64_t H_kv = k == Py_None ? 0 : size_of(k, 1, "k");
  const int32_t B = i32(numel(cu, "cu") - 1, "cu"), T = i32(h.T, "q");
  const Rows rq = rows(q, h.type, h.T, h.heads, h.d, "q"), ro = rows(q_out, h.type, h.T, h.heads, h.d, "q_out");
  Rows rk{nullptr, 0}, rko{nullptr, 0};
  if (k != Py_None) {
    rk = rows(k, h.type, h.T, H_kv, h.d, "k");
    rko = rows(k_out, h.type, h.T, H_kv, h.d, "k_out");
  }
  const int64_t half = numel(freq, "freq");
  const uint64_t* f = static_cast<uint64_t*>(array(freq, at::kLong, half, "freq"));
  const int32_t *c = ints(cu, (int64_t)B + 1, "cu"), *b = ints_or_null(base, B, "base"),
                *o = ints_or_null(off, T, "off");
  const int inter = truth(a[8]), back = truth(a[10]);
  const float mscale = (float)real(a[9]);
  const int32_t H = i32(h.heads, "q"), Hk = i32(H_kv, "k"), d = i32(h.d, "q"), rot = i32(2 * half, "freq");
  const tgdn_stream_t s = stream_of(a[11]);
  return unlocked([&] {
    return tgdn_rope(B, T, H, Hk, d, rot, inter, back, h.io, mscale, f, c, b, o, rq.at, rq.stride, rk.at,
                     rk.stride, ro.at, ro.stride, rko.at, rko.stride, s);
  });
}

int prompt_attention(PyObject* const* a) {
  PyObject *cu = a[0], *q = a[1], *k = a[2], *v = a[3], *o = a[4];
  const Heads h = heads_of(q, "q");
  const int64_t H_kv = size_of(k, 1, "k");
  const int32_t B = i32(numel(cu, "cu") - 1, "cu"), T = i32(h.T, "q");
  const Rows rq = rows(q, h.type, h.T, h.heads, h.d, "q"), rk = rows(k, h.type, h.T, H_kv, h.d, "k"),
             rv = rows(v, h.type, h.T, H_kv, h.d, "v"), ro = rows(o, h.type, h.T, h.heads, h.d, "o");
  const Space ws = space(a[7]);
  const int32_t* c = ints(cu, (int64_t)B + 1, "cu");
  int32_t* status = ints(a[6], B, "status");
  const float scale = (float)real(a[5]);
  const int32_t H = i32(h.heads, "q"), Hk = i32(H_kv, "k"), d = i32(h.d, "q");
  const tgdn_stream_t s = stream_of(a[8]);
  return unlocked([&] {
    return tgdn_prompt_attention(B, T, H, Hk, d, h.io, c, rq.at, rq.stride, rk.at, rk.stride, rv.at,
                                 rv.stride, scale, ro.at, ro.stride, status, ws.at, ws.bytes, s);
  });
}

int pages_reserve(PyObject* const* a) {
  const tgdn_pages p = pages_of(a[0]);
  const int32_t* add = ints(a[1], p.B, "add");
  void* ws = pages_space(a[2], p);
  const tgdn_stream_t s = stream_of(a[3]);
  return unlocked([&] { return tgdn_pages_reserve(&p, add, ws, s); });
}

// Rows [layers][T][H_kv][d], or [T][H_kv][d] for one layer.
struct Layers {
  void* at;
  int64_t layer, row;
};
Layers layers_of(PyObject* o, const Pool& pool, int64_t T, const char* name) {
  const at::Tensor& t = tensor(o, name);
  const auto z = t.sizes(), s = t.strides();
  const size_t n = z.size();
  if ((n != 3 && n != 4) || (n == 4 ? z[0] : 1) != pool.c.layers)
    raise(PyExc_ValueError, "%s: expected a tensor [%d][T][H_kv][d]", name, (int)pool.c.layers);
  (void)on_device(o, pool.type, name);
  if (z[n - 3] != T || z[n - 2] != pool.c.H_kv || z[n - 1] != pool.c.d)
    raise(PyExc_ValueError, "%s: shape of %lld elements, expected (%d, %lld, %d, %d)", name,
          (long long)t.numel(), (int)pool.c.layers, (long long)T, (int)pool.c.H_kv, (int)pool.c.d);
  if ((s[n - 1] != 1 && pool.c.d > 1) || (s[n - 2] != pool.c.d && pool.c.H_kv > 1))
    raise(PyExc_ValueError, "%s: the heads of a row must be contiguous", name);
  return {t.data_ptr(), pool.c.layers > 1 ? s[0] : 0,
          T > 1 ? s[n - 3] : (int64_t)pool.c.H_kv * pool.c.d};
}

int pages_append(PyObject* const* a) {
  PyObject *cu = a[1], *k = a[2], *v = a[3], *path = a[5], *n_path = a[6];
  const tgdn_pages p = pages_of(a[0]);
  const Pool pool = pool_of(a[4], p);
  const at::Tensor& tk = tensor(k, "k");
  if (tk.dim() < 3) raise(PyExc_ValueError, "k: expected a tensor [%d][T][H_kv][d]", (int)pool.c.layers);
  const int64_t T = tk.size(tk.dim() - 3);
  const Layers rk = layers_of(k, pool, T, "k"), rv = layers_of(v, pool, T, "v");
  const int32_t* c = ints(cu, (int64_t)p.B + 1, "cu");
  const int32_t len = path == Py_None ? 0 : i32(size_of(path, 1, "path"), "path");
  const int32_t* nodes = ints_or_null(path, (int64_t)p.B * len, "path");
  const int32_t* n = path == Py_None ? nullptr : ints(n_path, p.B, "n_path");
  const int32_t rows = i32(T, "k"), advance = truth(a[7]);
  const tgdn_stream_t s = stream_of(a[8]);
  return unlocked([&] {
    return tgdn_pages_append(&p, &pool.c, rows, c, nodes, len, n, rk.at, rk.layer, rk.row, rv.at, rv.layer,
                             rv.row, advance, s);
  });
}

int pages_fork(PyObject* const* a) {
  const tgdn_pages p = pages_of(a[0]);
  const int32_t n = i32(numel(a[1], "src"), "src");
  const Pool pool = pool_of(a[3], p);
  const int32_t *src = ints(a[1], n, "src"), *dst = ints(a[2], n, "dst");
  int32_t* status = ints(a[4], n, "status");
  void* ws = pages_space(a[5], p);
  const tgdn_stream_t s = stream_of(a[6]);
  return unlocked([&] { return tgdn_pages_fork(&p, &pool.c, n, src, dst, status, ws, s); });
}

int pages_free(PyObject* const* a) {
  const tgdn_pages p = pages_of(a[0]);
  const int32_t n = i32(numel(a[1], "seq"), "seq");
  const int32_t* seq = ints(a[1], n, "seq");
  const tgdn_stream_t s = stream_of(a[2]);
  return unlocked([&] { return tgdn_pages_free(&p, n, seq, s); });
}

int pages_compact(PyObject* const* a) {
  const tgdn_pages p = pages_of(a[0]);
  const Pool pool = pool_of(a[1], p);
  int32_t* n_live = ints(a[2], 1, "n_live");
  void* ws = pages_space(a[3], p);
  const tgdn_stream_t s = stream_of(a[4]);
  return unlocked([&] { return tgdn_pages_compact(&p, &pool.c, n_live, ws, s); });
}

int paged_tree_attention(PyObject* const* a) {
  PyObject *q = a[2], *k = a[3], *v = a[4], *o = a[7];
  const Heads h = heads_of(q, "q");
  const tgdn_tree t = tree_of(a[0]);
  if (h.T != t.T)
    raise(PyExc_ValueError, "q: %lld rows, the tree has %d", (long long)h.T, (int)t.T);
  const tgdn_pages p = pages_of(a[1]);
  const int64_t H_kv = size_of(k, 1, "k_tree");
  const Rows rq = rows(q, h.type, h.T, h.heads, h.d, "q"), rk = rows(k, h.type, h.T, H_kv, h.d, "k_tree"),
             rv = rows(v, h.type, h.T, H_kv, h.d, "v_tree"), ro = rows(o, h.type, h.T, h.heads, h.d, "o");
  const int64_t n = (int64_t)p.n_pages * H_kv * p.page_size * h.d;
  const void *kp = array(a[5], h.type, n, "k_pages"), *vp = array(a[6], h.type, n, "v_pages");
  const Space ws = space(a[9]);
  const float scale = (float)real(a[8]);
  const int32_t H = i32(h.heads, "q"), Hk = i32(H_kv, "k_tree"), d = i32(h.d, "q");
  const tgdn_stream_t s = stream_of(a[10]);
  return unlocked([&] {
    return tgdn_paged_tree_attention(&t, &p, H, Hk, d, h.io, rq.at, rq.stride, rk.at, rk.stride, rv.at,
                                     rv.stride, kp, vp, scale, ro.at, ro.stride, ws.at, ws.bytes, s);
  });
}

// Python's entry: the arguments counted, C++ exceptions turned into Python's.
template <int (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  g_device = -1;
  try {
    if (n != N) raise(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return PyLong_FromLong(F(args));
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

#define CALL(name, n) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(rope, 12),         CALL(prompt_attention, 9),      CALL(pages_reserve, 4),
                         CALL(pages_append, 9),  CALL(pages_fork, 7),            CALL(pages_free, 3),
                         CALL(pages_compact, 5), CALL(paged_tree_attention, 11), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
  for (int i = 0; i < N_count; ++i)
    if ((names[i] = PyUnicode_InternFromString(kNames[i])) == nullptr) return nullptr;
  return PyModule_Create(&module);
}
