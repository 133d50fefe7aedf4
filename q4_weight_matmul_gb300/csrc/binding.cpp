// The Python module _calls: the attention block's calls from torch tensors to
// the C ABI (include/q4k.h).  Checking ten tensors and passing twenty
// arguments took some 6 us of interpreted code, twice the kernel of a single
// token's heads; here it takes a few hundred nanoseconds.  Every function
// takes its arguments by position, raises TypeError or ValueError for a tensor
// that is not what the call reads, and returns the call's q4k_status.  Like
// the rest of the binding it only marshals.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <dlfcn.h>
#include <q4k.h>

namespace {

decltype(&q4k_qk_norm_rope) g_qk_norm_rope;
decltype(&q4k_paged_attn) g_paged_attn;
decltype(&q4k_lora_add) g_lora_add;

struct Refused {};      // a Python exception is set

[[noreturn]] void refuse(PyObject* kind, const char* format, const char* name, long long a = 0, long long b = 0) {
  PyErr_Format(kind, format, name, a, b);
  throw Refused{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a CUDA tensor", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse(PyExc_TypeError, "%s must be a CUDA tensor", name);
  return t;
}

// The address of a contiguous tensor of `type` with exactly n elements.
void* address(const at::Tensor& t, at::ScalarType type, int64_t n, const char* name) {
  if (t.scalar_type() != type) refuse(PyExc_TypeError, "%s has another type than the call reads", name);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
  if (t.numel() != n) refuse(PyExc_ValueError, "%s must hold %lld elements, got %lld", name, n, t.numel());
  return t.data_ptr();
}
void* address(PyObject* o, at::ScalarType type, int64_t n, const char* name) {
  return address(tensor(o, name), type, n, name);
}
template <class T>
T* pointer(PyObject* o, at::ScalarType type, int64_t n, const char* name) {
  return static_cast<T*>(address(o, type, n, name));
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}
int small_integer(PyObject* o) {      // out of int's range: a value that every call refuses
  const int64_t v = integer(o);
  return v > INT32_MAX || v < INT32_MIN ? INT32_MIN : (int)v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused{};
  return v != 0;
}

// A stream argument: None (torch's current one), an object with cuda_stream, or a handle.
void* stream_of(PyObject* o) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
  PyObject* s = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream") : Py_NewRef(o);
  void* p = s ? PyLong_AsVoidPtr(s) : nullptr;
  Py_XDECREF(s);
  if (PyErr_Occurred()) throw Refused{};
  return p;
}

int half_type(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kHalf) return Q4K_F16;
  if (t.scalar_type() != at::kBFloat16) refuse(PyExc_TypeError, "%s must be float16 or bfloat16", name);
  return Q4K_BF16;
}

struct Cache {
  q4k_kv_cache c;
  at::ScalarType type;
};
Cache cache_of(PyObject* k, PyObject* v) {
  const at::Tensor &kt = tensor(k, "k_cache"), &vt = tensor(v, "v_cache");
  Cache r{};
  r.c.type = half_type(kt, "k_cache");
  r.type = kt.scalar_type();
  if (kt.dim() != 4)
    refuse(PyExc_TypeError, "%s must be [num_pages][kv_heads][page_size][head_dim]", "k_cache");
  if (vt.sizes() != kt.sizes()) refuse(PyExc_ValueError, "%s must have k_cache's shape", "v_cache");
  r.c.k = address(kt, r.type, kt.numel(), "k_cache");
  r.c.v = address(vt, r.type, kt.numel(), "v_cache");
  r.c.num_pages = kt.size(0);
  r.c.kv_heads = (int32_t)kt.size(1);
  r.c.page_size = (int32_t)kt.size(2);
  r.c.head_dim = (int32_t)kt.size(3);
  return r;
}

// (q, k, v, k_cache, v_cache, pos, slot, cos_sin, q_weight, k_weight, eps, interleaved, q_out, stream)
int qk_norm_rope(PyObject* const* a) {
  const Cache c = cache_of(a[3], a[4]);
  const at::Tensor& q = tensor(a[0], "q");
  if (q.dim() < 2) refuse(PyExc_ValueError, "%s must be [tokens][heads * head_dim]", "q");
  const int64_t tokens = q.size(0), dim = c.c.head_dim, heads = q.dim() == 3 ? q.size(1) : q.size(1) / std::max<int64_t>(dim, 1);
  const int64_t nq = tokens * heads * dim, nk = tokens * c.c.kv_heads * dim;
  int64_t max_pos = 0, rot = 0;
  const float* cos_sin = nullptr;
  if (a[7] != Py_None) {
    const at::Tensor& t = tensor(a[7], "cos_sin");
    if (t.dim() != 2) refuse(PyExc_ValueError, "%s must be [max_pos][rot_dim]", "cos_sin");
    max_pos = t.size(0), rot = t.size(1);
    if (rot) cos_sin = static_cast<const float*>(address(t, at::kFloat, max_pos * rot, "cos_sin"));
  }
  if (rot > INT32_MAX || heads > INT32_MAX) refuse(PyExc_ValueError, "%s is too wide", "q");
  return g_qk_norm_rope(
      static_cast<const float*>(address(q, at::kFloat, nq, "q")), pointer<const float>(a[1], at::kFloat, nk, "k"),
      pointer<const float>(a[2], at::kFloat, nk, "v"), tokens, (int)heads, &c.c,
      a[8] == Py_None ? nullptr : pointer<const float>(a[8], at::kFloat, dim, "q_weight"),
      a[9] == Py_None ? nullptr : pointer<const float>(a[9], at::kFloat, dim, "k_weight"), (float)number(a[10]), cos_sin,
      max_pos, (int)rot, truth(a[11]),
      rot ? pointer<const int32_t>(a[5], at::kInt, tokens, "pos") : nullptr,
      pointer<const int32_t>(a[6], at::kInt, tokens, "slot"), address(a[12], c.type, nq, "q_out"), stream_of(a[13]));
}

// (q, k_cache, v_cache, page_table, cu_q, kv_len, max_q, scale, window, out, workspace, stream)
int paged_attn(PyObject* const* a) {
  const Cache c = cache_of(a[1], a[2]);
  const at::Tensor &q = tensor(a[0], "q"), &table = tensor(a[3], "page_table"), &out = tensor(a[9], "out"),
                   &work = tensor(a[10], "workspace");
  if (q.dim() != 3 || q.size(2) != c.c.head_dim) refuse(PyExc_ValueError, "%s must be [tokens][heads][head_dim]", "q");
  if (table.dim() != 2) refuse(PyExc_ValueError, "%s must be [n_req][max_pages]", "page_table");
  if (out.sizes() != q.sizes()) refuse(PyExc_ValueError, "%s must have q's shape", "out");
  const int out_type = out.scalar_type() == at::kFloat ? Q4K_F32 : half_type(out, "out");
  const int64_t n_req = table.size(0), max_pages = table.size(1), n = q.numel();
  if (q.size(1) > INT32_MAX) refuse(PyExc_ValueError, "%s has too many heads", "q");
  const double scale = a[7] == Py_None ? 1.0 / std::sqrt((double)c.c.head_dim) : number(a[7]);
  return g_paged_attn(address(q, c.type, n, "q"), q.size(0), (int)q.size(1), &c.c,
                      static_cast<const int32_t*>(address(table, at::kInt, n_req * max_pages, "page_table")), max_pages,
                      pointer<const int32_t>(a[4], at::kInt, n_req + 1, "cu_q"),
                      pointer<const int32_t>(a[5], at::kInt, n_req, "kv_len"), n_req, integer(a[6]), (float)scale,
                      small_integer(a[8]), address(out, out.scalar_type(), n, "out"), out_type,
                      address(work, at::kByte, work.numel(), "workspace"), (size_t)work.numel(), stream_of(a[11]));
}

// (x, a, b, base, order, seg_start, seg_adapter, scale, y, workspace, stream); a, b, base, y: sequences of one length
int lora_add(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0], "x"), &work = tensor(a[9], "workspace"), &segments = tensor(a[6], "seg_adapter");
  if (x.dim() != 2) refuse(PyExc_ValueError, "%s must be [tokens][cols]", "x");
  const int64_t tokens = x.size(0), cols = x.size(1), n_seg = segments.numel();
  struct List {
    PyObject* seq;
    explicit List(PyObject* o) : seq(PySequence_Fast(o, "a, b, base and y must be lists")) {
      if (!seq) throw Refused{};
    }
    ~List() { Py_DECREF(seq); }
    Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(seq); }
    PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq, i); }
  } la(a[1]), lb(a[2]), lbase(a[3]), ly(a[8]);
  const Py_ssize_t n = la.size();
  if (n == 0 || lb.size() != n || lbase.size() != n || ly.size() != n)
    refuse(PyExc_ValueError, "%s, b, base and y must be lists of one length", "a");
  q4k_lora_mat mats[8];
  if (n > 8) return Q4K_ERR_UNSUPPORTED;
  const at::Tensor& first = tensor(la[0], "a");
  const int type = half_type(first, "a");
  if (first.dim() != 3) refuse(PyExc_ValueError, "every %s must be [n_adapters][rank][cols]", "a");
  const int64_t adapters = first.size(0), rank = first.size(1);
  for (Py_ssize_t m = 0; m < n; ++m) {
    const at::Tensor &am = tensor(la[m], "a"), &bm = tensor(lb[m], "b");
    if (am.sizes() != at::IntArrayRef({adapters, rank, cols}) || bm.dim() != 3 || bm.size(0) != adapters ||
        bm.size(2) != rank)
      refuse(PyExc_ValueError, "every %s must be [n_adapters][rank][cols], every b [n_adapters][rows][rank]", "a");
    const int64_t rows = bm.size(1);
    mats[m].a = address(am, first.scalar_type(), am.numel(), "a");
    mats[m].b = address(bm, first.scalar_type(), bm.numel(), "b");
    mats[m].base = lbase[m] == Py_None ? nullptr : pointer<const float>(lbase[m], at::kFloat, tokens * rows, "base");
    mats[m].y = pointer<float>(ly[m], at::kFloat, tokens * rows, "y");
    mats[m].rows = rows;
  }
  return g_lora_add((int)n, mats, adapters, (int)std::min<int64_t>(rank, INT32_MAX), type, cols,
                    static_cast<const float*>(address(x, at::kFloat, tokens * cols, "x")), tokens,
                    pointer<const int32_t>(a[4], at::kInt, tokens, "order"),
                    pointer<const int32_t>(a[5], at::kInt, n_seg + 1, "seg_start"),
                    static_cast<const int32_t*>(address(segments, at::kInt, n_seg, "seg_adapter")), n_seg,
                    pointer<const float>(a[7], at::kFloat, adapters, "scale"),
                    address(work, at::kByte, work.numel(), "workspace"), (size_t)work.numel(), stream_of(a[10]));
}

template <int (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) return PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
  if (!g_qk_norm_rope) return PyErr_Format(PyExc_RuntimeError, "the library has not been bound");
  try {
    return PyLong_FromLong(F(args));
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    return PyErr_Format(PyExc_RuntimeError, "%s", e.what());
  }
}

// bind(path): the C ABI's functions from the library at `path`.
PyObject* bind(PyObject*, PyObject* path) {
  const char* p = PyUnicode_AsUTF8(path);
  if (!p) return nullptr;
  void* lib = dlopen(p, RTLD_NOW | RTLD_LOCAL);
  if (!lib) return PyErr_Format(PyExc_RuntimeError, "%s", dlerror());
  g_qk_norm_rope = reinterpret_cast<decltype(g_qk_norm_rope)>(dlsym(lib, "q4k_qk_norm_rope"));
  g_paged_attn = reinterpret_cast<decltype(g_paged_attn)>(dlsym(lib, "q4k_paged_attn"));
  g_lora_add = reinterpret_cast<decltype(g_lora_add)>(dlsym(lib, "q4k_lora_add"));
  if (!g_qk_norm_rope || !g_paged_attn || !g_lora_add) {
    g_qk_norm_rope = nullptr;
    return PyErr_Format(PyExc_RuntimeError, "%s lacks a function", p);
  }
  Py_RETURN_NONE;
}

template <int (*F)(PyObject* const*), int N>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<F, N>));
}

PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr},
                         {"qk_norm_rope", fast<qk_norm_rope, 14>(), METH_FASTCALL, nullptr},
                         {"paged_attn", fast<paged_attn, 12>(), METH_FASTCALL, nullptr},
                         {"lora_add", fast<lora_add, 11>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
