// The cache calls of dilattn.py, marshalled in C++.
//
// A serving step makes these calls once for each layer and token, and their
// kernels take a few microseconds; looking at ten tensors from Python takes
// thirty. Each function here makes the same checks and the same C call as its
// namesake in dilattn.py, for the plain form of the call: tensors on the current
// device, the current stream. Whatever is not so, an argument that does not fit
// included, gives None, and nothing has been done: dilattn.py then goes through
// the call itself, names the fault or takes the rarer form.
//
// Otherwise a call gives (status, results ...), the status being the library's.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <dlfcn.h>

#include <initializer_list>

#include "dilattn.h"

namespace {

decltype(&dilattn_cache_write) g_write;
decltype(&dilattn_cache_read) g_read;
decltype(&dilattn_decode) g_decode;
decltype(&dilattn_decode_workspace_size) g_workspace_size;

using Sizes = std::initializer_list<int64_t>;

const at::Tensor* tensor(PyObject* o) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.defined() && !t.unsafeGetTensorImpl()->is_python_dispatch() && t.layout() == at::kStrided ? &t
                                                                                                     : nullptr;
}

bool on(const at::Tensor& t, int dev) { return t.is_cuda() && t.get_device() == dev; }

// A contiguous tensor of this shape and type on the device.
bool fits(const at::Tensor* t, at::ScalarType type, Sizes shape, int dev) {
  return t != nullptr && t->scalar_type() == type && on(*t, dev) && t->sizes() == c10::IntArrayRef(shape) &&
         t->is_contiguous();
}

// A bf16 [T, heads, d] tensor with whole rows; the distance of its tokens in elements, or -1.
int64_t rows(const at::Tensor* t, int64_t T, int64_t heads, int64_t d, int dev) {
  if (t == nullptr || t->scalar_type() != at::kBFloat16 || !on(*t, dev) ||
      t->sizes() != c10::IntArrayRef({T, heads, d}))
    return -1;
  const int64_t row = heads * d;
  if (t->is_contiguous()) return row;
  const int64_t stride = t->stride(0);
  if ((d > 1 && t->stride(2) != 1) || (heads > 1 && t->stride(1) != d) || stride < row || stride % 8 != 0)
    return -1;
  return stride;
}

// The cache and its table, as every call takes them.
struct CacheArgs {
  const at::Tensor *k, *v, *ks, *vs, *table;
  int64_t pages, Hkv, P, d, B, max_pages;
  int format, dev;
  bool read(PyObject* const* a) {  // k, v, k_scale, v_scale, table
    k = tensor(a[0]), v = tensor(a[1]), ks = tensor(a[2]), vs = tensor(a[3]), table = tensor(a[4]);
    if (k == nullptr || k->dim() != 4 || table == nullptr || table->dim() != 2) return false;
    if (k->scalar_type() == at::kFloat8_e4m3fn) format = DILATTN_CACHE_E4M3;
    else if (k->scalar_type() == at::kChar) format = DILATTN_CACHE_INT8;
    else return false;
    if (!k->is_cuda()) return false;
    dev = k->get_device();
    if (dev != c10::cuda::current_device()) return false;
    pages = k->size(0), Hkv = k->size(1), P = k->size(2), d = k->size(3);
    B = table->size(0), max_pages = table->size(1);
    constexpr int64_t most = 0x7fffffff;
    return pages <= most && Hkv <= most && B < most && max_pages <= most &&
           fits(k, k->scalar_type(), {pages, Hkv, P, d}, dev) && fits(v, k->scalar_type(), {pages, Hkv, P, d}, dev) &&
           fits(ks, at::kFloat, {pages, Hkv}, dev) && fits(vs, at::kFloat, {pages, Hkv}, dev) &&
           fits(table, at::kInt, {B, max_pages}, dev);
  }
};

// Positions of a ragged batch: start [B], offsets [B + 1] or None (T = B).
bool ranges(const CacheArgs& c, PyObject* start_o, PyObject* offsets_o, int64_t T, const int** start,
            const int** offsets) {
  const at::Tensor* s = tensor(start_o);
  if (T > 0x7fffffff || !fits(s, at::kInt, {c.B}, c.dev)) return false;
  *start = s->const_data_ptr<int>();
  *offsets = nullptr;
  if (offsets_o == Py_None) return T == c.B;
  const at::Tensor* o = tensor(offsets_o);
  if (!fits(o, at::kInt, {c.B + 1}, c.dev)) return false;
  *offsets = o->const_data_ptr<int>();
  return true;
}

at::Tensor empty(Sizes shape, at::ScalarType type, int dev) {
  return at::empty(shape, at::TensorOptions(type).device(at::kCUDA, dev));
}

cudaStream_t current_stream(int dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }

// A given output, or a new one.
bool output(PyObject* o, Sizes shape, at::ScalarType type, int dev, at::Tensor* out) {
  if (o == Py_None) {
    *out = empty(shape, type, dev);
    return true;
  }
  const at::Tensor* t = tensor(o);
  if (!fits(t, type, shape, dev)) return false;
  *out = *t;
  return true;
}

// The calls take their arguments by position; a wrong number of them is a mistake in dilattn.py.
bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return n == want;
}

// k_cache, v_cache, k_scale, v_scale, table, k, v, start, offsets -> (status,)
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 9)) return nullptr;
  CacheArgs c;
  if (!c.read(a)) Py_RETURN_NONE;
  const at::Tensor *k = tensor(a[5]), *v = tensor(a[6]);
  if (k == nullptr || k->dim() != 3) Py_RETURN_NONE;
  const int64_t T = k->size(0);
  const int64_t sk = rows(k, T, c.Hkv, c.d, c.dev), sv = rows(v, T, c.Hkv, c.d, c.dev);
  const int *start, *offsets;
  if (sk < 0 || sv < 0 || !ranges(c, a[7], a[8], T, &start, &offsets)) Py_RETURN_NONE;
  const cudaStream_t stream = current_stream(c.dev);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g_write(k->data_ptr(), v->data_ptr(), sk, sv, offsets, start, (int)T, c.table->const_data_ptr<int>(),
               (int)c.B, (int)c.max_pages, c.k->data_ptr(), c.v->data_ptr(), (float*)c.ks->data_ptr(),
               (float*)c.vs->data_ptr(), (int)c.pages, (int)c.Hkv, (int)c.P, (int)c.d, c.format, stream);
  Py_END_ALLOW_THREADS
  return Py_BuildValue("(i)", rc);
  END_HANDLE_TH_ERRORS
}

// k_cache, v_cache, k_scale, v_scale, table, start, offsets, total -> (status, k, v)
PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 8)) return nullptr;
  CacheArgs c;
  if (!c.read(a)) Py_RETURN_NONE;
  int64_t T = c.B;
  if (a[7] != Py_None) {
    if (!PyLong_CheckExact(a[7])) Py_RETURN_NONE;
    int over = 0;
    T = PyLong_AsLongLongAndOverflow(a[7], &over);
    if (over != 0 || T < 0) Py_RETURN_NONE;
  } else if (a[6] != Py_None) {
    Py_RETURN_NONE;
  }
  const int *start, *offsets;
  if (!ranges(c, a[5], a[6], T, &start, &offsets)) Py_RETURN_NONE;
  at::Tensor k = empty({T, c.Hkv, c.d}, at::kBFloat16, c.dev), v = empty({T, c.Hkv, c.d}, at::kBFloat16, c.dev);
  const cudaStream_t stream = current_stream(c.dev);
  const long long row = c.Hkv * c.d;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g_read(c.k->data_ptr(), c.v->data_ptr(), (const float*)c.ks->data_ptr(), (const float*)c.vs->data_ptr(),
              (int)c.pages, (int)c.Hkv, (int)c.P, (int)c.d, c.format, c.table->const_data_ptr<int>(), (int)c.B,
              (int)c.max_pages, offsets, start, (int)T, k.data_ptr(), v.data_ptr(), row, row, stream);
  Py_END_ALLOW_THREADS
  return Py_BuildValue("(iNN)", rc, THPVariable_Wrap(std::move(k)), THPVariable_Wrap(std::move(v)));
  END_HANDLE_TH_ERRORS
}

// k_cache, v_cache, k_scale, v_scale, table, q, pos, patterns, seq, out, lse, workspace
// -> (status, out, lse)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 12)) return nullptr;
  CacheArgs c;
  if (!c.read(a)) Py_RETURN_NONE;
  const at::Tensor *q = tensor(a[5]), *pos = tensor(a[6]);
  if (q == nullptr || q->dim() != 3 || c.Hkv < 1) Py_RETURN_NONE;
  const int64_t T = q->size(0), H = q->size(1);
  if (T > 0x7fffffff || H < 1 || H > 0x7fffffff || H % c.Hkv != 0) Py_RETURN_NONE;
  const int64_t sq = rows(q, T, H, c.d, c.dev);
  if (sq < 0 || !fits(pos, at::kInt, {T}, c.dev)) Py_RETURN_NONE;
  int w[DILATTN_MAX_PATTERNS], r[DILATTN_MAX_PATTERNS];
  PyObject* pats = a[7];  // a list or tuple of pairs of int
  if (!PyList_CheckExact(pats) && !PyTuple_CheckExact(pats)) Py_RETURN_NONE;
  const Py_ssize_t npat = PySequence_Fast_GET_SIZE(pats);
  if (npat < 1 || npat > DILATTN_MAX_PATTERNS) Py_RETURN_NONE;
  for (Py_ssize_t i = 0; i < npat; ++i) {
    PyObject* p = PySequence_Fast_GET_ITEM(pats, i);
    if ((!PyTuple_CheckExact(p) && !PyList_CheckExact(p)) || PySequence_Fast_GET_SIZE(p) != 2) Py_RETURN_NONE;
    int* to[2] = {&w[i], &r[i]};
    for (int j = 0; j < 2; ++j) {
      PyObject* x = PySequence_Fast_GET_ITEM(p, j);
      int over = 0;
      const long long y = PyLong_CheckExact(x) ? PyLong_AsLongLongAndOverflow(x, &over) : -1;
      if (over != 0 || y < 1 || y > 0x7fffffff) Py_RETURN_NONE;
      *to[j] = (int)y;
    }
  }
  const int* seq = nullptr;
  if (a[8] != Py_None) {
    const at::Tensor* s = tensor(a[8]);
    if (!fits(s, at::kInt, {T}, c.dev)) Py_RETURN_NONE;
    seq = s->const_data_ptr<int>();
  } else if (T > c.B) {
    Py_RETURN_NONE;
  }
  at::Tensor out, lse, workspace;
  if (!output(a[9], {T, H, c.d}, at::kBFloat16, c.dev, &out) || !output(a[10], {T, H}, at::kFloat, c.dev, &lse))
    Py_RETURN_NONE;
  if (a[11] == Py_None) {
    const size_t need = g_workspace_size((int)T, (int)H, (int)c.Hkv, (int)c.d);
    workspace = empty({(int64_t)(need > 256 ? need : 256)}, at::kByte, c.dev);
  } else {
    const at::Tensor* t = tensor(a[11]);
    if (t == nullptr || t->dim() != 1 || !fits(t, at::kByte, {t->size(0)}, c.dev)) Py_RETURN_NONE;
    workspace = *t;
  }
  const cudaStream_t stream = current_stream(c.dev);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g_decode(q->data_ptr(), sq, c.k->data_ptr(), c.v->data_ptr(), (const float*)c.ks->data_ptr(),
                (const float*)c.vs->data_ptr(), (int)c.pages, (int)c.Hkv, (int)c.P, (int)c.d, c.format,
                c.table->const_data_ptr<int>(), (int)c.B, (int)c.max_pages, seq, pos->const_data_ptr<int>(),
                out.data_ptr(), (float*)lse.data_ptr(), (int)T, (int)H, w, r, (int)npat, workspace.data_ptr(),
                (size_t)workspace.numel(), stream);
  Py_END_ALLOW_THREADS
  return Py_BuildValue("(iNN)", rc, THPVariable_Wrap(std::move(out)), THPVariable_Wrap(std::move(lse)));
  END_HANDLE_TH_ERRORS
}

template <typename F>
bool find(void* lib, const char* name, F* f) {
  *f = reinterpret_cast<F>(dlsym(lib, name));
  return *f != nullptr;
}

// bind(path): the library whose functions are called.
PyObject* bind(PyObject*, PyObject* path) {
  const char* name = PyUnicode_AsUTF8(path);
  if (name == nullptr) return nullptr;
  void* lib = dlopen(name, RTLD_NOW | RTLD_LOCAL);
  if (lib == nullptr || !find(lib, "dilattn_cache_write", &g_write) || !find(lib, "dilattn_cache_read", &g_read) ||
      !find(lib, "dilattn_decode", &g_decode) ||
      !find(lib, "dilattn_decode_workspace_size", &g_workspace_size)) {
    PyErr_SetString(PyExc_RuntimeError, dlerror());
    return nullptr;
  }
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"bind", bind, METH_O, nullptr},
    {"cache_write", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_write)), METH_FASTCALL, nullptr},
    {"cache_read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_read)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&kModule); }
