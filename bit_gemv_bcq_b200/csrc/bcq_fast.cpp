// bcq_fast.cpp -- the binding's common calls without the interpreter's part:
// a CPython module (_fast) over the C ABI of include/bcq.h for torch tensors.
//
// Every function does what its namesake in api.py does, for the calls that
// need nothing special: tensors of one CUDA device, which is the current one,
// on its current stream, in shapes and distances that the library takes.  For
// anything else, a call that is to be refused among it, it does nothing and
// returns NotImplemented, and api.py goes on and raises what there is to raise.
// What a usual call is, is checked here once more: a check that api.py gains or
// loses has its counterpart below (test_both_ways_refuse_the_same_calls compares
// them).  A call of kv4_attention takes half the host's time here (its smallest
// takes less than that on the GPU).
//
// The library is not linked: api.py hands over its entry points' addresses.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>

#include "bcq.h"

namespace {

decltype(&bcq_quantize_i8) p_quantize_i8;
decltype(&bcq_gemm_i8) p_gemm_i8;
decltype(&bcq_linear_i8_workspace_bytes) p_linear_bytes;
decltype(&bcq_linear_i8) p_linear_i8;
decltype(&bcq_kv4_append) p_kv4_append;
decltype(&bcq_kv4_read) p_kv4_read;
decltype(&bcq_kv4_attention_workspace_bytes) p_attention_bytes;
decltype(&bcq_kv4_attention) p_kv4_attention;

PyObject* no() { Py_RETURN_NOTIMPLEMENTED; }

// Calls an entry point without the interpreter's lock (a full launch queue
// makes it wait).
template <typename F>
bool called(const F& f) {
  PyThreadState* state = PyEval_SaveThread();
  const bcq_status s = f();
  PyEval_RestoreThread(state);
  return s == BCQ_OK;
}

// A CUDA tensor argument (index: its device's number, or -1 for any).
bool cuda_tensor(PyObject* o, const at::Tensor** t, int* index) {
  if (!THPVariable_Check(o)) return false;
  *t = &THPVariable_Unpack(o);
  if (!(*t)->is_cuda()) return false;
  const int at = (*t)->get_device();
  if (*index < 0) *index = at;
  return at == *index;
}

bool on_current(int index) { return c10::cuda::current_device() == index; }
void* stream_of(int index) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream(); }

int dtype_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kHalf: return BCQ_F16;
    case at::kBFloat16: return BCQ_BF16;
    case at::kFloat: return BCQ_F32;
    default: return -1;
  }
}
at::ScalarType type_of(long dtype) {
  return dtype == BCQ_F16 ? at::kHalf : dtype == BCQ_BF16 ? at::kBFloat16 : at::kFloat;
}

// (the dispatcher, and a tensor around a workspace, are a microsecond of the
// call's)
at::Tensor empty(const at::Tensor& like, at::IntArrayRef size, at::ScalarType type) {
  return at::Tensor(at::detail::empty_cuda(size, type, like.device(), std::nullopt));
}
// Memory in the current stream's order, until the end of the call.
c10::DataPtr workspace(size_t bytes) { return c10::cuda::CUDACachingAllocator::get()->allocate(bytes); }

// A matrix with contiguous rows that do not overlap; its row distance.
bool matrix(const at::Tensor& t, int64_t* rows, int64_t* cols, int64_t* ld) {
  if (t.dim() != 2) return false;
  *rows = t.size(0);
  *cols = t.size(1);
  *ld = t.stride(0);
  if (*rows < 2 || *cols < 2 || t.stride(1) != 1 || *ld < *cols) {
    if (*rows != 1 || *cols < 2 || t.stride(1) != 1) return false;
    *ld = (*cols + 15) / 16 * 16;
  }
  return *rows <= INT32_MAX && *cols <= INT32_MAX;
}
bool codes(const at::Tensor& t, int64_t* rows, int64_t* cols, int64_t* ld) {
  return t.scalar_type() == at::kChar && matrix(t, rows, cols, ld) && *ld % 16 == 0 &&
         reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0;
}
bool vector(const at::Tensor& t, at::ScalarType type, int64_t size) {
  return t.scalar_type() == type && t.dim() == 1 && t.size(0) == size && t.is_contiguous();
}

// out (None: a new one) of a product.
bool product_out(PyObject* o, int64_t M, int64_t N, at::ScalarType type, const at::Tensor& like,
                 int index, at::Tensor* y, int64_t* ldy) {
  if (o == Py_None) {
    *y = empty(like, {M, N}, type);
    *ldy = N;
    return true;
  }
  const at::Tensor* t;
  int64_t rows, cols;
  if (!cuda_tensor(o, &t, &index) || t->scalar_type() != type || !matrix(*t, &rows, &cols, ldy) ||
      rows != M || cols != N)
    return false;
  *y = *t;
  return true;
}

PyObject* done(const at::Tensor& y, PyObject* out) {
  if (out == Py_None) return THPVariable_Wrap(y);
  Py_INCREF(out);
  return out;
}

// quantize_i8(x)
PyObject* quantize_i8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const at::Tensor* x;
  int index = -1;
  int64_t M, K, ldx;
  if (n != 1 || !cuda_tensor(a[0], &x, &index) || !on_current(index)) return no();
  const int dtype = dtype_of(*x);
  if ((dtype != BCQ_F16 && dtype != BCQ_BF16) || !matrix(*x, &M, &K, &ldx)) return no();
  const int64_t ldq = (K + 15) / 16 * 16;
  at::Tensor q = empty(*x, {M, ldq}, at::kChar), scale = empty(*x, {M}, at::kFloat);
  if (!called([&] { return p_quantize_i8(x->data_ptr(), dtype, (int)M, (int)K, ldx, (int8_t*)q.data_ptr(), ldq,
                    (float*)scale.data_ptr(), stream_of(index)); }))
    return no();
  if (ldq != K) q = q.narrow(1, 0, K);
  return Py_BuildValue("(NN)", THPVariable_Wrap(q), THPVariable_Wrap(scale));
}

// gemm_i8(x, x_scale, w, w_scale, dtype, out)
PyObject* gemm_i8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const at::Tensor *x, *sx, *w, *sw;
  int index = -1;
  int64_t M, N, K, KW, ldx, ldw, ldy;
  if (n != 6 || !cuda_tensor(a[0], &x, &index) || !cuda_tensor(a[1], &sx, &index) ||
      !cuda_tensor(a[2], &w, &index) || !cuda_tensor(a[3], &sw, &index) || !on_current(index) ||
      !codes(*x, &M, &K, &ldx) || !codes(*w, &N, &KW, &ldw) || K != KW ||
      !vector(*sx, at::kFloat, M) || !vector(*sw, at::kFloat, N))
    return no();
  const long dtype = PyLong_AsLong(a[4]);
  at::Tensor y;
  if (!product_out(a[5], M, N, type_of(dtype), *x, index, &y, &ldy)) return no();
  if (!called([&] { return p_gemm_i8((const int8_t*)x->data_ptr(), ldx, (const float*)sx->data_ptr(),
                (const int8_t*)w->data_ptr(), ldw, (const float*)sw->data_ptr(), (int)M, (int)N,
                (int)K, y.data_ptr(), (int)dtype, ldy, stream_of(index)); }))
    return no();
  return done(y, a[5]);
}

// linear_i8(x, w, w_scale, out)
PyObject* linear_i8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const at::Tensor *x, *w, *sw;
  int index = -1;
  int64_t M, N, K, KW, ldx, ldw, ldy;
  if (n != 4 || !cuda_tensor(a[0], &x, &index) || !cuda_tensor(a[1], &w, &index) ||
      !cuda_tensor(a[2], &sw, &index) || !on_current(index))
    return no();
  const int dtype = dtype_of(*x);
  if ((dtype != BCQ_F16 && dtype != BCQ_BF16) || !matrix(*x, &M, &K, &ldx) ||
      !codes(*w, &N, &KW, &ldw) || K != KW || !vector(*sw, at::kFloat, N))
    return no();
  at::Tensor y;
  if (!product_out(a[3], M, N, x->scalar_type(), *x, index, &y, &ldy)) return no();
  const size_t need = p_linear_bytes((int)M, (int)K);
  if (need == 0) return no();
  const c10::DataPtr ws = workspace(need);
  if (!called([&] { return p_linear_i8(x->data_ptr(), dtype, ldx, (const int8_t*)w->data_ptr(), ldw,
                  (const float*)sw->data_ptr(), (int)M, (int)N, (int)K, y.data_ptr(), ldy,
                  ws.get(), need, stream_of(index)); }))
    return no();
  return done(y, a[3]);
}

// The cache's tensors (arguments 0..3: k, k_param, v, v_param) and the tables
// (4..6: table, kv_len, cu or None).
struct Kv4Args {
  bcq_kv4 c;
  const int32_t *table, *kv_len, *cu;
  int B, W, index;
  const at::Tensor* k;
};
bool kv4_args(PyObject* const* a, Kv4Args* s) {
  const at::Tensor *k, *kp, *v, *vp, *table, *len, *cu;
  s->index = -1;
  if (!cuda_tensor(a[0], &k, &s->index) || !cuda_tensor(a[1], &kp, &s->index) ||
      !cuda_tensor(a[2], &v, &s->index) || !cuda_tensor(a[3], &vp, &s->index) ||
      !cuda_tensor(a[4], &table, &s->index) || !cuda_tensor(a[5], &len, &s->index) ||
      !on_current(s->index) || k->dim() != 4)
    return false;
  s->k = k;
  const int64_t groups = k->size(3) / 32;
  for (const at::Tensor* t : {k, v})
    if (t->scalar_type() != at::kByte || !t->is_contiguous() || t->sizes() != k->sizes()) return false;
  for (const at::Tensor* t : {kp, vp})
    if (t->scalar_type() != at::kHalf || !t->is_contiguous() ||
        t->numel() != k->size(0) * k->size(1) * k->size(2) * groups * 2)
      return false;
  if (k->size(0) > INT32_MAX || k->size(1) > INT32_MAX || k->size(2) > INT32_MAX ||
      table->scalar_type() != at::kInt || table->dim() != 2 || !table->is_contiguous() ||
      table->size(0) > INT32_MAX || table->size(1) > INT32_MAX)
    return false;
  s->c = {(uint8_t*)k->data_ptr(), (uint16_t*)kp->data_ptr(), (uint8_t*)v->data_ptr(),
          (uint16_t*)vp->data_ptr(), (int)k->size(0), (int)k->size(1), (int)k->size(2),
          (int)k->size(3) * 2};
  s->B = (int)table->size(0);
  s->W = (int)table->size(1);
  s->table = (const int32_t*)table->data_ptr();
  if (!vector(*len, at::kInt, s->B)) return false;
  s->kv_len = (const int32_t*)len->data_ptr();
  s->cu = nullptr;
  if (a[6] == Py_None) return true;
  if (!cuda_tensor(a[6], &cu, &s->index) || !vector(*cu, at::kInt, (int64_t)s->B + 1)) return false;
  s->cu = (const int32_t*)cu->data_ptr();
  return true;
}

// Rows [T][heads][D] with contiguous vectors on 16 bytes.
bool heads_of(const at::Tensor& t, int64_t D, int64_t* T, int64_t* H, int64_t* ld, int64_t* hd) {
  if ((t.scalar_type() != at::kHalf && t.scalar_type() != at::kBFloat16) || t.dim() != 3 ||
      t.size(2) != D || t.stride(2) != 1)
    return false;
  *T = t.size(0);
  *H = t.size(1);
  *ld = *T <= 1 ? 0 : t.stride(0);
  *hd = *H <= 1 ? 0 : t.stride(1);
  return *T <= INT32_MAX && *H <= INT32_MAX && *ld % 8 == 0 && *hd % 8 == 0 &&
         reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0;
}

// kv4_append(cache.., tables.., k, v)
PyObject* kv4_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Kv4Args s;
  const at::Tensor *k, *v;
  int64_t T, TV, H, HV, ldk, hdk, ldv, hdv;
  if (n != 9 || !kv4_args(a, &s) || !cuda_tensor(a[7], &k, &s.index) ||
      !cuda_tensor(a[8], &v, &s.index) || !heads_of(*k, s.c.head_dim, &T, &H, &ldk, &hdk) ||
      !heads_of(*v, s.c.head_dim, &TV, &HV, &ldv, &hdv) || k->scalar_type() != v->scalar_type() ||
      T != TV || H != s.c.heads || HV != s.c.heads || (!s.cu && T != s.B))
    return no();
  if (!called([&] { return p_kv4_append(&s.c, k->data_ptr(), ldk, hdk, v->data_ptr(), ldv, hdv, dtype_of(*k), (int)T,
                   s.table, s.W, s.kv_len, s.cu, s.B, stream_of(s.index)); }))
    return no();
  Py_RETURN_NONE;
}

// kv4_read(cache.., tables.., tokens, dtype)
PyObject* kv4_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Kv4Args s;
  if (n != 9 || !kv4_args(a, &s)) return no();
  const long T = PyLong_AsLong(a[7]), dtype = PyLong_AsLong(a[8]);
  if (T < 0 || T > INT32_MAX || (!s.cu && T != s.B)) {
    PyErr_Clear();
    return no();
  }
  const int64_t size[3] = {T, s.c.heads, s.c.head_dim};
  at::Tensor k = empty(*s.k, size, type_of(dtype)), v = empty(*s.k, size, type_of(dtype));
  if (!called([&] { return p_kv4_read(&s.c, k.data_ptr(), v.data_ptr(), (int)dtype, (int)T, s.table, s.W, s.kv_len,
                 s.cu, s.B, stream_of(s.index)); }))
    return no();
  return Py_BuildValue("(NN)", THPVariable_Wrap(k), THPVariable_Wrap(v));
}

// kv4_attention(cache.., tables.., q, max_q, max_kv, causal, window, scale, return_lse)
// (max_q, max_kv, scale: None for the defaults)
PyObject* kv4_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Kv4Args s;
  const at::Tensor* q;
  int64_t T, H, ld, hd;
  if (n != 14 || !kv4_args(a, &s) || !cuda_tensor(a[7], &q, &s.index) ||
      !heads_of(*q, s.c.head_dim, &T, &H, &ld, &hd) || (!s.cu && T != s.B) || T < 1)
    return no();
  const long max_q = a[8] == Py_None ? (s.cu ? (long)T : 1) : PyLong_AsLong(a[8]);
  const long max_kv = a[9] == Py_None ? (long)s.W * s.c.page_size : PyLong_AsLong(a[9]);
  const int causal = PyObject_IsTrue(a[10]), lse_too = PyObject_IsTrue(a[13]);
  const long window = PyLong_AsLong(a[11]);
  const double scale = a[12] == Py_None ? 1.0 / std::sqrt((double)s.c.head_dim) : PyFloat_AsDouble(a[12]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return no();
  }
  if (max_q < 1 || max_q > INT32_MAX || max_kv < 1 || max_kv > INT32_MAX || window < 0 ||
      window > INT32_MAX)
    return no();
  const int64_t D = s.c.head_dim;
  const size_t need = p_attention_bytes(&s.c, (int)T, (int)H, s.B, (int)max_q, (int)max_kv, (int)window);
  at::Tensor out = empty(*q, {T, H, D}, q->scalar_type()), lse;
  c10::DataPtr ws;
  if (lse_too) lse = empty(*q, {T, H}, at::kFloat);
  if (need) ws = workspace(need);
  if (!called([&] { return p_kv4_attention(&s.c, q->data_ptr(), ld, hd, dtype_of(*q), (int)T, (int)H, s.table, s.W,
                      s.kv_len, s.cu, s.B, (int)max_q, (int)max_kv, causal, (int)window,
                      (float)scale, out.data_ptr(), H * D, D, lse_too ? (float*)lse.data_ptr() : nullptr,
                      ws.get(), need, stream_of(s.index)); }))
    return no();
  if (!lse_too) return THPVariable_Wrap(out);
  return Py_BuildValue("(NN)", THPVariable_Wrap(out), THPVariable_Wrap(lse));
}

// bind(addresses): the entry points, in the order below.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "bind takes 8 addresses");
    return nullptr;
  }
  void* p[8];
  for (int i = 0; i < 8; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
      return nullptr;
    }
  }
  p_quantize_i8 = (decltype(p_quantize_i8))p[0];
  p_gemm_i8 = (decltype(p_gemm_i8))p[1];
  p_linear_bytes = (decltype(p_linear_bytes))p[2];
  p_linear_i8 = (decltype(p_linear_i8))p[3];
  p_kv4_append = (decltype(p_kv4_append))p[4];
  p_kv4_read = (decltype(p_kv4_read))p[5];
  p_attention_bytes = (decltype(p_attention_bytes))p[6];
  p_kv4_attention = (decltype(p_kv4_attention))p[7];
  Py_RETURN_NONE;
}

// No C++ exception leaves the module (an allocation that fails, a tensor that
// is none of the usual ones): the call is api.py's then.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guard(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (...) {
    PyErr_Clear();
    return no();
  }
}

#define BCQ_METHOD(f) {#f, (PyCFunction)(void (*)(void))guard<f>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {BCQ_METHOD(quantize_i8), BCQ_METHOD(gemm_i8), BCQ_METHOD(linear_i8),
                         BCQ_METHOD(kv4_append), BCQ_METHOD(kv4_read), BCQ_METHOD(kv4_attention),
                         {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast() { return PyModule_Create(&module); }
