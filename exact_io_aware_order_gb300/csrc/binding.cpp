// The calls of the 8-bit cache from Python without the interpreter's share of
// their cost.
//
// A decode step over a short cache takes the GPU a few microseconds; api.py's
// checks, three allocations and a ctypes call of 27 arguments take 18.  These
// functions make the same checks on the tensors themselves, allocate, and call
// the same C entry points.  They take the plain case only: ordinary tensors on
// the current device, the current stream, every check passed and the call
// accepted.  Anything else returns NotImplemented, and api.py goes through it
// again its own way, where each refusal has its message; so what a call means is
// written there.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "attn.h"

namespace {

// libattn.so's entry points, handed over by api.py.
decltype(&attn_cache_write_fp8) g_write = nullptr;
decltype(&attn_cache_read_fp8) g_read = nullptr;
decltype(&attn_decode_fp8) g_decode = nullptr;
decltype(&attn_decode_fp8_workspace_bytes) g_workspace_bytes = nullptr;

PyObject* refuse() { Py_RETURN_NOTIMPLEMENTED; }

// An ordinary tensor, or null: no subclass, and none of those that have a shape
// and a device but no storage (what torch.vmap or torch.func.grad hands its
// function is a plain torch.Tensor to Python).
const at::Tensor* tensor(PyObject* o) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor* t = &THPVariable_Unpack(o);
  return t->has_storage() ? t : nullptr;
}
bool is(const at::Tensor* t, at::ScalarType type, int64_t ndim, c10::Device dev) {
  return t && t->scalar_type() == type && t->dim() == ndim && t->device() == dev &&
         t->is_contiguous();
}
bool is_lens(const at::Tensor* t, c10::Device dev, int64_t n) {
  return is(t, at::kInt, 1, dev) && t->size(0) == n;
}
bool integer(PyObject* o, int64_t* x) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  *x = PyLong_AsLongLongAndOverflow(o, &over);
  return over == 0 && *x >= -2147483647LL && *x <= 2147483647LL;
}
bool number(PyObject* o, double* x) {
  if (PyFloat_CheckExact(o)) {
    *x = PyFloat_AS_DOUBLE(o);
    return true;
  }
  int64_t i;
  if (!integer(o, &i)) return false;
  *x = static_cast<double>(i);
  return true;
}
// data_ptr() may throw, so it is called with the interpreter's lock held.
template <typename T>
T* data(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

// A current device with a tensor on it.
bool on_current_device(const at::Tensor* t) {
  return t && t->is_cuda() && t->device().index() == c10::cuda::current_device();
}
void* stream_of(c10::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// The interpreter's lock given up for a scope, and taken again however it ends.
class WithoutLock {
 public:
  WithoutLock() : state_(PyEval_SaveThread()) {}
  ~WithoutLock() { PyEval_RestoreThread(state_); }
  WithoutLock(const WithoutLock&) = delete;
  WithoutLock& operator=(const WithoutLock&) = delete;

 private:
  PyThreadState* state_;
};

struct Cache {
  uint8_t *k, *v;
  float *ks, *vs;
  int32_t* table;
  int n_kv, d, block_size, max_blocks, num_blocks, capacity;
};

// k_cache, v_cache, k_scales, v_scales at a[0..3], the block table and block_size.
bool cache(PyObject* const* a, PyObject* table, PyObject* block_size, c10::Device dev,
           int64_t num_seqs, Cache* c) {
  const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]), *ks = tensor(a[2]), *vs = tensor(a[3]);
  const at::Tensor* bt = nullptr;
  if (!is(k, at::kByte, 4, dev) || !is(v, at::kByte, 4, dev) ||
      v->sizes() != k->sizes())
    return false;
  const int64_t n = k->size(0), rows = k->size(1), n_kv = k->size(2);
  int64_t bs = 0;
  if (block_size != Py_None && (!integer(block_size, &bs) || bs < 1)) return false;
  int64_t scale_dims;
  if (table != Py_None) {
    bt = tensor(table);
    if (!is(bt, at::kInt, 2, dev) || bt->size(0) != num_seqs || (bs && bs != rows))
      return false;
    const int64_t most = bt->size(1);
    // A table without columns has no address, which would mean a contiguous cache.
    if (most < 1 || rows > INT32_MAX || n > INT32_MAX || most > INT32_MAX ||
        rows * most > INT32_MAX)
      return false;
    c->block_size = (int)rows, c->max_blocks = (int)most, c->num_blocks = (int)n;
    c->capacity = (int)(rows * most);
    scale_dims = 2;
  } else {
    if (n != num_seqs || bs < 1 || rows > INT32_MAX) return false;
    c->block_size = (int)bs, c->max_blocks = 0, c->num_blocks = 0, c->capacity = (int)rows;
    scale_dims = 3;
  }
  for (const at::Tensor* s : {ks, vs}) {
    if (!is(s, at::kFloat, scale_dims, dev) || s->size(0) != n) return false;
    if (scale_dims == 2 ? s->size(1) != n_kv
                        : s->size(1) != (rows + bs - 1) / bs || s->size(2) != n_kv)
      return false;
  }
  if (n_kv > INT32_MAX || k->size(3) > INT32_MAX) return false;
  c->n_kv = (int)n_kv, c->d = (int)k->size(3);
  c->k = data<uint8_t>(k), c->v = data<uint8_t>(v);
  c->ks = data<float>(ks), c->vs = data<float>(vs), c->table = data<int32_t>(bt);
  return true;
}

// (heads, tokens, head_dim) or (tokens, heads, head_dim) bf16 rows.
bool is_rows(const at::Tensor* t, c10::Device dev) {
  return t && t->scalar_type() == at::kBFloat16 && t->dim() == 3 && t->device() == dev &&
         t->stride(2) == 1 && t->stride(0) % 8 == 0 && t->stride(1) % 8 == 0;
}

// cache_write_fp8(k_new, v_new, k_cache, v_cache, k_scales, v_scales, kv_lens,
// cu_seqlens, block_table, block_size)
PyObject* cache_write_fp8(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 10) return refuse();
  const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]), *lens = tensor(a[6]);
  if (!on_current_device(k) || !lens || lens->dim() != 1) return refuse();
  const c10::Device dev = k->device();
  const int64_t B = lens->size(0);
  Cache c;
  if (!is_rows(k, dev) || !is_rows(v, dev) || v->sizes() != k->sizes() ||
      !is_lens(lens, dev, B) || !cache(a + 2, a[8], a[9], dev, B, &c))
    return refuse();
  const bool packed = a[7] != Py_None;
  const at::Tensor* cu = packed ? tensor(a[7]) : nullptr;
  const int tok = packed ? 1 : 0, head = 1 - tok;
  const int64_t total = k->size(tok);
  if ((packed ? !is_lens(cu, dev, B + 1) : total != B) || k->size(head) != c.n_kv ||
      k->size(2) != c.d || total > INT32_MAX || B > INT32_MAX)
    return refuse();
  const attn_bf16 *kp = data<attn_bf16>(k), *vp = data<attn_bf16>(v);
  const int32_t *cup = data<int32_t>(cu), *lensp = data<int32_t>(lens);
  const int64_t kt = k->stride(tok), kh = k->stride(head), vt = v->stride(tok), vh = v->stride(head);
  void* stream = stream_of(dev);
  int st;
  {
    WithoutLock unlocked;
    st = g_write(kp, vp, kt, kh, vt, vh, c.k, c.v, c.ks, c.vs, c.table, cup, lensp, (int)B,
                 (int)total, c.n_kv, c.d, c.block_size, c.max_blocks, c.num_blocks, c.capacity,
                 stream);
  }
  if (st != ATTN_OK) return refuse();
  Py_RETURN_NONE;
}

// cache_read_fp8(k_cache, v_cache, k_scales, v_scales, cu_seqlens, total,
// block_table, starts, block_size), outputs allocated
PyObject* cache_read_fp8(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  int64_t total;
  if (n_args != 9 || !integer(a[5], &total) || total < 1) return refuse();
  const at::Tensor *k0 = tensor(a[0]), *cu = tensor(a[4]);
  if (!on_current_device(k0) || !cu || cu->dim() != 1 || cu->size(0) < 2) return refuse();
  const c10::Device dev = k0->device();
  const int64_t B = cu->size(0) - 1;
  const at::Tensor* starts = a[7] != Py_None ? tensor(a[7]) : nullptr;
  Cache c;
  if (!is_lens(cu, dev, B + 1) || (a[7] != Py_None && !is_lens(starts, dev, B)) ||
      !cache(a, a[6], a[8], dev, B, &c) || B > INT32_MAX)
    return refuse();
  const auto opt = at::TensorOptions().dtype(at::kBFloat16).device(dev);
  const at::Tensor k = at::empty({c.n_kv, total, c.d}, opt), v = at::empty({c.n_kv, total, c.d}, opt);
  attn_bf16 *kp = data<attn_bf16>(&k), *vp = data<attn_bf16>(&v);
  const int32_t *cup = data<int32_t>(cu), *startsp = data<int32_t>(starts);
  const int64_t head = total * c.d;
  void* stream = stream_of(dev);
  int st;
  {
    WithoutLock unlocked;
    st = g_read(c.k, c.v, c.ks, c.vs, kp, vp, c.d, head, c.d, head, c.table, cup, startsp, (int)B,
                (int)total, c.n_kv, c.d, c.block_size, c.max_blocks, c.num_blocks, c.capacity,
                stream);
  }
  if (st != ATTN_OK) return refuse();
  return Py_BuildValue("(NN)", THPVariable_Wrap(k), THPVariable_Wrap(v));
}

// decode_fp8(q, k_new, v_new, k_cache, v_cache, k_scales, v_scales, kv_lens,
// block_table, num_splits, max_kv_len, scale, out, lse, workspace, window_left,
// softcap, alibi_slopes, block_size)
PyObject* decode_fp8(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 19) return refuse();
  const at::Tensor *q = tensor(a[0]), *lens = tensor(a[7]);
  if (!on_current_device(q) || !is(q, at::kBFloat16, 3, q->device())) return refuse();
  const c10::Device dev = q->device();
  const int64_t B = q->size(0), n_q = q->size(1), d = q->size(2);
  Cache c;
  int64_t splits, window;
  double softcap, scale;
  if (B > INT32_MAX || n_q > INT32_MAX || !is_lens(lens, dev, B) ||
      !cache(a + 3, a[8], a[18], dev, B, &c) || c.d != d || !integer(a[9], &splits) ||
      splits < 0 || splits > ATTN_MAX_SPLITS || !integer(a[15], &window) ||
      !number(a[16], &softcap))
    return refuse();
  const at::Tensor *kn = nullptr, *vn = nullptr;
  if (a[1] != Py_None) {
    kn = tensor(a[1]);
    vn = tensor(a[2]);
    for (const at::Tensor* t : {kn, vn})
      if (!is(t, at::kBFloat16, 3, dev) || t->size(0) != B || t->size(1) != c.n_kv ||
          t->size(2) != d)
        return refuse();
  }
  int64_t max_len = c.capacity;
  if (a[10] != Py_None) {
    int64_t x;
    if (!integer(a[10], &x) || (a[8] == Py_None && x > c.capacity)) return refuse();
    if (a[8] != Py_None) max_len = x;
  }
  if (a[11] == Py_None) scale = 1.0 / std::sqrt((double)d);
  else if (!number(a[11], &scale)) return refuse();
  const at::Tensor* slopes = nullptr;
  if (a[17] != Py_None) {
    slopes = tensor(a[17]);
    if (!is(slopes, at::kFloat, 1, dev) || slopes->size(0) != n_q) return refuse();
  }
  at::Tensor out, lse, ws;
  if (a[12] != Py_None) {
    const at::Tensor* t = tensor(a[12]);
    if (!is(t, at::kFloat, 3, dev) || t->sizes() != q->sizes()) return refuse();
    out = *t;
  }
  if (a[13] != Py_None) {
    const at::Tensor* t = tensor(a[13]);
    if (!is(t, at::kFloat, 2, dev) || t->size(0) != B || t->size(1) != n_q) return refuse();
    lse = *t;
  }
  const auto f32 = at::TensorOptions().dtype(at::kFloat).device(dev);
  if (!out.defined()) out = at::empty({B, n_q, d}, f32);
  if (!lse.defined()) lse = at::empty({B, n_q}, f32);
  if (a[14] != Py_None) {
    const at::Tensor* t = tensor(a[14]);
    if (!is(t, at::kByte, 1, dev)) return refuse();
    ws = *t;
  } else {
    const size_t n = g_workspace_bytes((int)splits, (int)B, (int)n_q, c.n_kv, c.d, (int)max_len,
                                       (int)window);
    if (n > 0) ws = at::empty({(int64_t)n}, f32.dtype(at::kByte));
  }
  const attn_bf16 *qp = data<attn_bf16>(q), *knp = data<attn_bf16>(kn), *vnp = data<attn_bf16>(vn);
  const int32_t* lensp = data<int32_t>(lens);
  const float* slopesp = data<float>(slopes);
  float *outp = data<float>(&out), *lsep = data<float>(&lse);
  void* wsp = ws.defined() ? ws.data_ptr() : nullptr;
  const size_t wsn = ws.defined() ? (size_t)ws.numel() : 0;
  void* stream = stream_of(dev);
  int st;
  {
    WithoutLock unlocked;
    st = g_decode(qp, knp, vnp, c.k, c.v, c.ks, c.vs, c.table, lensp, (int)splits, wsp, wsn, outp,
                  lsep, (int)B, (int)n_q, c.n_kv, c.d, c.block_size, c.max_blocks, c.num_blocks,
                  (int)max_len, (float)scale, (int)window, (float)softcap, slopesp, stream);
  }
  if (st != ATTN_OK) return refuse();
  return Py_BuildValue("(NN)", THPVariable_Wrap(out), THPVariable_Wrap(lse));
}

// init(addresses of attn_cache_write_fp8, attn_cache_read_fp8, attn_decode_fp8,
// attn_decode_fp8_workspace_bytes)
PyObject* init(PyObject*, PyObject* args) {
  unsigned long long w, r, d, b;
  if (!PyArg_ParseTuple(args, "KKKK", &w, &r, &d, &b)) return nullptr;
  g_write = reinterpret_cast<decltype(g_write)>(w);
  g_read = reinterpret_cast<decltype(g_read)>(r);
  g_decode = reinterpret_cast<decltype(g_decode)>(d);
  g_workspace_bytes = reinterpret_cast<decltype(g_workspace_bytes)>(b);
  Py_RETURN_NONE;
}

// takes(x): whether x is a tensor whose memory these functions would look at (the
// tests ask, on tensors that no GPU is needed for).
PyObject* takes(PyObject*, PyObject* x) { return PyBool_FromLong(tensor(x) != nullptr); }

// No C++ exception leaves for the interpreter.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (...) {
    return refuse();
  }
}

PyMethodDef kMethods[] = {
    {"init", init, METH_VARARGS, nullptr},
    {"takes", takes, METH_O, nullptr},
    {"cache_write_fp8", (PyCFunction)(void (*)(void))guarded<cache_write_fp8>, METH_FASTCALL, nullptr},
    {"cache_read_fp8", (PyCFunction)(void (*)(void))guarded<cache_read_fp8>, METH_FASTCALL, nullptr},
    {"decode_fp8", (PyCFunction)(void (*)(void))guarded<decode_fp8>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
