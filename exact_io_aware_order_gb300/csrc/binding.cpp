// The calls of the 8-bit cache, of rotary positions and of a decode step with drafted
// tokens from Python without the interpreter's share of their cost.
//
// A decode step over a short cache takes the GPU a few microseconds; api.py's
// checks, three allocations and a ctypes call of 27 arguments take 18.  These
// functions make the same checks on the tensors themselves, allocate, and call
// the same C entry points.  They take the plain case only: ordinary tensors on
// the current device, the current stream, every check passed and the call
// accepted.  Anything else returns NotImplemented, and api.py or drafts.py goes
// through it again its own way, where each refusal has its message; so what a call
// means is written there.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
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
decltype(&attn_rope) g_rope = nullptr;
decltype(&attn_cache_append) g_append = nullptr;
decltype(&attn_decode_tree) g_tree = nullptr;
decltype(&attn_decode_tree_workspace_bytes) g_tree_bytes = nullptr;
decltype(&attn_verify_tree) g_verify = nullptr;

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

bool truth(PyObject* o, int* x) {
  if (!PyBool_Check(o)) return false;
  *x = o == Py_True;
  return true;
}
// A vector of n entries (any number for n < 0).
bool is_vector(const at::Tensor* t, at::ScalarType type, c10::Device dev, int64_t n) {
  return is(t, type, 1, dev) && (n < 0 ? t->size(0) <= INT32_MAX : t->size(0) == n);
}
// bf16 rows on dev: values of a row contiguous, other strides multiples of 8.
bool is_strided(const at::Tensor* t, c10::Device dev, int64_t ndim) {
  if (!t || t->scalar_type() != at::kBFloat16 || t->dim() != ndim || t->device() != dev ||
      t->stride(ndim - 1) != 1)
    return false;
  for (int64_t i = 0; i < ndim; ++i)
    if ((i < ndim - 1 && t->stride(i) % 8 != 0) || t->size(i) > INT32_MAX) return false;
  return true;
}

// rope(q, k, inv_freq, positions, interleaved, inverse, magnitude, q_out, k_out)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 9) return refuse();
  const at::Tensor *q = tensor(a[0]), *f = tensor(a[2]);
  if (!on_current_device(q) || (q->dim() != 3 && q->dim() != 4)) return refuse();
  const c10::Device dev = q->device();
  const int64_t nd = q->dim(), B = nd == 4 ? q->size(0) : 1, n = q->size(nd - 2), d = q->size(nd - 1);
  const at::Tensor* k = a[1] != Py_None ? tensor(a[1]) : nullptr;
  int inter, inverse;
  double magnitude;
  if (!is_strided(q, dev, nd) || !is_vector(f, at::kDouble, dev, -1) || f->size(0) > 1024 ||
      !truth(a[4], &inter) || !truth(a[5], &inverse) || !number(a[6], &magnitude))
    return refuse();
  if (a[1] != Py_None && (!is_strided(k, dev, nd) || (nd == 4 && k->size(0) != B) ||
                          k->size(nd - 2) != n || k->size(nd - 1) != d))
    return refuse();
  const at::Tensor* pos = nullptr;
  int64_t pos_stride = 0;
  if (a[3] != Py_None) {
    pos = tensor(a[3]);
    if (!pos) return refuse();
    if (pos->dim() == 2 && nd == 4) {
      if (!is(pos, at::kInt, 2, dev) || pos->size(0) != B || pos->size(1) != n) return refuse();
      pos_stride = n;
    } else if (!is_vector(pos, at::kInt, dev, n)) {
      return refuse();
    }
  }
  at::Tensor out[2];
  const at::Tensor* in[2] = {q, k};
  for (int i = 0; i < 2; ++i) {
    PyObject* o = a[7 + i];
    if (o != Py_None) {
      const at::Tensor* t = tensor(o);
      if (!in[i] || !is_strided(t, dev, nd) || t->sizes() != in[i]->sizes()) return refuse();
      out[i] = *t;
    } else if (in[i]) {
      out[i] = at::empty_like(*in[i]);
      if (!is_strided(&out[i], dev, nd)) return refuse();
    }
  }
  const attn_bf16* src[2] = {data<attn_bf16>(q), data<attn_bf16>(k)};
  attn_bf16* dst[2] = {data<attn_bf16>(&out[0]), k ? data<attn_bf16>(&out[1]) : nullptr};
  int64_t st[2][2][3] = {};
  for (int i = 0; i < (k ? 2 : 1); ++i)
    for (int64_t x = 0; x < nd - 1; ++x) {
      st[i][0][x + 4 - nd] = in[i]->stride(x);
      st[i][1][x + 4 - nd] = out[i].stride(x);
    }
  const double* fp = data<double>(f);
  const int32_t* pp = data<int32_t>(pos);
  const int rot = 2 * (int)f->size(0);
  void* stream = stream_of(dev);
  int status;
  {
    WithoutLock unlocked;
    status = g_rope(src[0], st[0][0][0], st[0][0][1], st[0][0][2], dst[0], st[0][1][0], st[0][1][1],
                    st[0][1][2], src[1], st[1][0][0], st[1][0][1], st[1][0][2], dst[1], st[1][1][0],
                    st[1][1][1], st[1][1][2], fp, pp, pos_stride, (int)B, (int)q->size(nd - 3),
                    k ? (int)k->size(nd - 3) : 0, (int)n, (int)d, rot, inter, inverse,
                    (float)magnitude, stream);
  }
  if (status != ATTN_OK) return refuse();
  if (!k) return Py_BuildValue("(NO)", THPVariable_Wrap(out[0]), Py_None);
  return Py_BuildValue("(NN)", THPVariable_Wrap(out[0]), THPVariable_Wrap(out[1]));
}

struct Cache16 {
  attn_bf16 *k, *v;
  int32_t* table;
  int n_kv, d, block_size, max_blocks, num_blocks, capacity;
};

// A bf16 cache of num_seqs sequences.
bool cache16(PyObject* ko, PyObject* vo, PyObject* to, c10::Device dev, int64_t num_seqs, Cache16* c) {
  const at::Tensor *k = tensor(ko), *v = tensor(vo);
  if (!is(k, at::kBFloat16, 4, dev) || !is(v, at::kBFloat16, 4, dev) || v->sizes() != k->sizes())
    return false;
  const int64_t n = k->size(0), rows = k->size(1);
  if (n > INT32_MAX || rows > INT32_MAX || k->size(2) > INT32_MAX || k->size(3) > INT32_MAX)
    return false;
  const at::Tensor* t = nullptr;
  if (to != Py_None) {
    t = tensor(to);
    if (!is(t, at::kInt, 2, dev) || t->size(0) != num_seqs || t->size(1) < 1 ||
        t->size(1) > INT32_MAX || rows * t->size(1) > INT32_MAX)
      return false;
    c->block_size = (int)rows, c->max_blocks = (int)t->size(1), c->num_blocks = (int)n;
    c->capacity = (int)(rows * t->size(1));
  } else {
    if (n != num_seqs) return false;
    c->block_size = c->max_blocks = c->num_blocks = 0;
    c->capacity = (int)rows;
  }
  c->n_kv = (int)k->size(2), c->d = (int)k->size(3);
  c->k = data<attn_bf16>(k), c->v = data<attn_bf16>(v), c->table = data<int32_t>(t);
  return true;
}

// cache_append(k_new, v_new, k_cache, v_cache, kv_lens, cu_seqlens, block_table, inv_freq,
// positions, q, interleaved, magnitude, q_out)
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 13) return refuse();
  const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]), *lens = tensor(a[4]);
  if (!on_current_device(k) || !lens || lens->dim() != 1) return refuse();
  const c10::Device dev = k->device();
  const int64_t B = lens->size(0);
  Cache16 c;
  int inter;
  double magnitude;
  if (!is_strided(k, dev, 3) || !is_strided(v, dev, 3) || v->sizes() != k->sizes() ||
      !is_vector(lens, at::kInt, dev, -1) || !cache16(a[2], a[3], a[6], dev, B, &c) ||
      !truth(a[10], &inter) || !number(a[11], &magnitude))
    return refuse();
  const bool packed = a[5] != Py_None;
  const int tok = packed ? 1 : 0, head = 1 - tok;
  const int64_t total = k->size(tok);
  const at::Tensor* cu = packed ? tensor(a[5]) : nullptr;
  if ((packed ? !is_vector(cu, at::kInt, dev, B + 1) : total != B) || k->size(head) != c.n_kv ||
      k->size(2) != c.d)
    return refuse();
  const at::Tensor *f = nullptr, *pos = nullptr, *q = nullptr;
  if (a[7] != Py_None) {
    f = tensor(a[7]);
    if (!is_vector(f, at::kDouble, dev, -1) || f->size(0) > 1024) return refuse();
  }
  if (a[8] != Py_None) {
    pos = tensor(a[8]);
    if (!is_vector(pos, at::kInt, dev, total)) return refuse();
  }
  at::Tensor out;
  if (a[9] != Py_None) {
    q = tensor(a[9]);
    if (!f || !is_strided(q, dev, 3) || q->size(tok) != total || q->size(2) != c.d) return refuse();
    if (a[12] != Py_None) {
      const at::Tensor* t = tensor(a[12]);
      if (!is_strided(t, dev, 3) || t->sizes() != q->sizes()) return refuse();
      out = *t;
    } else {
      out = at::empty_like(*q);
      if (!is_strided(&out, dev, 3)) return refuse();
    }
  } else if (a[12] != Py_None) {
    return refuse();
  }
  const attn_bf16 *kp = data<attn_bf16>(k), *vp = data<attn_bf16>(v), *qp = data<attn_bf16>(q);
  attn_bf16* op = q ? data<attn_bf16>(&out) : nullptr;
  const int32_t *cup = data<int32_t>(cu), *lensp = data<int32_t>(lens), *pp = data<int32_t>(pos);
  const double* fp = data<double>(f);
  const int64_t kt = k->stride(tok), kh = k->stride(head), vt = v->stride(tok), vh = v->stride(head);
  const int64_t qt = q ? q->stride(tok) : 0, qh = q ? q->stride(head) : 0;
  const int64_t ot = q ? out.stride(tok) : 0, oh = q ? out.stride(head) : 0;
  const int n_q = q ? (int)q->size(head) : 0, rot = f ? 2 * (int)f->size(0) : 0;
  void* stream = stream_of(dev);
  int status;
  {
    WithoutLock unlocked;
    status = g_append(kp, vp, kt, kh, vt, vh, qp, qt, qh, op, ot, oh, c.k, c.v, c.table, cup, lensp,
                      fp, pp, (int)B, (int)total, n_q, c.n_kv, c.d, rot, inter, (float)magnitude,
                      c.block_size, c.max_blocks, c.num_blocks, c.capacity, stream);
  }
  if (status != ATTN_OK) return refuse();
  if (!q) Py_RETURN_NONE;
  return THPVariable_Wrap(out);
}

// An output that is given (checked) or allocated; false where it is not as it should be.
bool output(PyObject* o, at::ScalarType type, c10::Device dev, at::IntArrayRef shape, at::Tensor* t) {
  if (o == Py_None) {
    *t = at::empty(shape, at::TensorOptions().dtype(type).device(dev));
    return true;
  }
  const at::Tensor* x = tensor(o);
  if (!is(x, type, (int64_t)shape.size(), dev) || x->sizes() != shape) return false;
  *t = *x;
  return true;
}

// decode_tree(q, k_cache, v_cache, kv_lens, cu_nodes, tree_mask, block_table, max_kv_len, scale,
// out, lse, workspace, window_left, softcap, alibi_slopes, bf16 output)
PyObject* decode_tree(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 16) return refuse();
  const at::Tensor *q = tensor(a[0]), *lens = tensor(a[3]), *cu = tensor(a[4]);
  if (!on_current_device(q) || !is(q, at::kBFloat16, 3, q->device()) || !lens || lens->dim() != 1)
    return refuse();
  const c10::Device dev = q->device();
  const int64_t B = lens->size(0), total = q->size(0), n_q = q->size(1), d = q->size(2);
  Cache16 c;
  int64_t window;
  int bf16;
  double softcap, scale;
  if (total > INT32_MAX || n_q > INT32_MAX || !is_vector(lens, at::kInt, dev, -1) ||
      !is_vector(cu, at::kInt, dev, B + 1) || !cache16(a[1], a[2], a[6], dev, B, &c) || c.d != d ||
      !integer(a[12], &window) || !number(a[13], &softcap) || !truth(a[15], &bf16))
    return refuse();
  int64_t max_len = c.capacity;
  if (a[7] != Py_None) {
    int64_t x;
    if (!integer(a[7], &x) || (a[6] == Py_None && x > c.capacity)) return refuse();
    if (a[6] != Py_None) max_len = x;
  }
  if (a[8] == Py_None) scale = 1.0 / std::sqrt((double)d);
  else if (!number(a[8], &scale)) return refuse();
  const at::Tensor *mask = nullptr, *slopes = nullptr;
  if (a[5] != Py_None) {
    mask = tensor(a[5]);
    if (!is_vector(mask, at::kLong, dev, total)) return refuse();
  }
  if (a[14] != Py_None) {
    slopes = tensor(a[14]);
    if (!is_vector(slopes, at::kFloat, dev, n_q)) return refuse();
  }
  at::Tensor out, lse, ws;
  if (!output(a[9], bf16 ? at::kBFloat16 : at::kFloat, dev, {total, n_q, d}, &out) ||
      !output(a[10], at::kFloat, dev, {total, n_q}, &lse))
    return refuse();
  if (a[11] != Py_None) {
    const at::Tensor* t = tensor(a[11]);
    if (!is(t, at::kByte, 1, dev)) return refuse();
    ws = *t;
  } else {
    const size_t n = g_tree_bytes((int)B, (int)total, (int)n_q, c.n_kv, c.d, (int)max_len, (int)window);
    if (n > 0) ws = at::empty({(int64_t)n}, at::TensorOptions().dtype(at::kByte).device(dev));
  }
  const attn_bf16* qp = data<attn_bf16>(q);
  const int32_t *lensp = data<int32_t>(lens), *cup = data<int32_t>(cu);
  const int64_t* maskp = data<int64_t>(mask);
  const float* slopesp = data<float>(slopes);
  void *outp = out.data_ptr(), *wsp = ws.defined() ? ws.data_ptr() : nullptr;
  float* lsep = data<float>(&lse);
  const size_t wsn = ws.defined() ? (size_t)ws.numel() : 0;
  void* stream = stream_of(dev);
  int status;
  {
    WithoutLock unlocked;
    status = g_tree(qp, c.k, c.v, c.table, lensp, cup, maskp, wsp, wsn, outp, lsep, (int)B,
                    (int)total, (int)n_q, c.n_kv, c.d, c.block_size, c.max_blocks, c.num_blocks,
                    (int)max_len, (float)scale, (int)window, (float)softcap, slopesp,
                    bf16 ? ATTN_TREE_OUT_BF16 : 0u, stream);
  }
  if (status != ATTN_OK) return refuse();
  return Py_BuildValue("(NN)", THPVariable_Wrap(out), THPVariable_Wrap(lse));
}

// fp32 (total, vocab) with contiguous rows.
bool is_probs(const at::Tensor* t, c10::Device dev) {
  return t && t->scalar_type() == at::kFloat && t->dim() == 2 && t->device() == dev &&
         t->size(0) <= INT32_MAX && t->size(1) <= INT32_MAX && (t->stride(1) == 1 || t->size(1) == 1);
}

// verify_tree(target_probs, draft_tokens, parents, cu_nodes, u_accept, u_sample, draft_probs,
// num_accepted, path, next_token)
PyObject* verify_tree(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 10) return refuse();
  const at::Tensor *p = tensor(a[0]), *tok = tensor(a[1]), *par = tensor(a[2]), *cu = tensor(a[3]),
                   *u = tensor(a[4]), *ul = tensor(a[5]);
  if (!on_current_device(p) || !is_probs(p, p->device()) || !cu || cu->dim() != 1 || cu->size(0) < 2)
    return refuse();
  const c10::Device dev = p->device();
  const int64_t total = p->size(0), V = p->size(1), B = cu->size(0) - 1;
  const at::Tensor* q = nullptr;
  if (a[6] != Py_None) {
    q = tensor(a[6]);
    if (!is_probs(q, dev) || q->sizes() != p->sizes()) return refuse();
  }
  at::Tensor out[3];
  if (!is_vector(cu, at::kInt, dev, -1) || !is_vector(tok, at::kInt, dev, total) ||
      !is_vector(par, at::kInt, dev, total) || !is_vector(u, at::kFloat, dev, total) ||
      !is_vector(ul, at::kFloat, dev, B) || !output(a[7], at::kInt, dev, {B}, &out[0]) ||
      !output(a[8], at::kInt, dev, {B, 64}, &out[1]) || !output(a[9], at::kInt, dev, {B}, &out[2]))
    return refuse();
  const float *pp = data<float>(p), *qp = data<float>(q), *up = data<float>(u), *ulp = data<float>(ul);
  const int32_t *tp = data<int32_t>(tok), *rp = data<int32_t>(par), *cup = data<int32_t>(cu);
  int32_t* op[3];
  for (int i = 0; i < 3; ++i) op[i] = data<int32_t>(&out[i]);
  const int64_t ps = total > 1 ? p->stride(0) : V, qs = !q ? 0 : total > 1 ? q->stride(0) : V;
  void* stream = stream_of(dev);
  int status;
  {
    WithoutLock unlocked;
    status = g_verify(pp, ps, qp, qs, tp, rp, cup, up, ulp, op[0], op[1], op[2], (int)B, (int)total,
                      (int)V, stream);
  }
  if (status != ATTN_OK) return refuse();
  return Py_BuildValue("(NNN)", THPVariable_Wrap(out[0]), THPVariable_Wrap(out[1]),
                       THPVariable_Wrap(out[2]));
}

// init(addresses of attn_cache_write_fp8, attn_cache_read_fp8, attn_decode_fp8,
// attn_decode_fp8_workspace_bytes, attn_rope, attn_cache_append, attn_decode_tree,
// attn_decode_tree_workspace_bytes, attn_verify_tree)
PyObject* init(PyObject*, PyObject* args) {
  unsigned long long w, r, d, b, o, p, t, n, v;
  if (!PyArg_ParseTuple(args, "KKKKKKKKK", &w, &r, &d, &b, &o, &p, &t, &n, &v)) return nullptr;
  g_write = reinterpret_cast<decltype(g_write)>(w);
  g_read = reinterpret_cast<decltype(g_read)>(r);
  g_decode = reinterpret_cast<decltype(g_decode)>(d);
  g_workspace_bytes = reinterpret_cast<decltype(g_workspace_bytes)>(b);
  g_rope = reinterpret_cast<decltype(g_rope)>(o);
  g_append = reinterpret_cast<decltype(g_append)>(p);
  g_tree = reinterpret_cast<decltype(g_tree)>(t);
  g_tree_bytes = reinterpret_cast<decltype(g_tree_bytes)>(n);
  g_verify = reinterpret_cast<decltype(g_verify)>(v);
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
    {"rope", (PyCFunction)(void (*)(void))guarded<rope>, METH_FASTCALL, nullptr},
    {"cache_append", (PyCFunction)(void (*)(void))guarded<cache_append>, METH_FASTCALL, nullptr},
    {"decode_tree", (PyCFunction)(void (*)(void))guarded<decode_tree>, METH_FASTCALL, nullptr},
    {"verify_tree", (PyCFunction)(void (*)(void))guarded<verify_tree>, METH_FASTCALL, nullptr},
    {"decode_fp8", (PyCFunction)(void (*)(void))guarded<decode_fp8>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
