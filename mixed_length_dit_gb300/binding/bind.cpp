// The short way from PyTorch tensors to the C ABI for the calls of paged.py.
//
// A call on a single token is bound by the host: the checks and the marshalling
// of the long way, in Python, took three times the launch itself.  Here they are
// made on the tensors directly (us a call, the long way and this one: rotation
// of 1531 tokens 20.3 and 8.2, append of a token to each of 64 sequences 21.9 and 6.1, attention of
// one token 28.1 and 14.4, a fork with three copies of its tables 47 and 28).
//
// A call that is all as it should be (tensors of the right shapes, types and
// layout on the current device, its own stream) goes to the library at once.
// Anything else returns None without having done anything, and paged.py takes
// the long way: it says what is wrong, or handles what is unusual.  Status codes
// of the library come back as ints.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>

#include "zl_attn.h"

namespace {

// An argument that has to be a tensor; null if it is not.
const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// The arguments of one call.  `ok` turns false with the first that does not
// read as asked.
struct Args {
  PyObject* const* v;
  Py_ssize_t n, i = 0;
  bool ok = true;

  PyObject* next() {
    if (i >= n) ok = false;
    return ok ? v[i++] : Py_None;
  }
  const at::Tensor* t() {
    const at::Tensor* x = tensor(next());
    if (!x) ok = false;
    return x;
  }
  // a tensor or None
  const at::Tensor* maybe() {
    PyObject* o = next();
    if (o == Py_None) return nullptr;
    const at::Tensor* x = tensor(o);
    if (!x) ok = false;
    return x;
  }
  int64_t integer() {
    PyObject* o = next();
    if (!ok || !PyLong_Check(o)) {
      ok = false;
      return 0;
    }
    int overflow = 0;
    const int64_t x = PyLong_AsLongLongAndOverflow(o, &overflow);
    if (overflow) ok = false;
    return x;
  }
  int32_t int32() {
    const int64_t x = integer();
    if (x < INT32_MIN || x > INT32_MAX) ok = false;
    return static_cast<int32_t>(x);
  }
  void* pointer() { return reinterpret_cast<void*>(integer()); }
  bool truth() {
    const int x = PyObject_IsTrue(next());
    if (x < 0) {
      PyErr_Clear();
      ok = false;
    }
    return x > 0;
  }
  bool done() const { return ok && i == n; }
};

// [tokens, heads, dim] of `type` on the device, heads and columns contiguous;
// the elements between tokens, or -1.
int64_t rows(const at::Tensor& t, int64_t tokens, int64_t heads, int64_t dim, at::ScalarType type, c10::Device dev) {
  if (t.dim() != 3 || t.scalar_type() != type || t.device() != dev) return -1;
  const auto s = t.sizes();
  if (s[0] != tokens || s[1] != heads || s[2] != dim) return -1;
  const auto st = t.strides();
  if (st[2] != 1 || (heads > 1 && st[1] != dim)) return -1;
  return tokens > 1 ? st[0] : heads * dim;
}

bool ints(const at::Tensor& t, c10::Device dev) {
  return t.scalar_type() == at::kInt && t.device() == dev && t.is_contiguous();
}

// The tensors' device, if calls go there now.
bool current(c10::Device dev) { return dev.is_cuda() && dev.index() == c10::cuda::current_device(); }

void* stream_of(c10::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

at::Tensor fresh(const at::Tensor& like, at::IntArrayRef sizes, at::ScalarType type) {
  return at::empty(sizes, like.options().dtype(type).requires_grad(false));
}

// Other Python threads run while a call allocates and launches (a launch can
// wait for a full queue).  The arguments stay: their caller holds them.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

PyObject* none() { Py_RETURN_NONE; }
PyObject* status(zl_status st) { return PyLong_FromLong(st); }

struct Scratch {
  void* p = nullptr;
  size_t bytes = 0;
  bool ok = true;
  Scratch(const at::Tensor* t, c10::Device dev) {
    if (!t) return;
    ok = t->device() == dev && t->is_contiguous();
    p = t->data_ptr();
    bytes = t->nbytes();
  }
};

// bwd, q, k | None, positions, plan, axes of the plan, its head_dim
PyObject* rope(Args& a) {
  const bool bwd = a.truth();
  const at::Tensor* q = a.t();
  const at::Tensor* k = a.maybe();
  const at::Tensor* pos = a.t();
  const auto* plan = static_cast<const zl_rope_t*>(a.pointer());
  const int64_t axes = a.integer(), hd = a.integer();
  if (!a.done() || q->dim() != 3 || (k && k->dim() != 3) || !current(q->device())) return none();
  const c10::Device dev = q->device();
  const at::ScalarType type = q->scalar_type();
  if (type != at::kBFloat16 && type != at::kFloat) return none();
  const int64_t tokens = q->size(0), nq = q->size(1), nk = k ? k->size(1) : 0;
  const int64_t qs = rows(*q, tokens, nq, hd, type, dev), ks = k ? rows(*k, tokens, nk, hd, type, dev) : 0;
  if (tokens == 0 || nq > INT32_MAX || nk > INT32_MAX || qs < 0 || ks < 0 || !plan) return none();
  if (pos->scalar_type() != at::kInt || pos->device() != dev) return none();
  const bool flat = axes == 1 && pos->dim() == 1 && pos->size(0) == tokens;
  if (!flat && !(pos->dim() == 2 && pos->size(0) == axes && pos->size(1) == tokens)) return none();
  if (tokens > 1 && pos->strides().back() != 1) return none();
  at::Tensor qo, ko;
  zl_status st;
  {
    Unlocked u;
    qo = fresh(*q, {tokens, nq, hd}, type);
    if (k) ko = fresh(*q, {tokens, nk, hd}, type);
    const auto fn = bwd ? zl_rope_bwd : zl_rope_fwd;
    st = fn(plan, q->data_ptr(), qs, k ? k->data_ptr() : nullptr, ks, pos->data_ptr<int32_t>(),
            axes > 1 ? pos->stride(0) : tokens, tokens, static_cast<int32_t>(nq), static_cast<int32_t>(nk),
            type == at::kBFloat16 ? ZL_BF16 : ZL_FP32, qo.data_ptr(), nq * hd, k ? ko.data_ptr() : nullptr, nk * hd,
            stream_of(dev));
  }
  if (st != ZL_OK) return status(st);
  PyObject* x = THPVariable_Wrap(std::move(qo));
  PyObject* y = k ? THPVariable_Wrap(std::move(ko)) : none();
  PyObject* r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

// k_pages, v_pages, page_table, kv_lens of `seqs` sequences, checked.
bool cache_of(Args& a, zl_paged_cache_t* c, c10::Device* dev) {
  const at::Tensor* kp = a.t();
  const at::Tensor* vp = a.t();
  const at::Tensor* table = a.t();
  const at::Tensor* lens = a.t();
  if (!a.ok || kp->dim() != 4 || table->dim() != 2 || lens->dim() != 1 || !current(kp->device())) return false;
  *dev = kp->device();
  if (kp->scalar_type() != at::kBFloat16 || vp->scalar_type() != at::kBFloat16 || vp->device() != *dev) return false;
  if (kp->sizes() != vp->sizes() || !kp->is_contiguous() || !vp->is_contiguous()) return false;
  if (!ints(*table, *dev) || !ints(*lens, *dev) || lens->size(0) != table->size(0)) return false;
  for (const int64_t x : {kp->size(0), kp->size(1), kp->size(2), kp->size(3), table->size(0), table->size(1)})
    if (x > INT32_MAX) return false;
  *c = zl_paged_cache_t{kp->data_ptr(), vp->data_ptr(), table->data_ptr<int32_t>(), lens->data_ptr<int32_t>(),
                        static_cast<int32_t>(table->size(1)), static_cast<int32_t>(kp->size(0)),
                        static_cast<int32_t>(kp->size(2)), static_cast<int32_t>(kp->size(1)),
                        static_cast<int32_t>(kp->size(3)), 0};
  return true;
}

// k, v, the cache, its tables, cu (address, entries, last), q | None, plan | 0;
// STATUS: and the status of the extend before it
template <bool STATUS>
PyObject* append(Args& a) {
  const at::Tensor* k = a.t();
  const at::Tensor* v = a.t();
  zl_paged_cache_t c;
  c10::Device dev(c10::kCPU);
  const at::Tensor* lens = a.ok && a.i + 3 < a.n ? tensor(a.v[a.i + 3]) : nullptr;
  if (!lens || !cache_of(a, &c, &dev)) return none();
  const auto* cu = static_cast<const int32_t*>(a.pointer());
  const int32_t n = a.int32();
  const int64_t tokens = a.integer();
  const at::Tensor* q = a.maybe();
  const auto* plan = static_cast<const zl_rope_t*>(a.pointer());
  const at::Tensor* extended = STATUS ? a.t() : nullptr;
  if (!a.done() || lens->size(0) != n - 1 || tokens == 0) return none();
  if (extended && (!ints(*extended, dev) || extended->dim() != 1 || extended->size(0) != 1)) return none();
  const int64_t ks = rows(*k, tokens, c.num_kv_heads, c.head_dim, at::kBFloat16, dev);
  const int64_t vs = rows(*v, tokens, c.num_kv_heads, c.head_dim, at::kBFloat16, dev);
  int64_t qs = 0, nq = 0;
  if (q) {
    if (q->dim() != 3) return none();
    nq = q->size(1);
    qs = rows(*q, tokens, nq, c.head_dim, at::kBFloat16, dev);
  }
  if (ks < 0 || vs < 0 || qs < 0 || nq > INT32_MAX) return none();
  at::Tensor qo;
  zl_status st;
  {
    Unlocked u;
    if (q) qo = fresh(*q, {tokens, nq, c.head_dim}, at::kBFloat16);
    st = zl_paged_append_ex(&c, k->data_ptr(), ks, v->data_ptr(), vs, cu, n - 1, plan, nullptr, 0,
                            q ? q->data_ptr() : nullptr, qs, static_cast<int32_t>(nq), q ? qo.data_ptr() : nullptr,
                            nq * c.head_dim, extended ? extended->data_ptr<int32_t>() : nullptr, stream_of(dev));
  }
  if (st != ZL_OK) return status(st);
  // what was asked for, in a tuple: None alone means the long way
  PyObject* x = q ? THPVariable_Wrap(std::move(qo)) : none();
  PyObject* r = x ? PyTuple_Pack(1, x) : nullptr;
  Py_XDECREF(x);
  return r;
}

// q, the cache, its tables, cu (address, entries, last), max_kv_len, causal,
// window, scale, out | None, lse | None, workspace | None
PyObject* attn(Args& a) {
  const at::Tensor* q = a.t();
  zl_paged_cache_t c;
  c10::Device dev(c10::kCPU);
  const at::Tensor* lens = a.ok && a.i + 3 < a.n ? tensor(a.v[a.i + 3]) : nullptr;
  if (!lens || !cache_of(a, &c, &dev)) return none();
  const auto* cu = static_cast<const int32_t*>(a.pointer());
  const int32_t n = a.int32();
  const int64_t tq = a.integer();
  const int32_t most = a.int32();
  const bool causal = a.truth();
  const int32_t window = a.int32();
  PyObject* s = a.next();
  const at::Tensor* out = a.maybe();
  const at::Tensor* lse = a.maybe();
  const at::Tensor* ws = a.maybe();
  if (!a.done() || lens->size(0) != n - 1 || q->dim() != 3) return none();
  double scale = 1.0 / std::sqrt(static_cast<double>(c.head_dim));
  if (s != Py_None) {
    if (!PyFloat_Check(s)) return none();
    scale = PyFloat_AS_DOUBLE(s);
  }
  const int64_t nh = q->size(1);
  const int64_t qs = rows(*q, tq, nh, c.head_dim, at::kBFloat16, dev);
  if (qs < 0 || nh > INT32_MAX) return none();
  if (out && (out->scalar_type() != at::kBFloat16 || out->device() != dev || out->sizes() != q->sizes() ||
              !out->is_contiguous()))
    return none();
  if (lse && (lse->scalar_type() != at::kFloat || lse->device() != dev || lse->dim() != 2 || lse->size(0) != nh ||
              lse->size(1) != tq || !lse->is_contiguous()))
    return none();
  at::Tensor o = out ? *out : at::Tensor(), l = lse ? *lse : at::Tensor(), w = ws ? *ws : at::Tensor();
  if (ws && !Scratch(ws, dev).ok) return none();
  zl_status st = ZL_OK;
  {
    Unlocked u;
    const auto heads = static_cast<int32_t>(nh);
    if (!out) o = fresh(*q, {tq, nh, c.head_dim}, at::kBFloat16);
    if (!lse) l = fresh(*q, {nh, tq}, at::kFloat);
    if (!ws) {
      size_t bytes = 0;
      st = zl_paged_attn_workspace_size(cu, n - 1, most, heads, c.num_kv_heads, c.head_dim, &bytes);
      if (st == ZL_OK) w = fresh(*q, {static_cast<int64_t>(bytes)}, at::kByte);
    }
    if (st == ZL_OK) {
      const Scratch scratch(&w, dev);
      st = zl_paged_attn(&c, q->data_ptr(), qs, cu, n - 1, most, heads, static_cast<float>(scale), causal ? 1 : 0,
                         window, o.data_ptr(), l.data_ptr<float>(), scratch.p, scratch.bytes, stream_of(dev));
    }
  }
  if (st != ZL_OK) return status(st);
  PyObject* x = THPVariable_Wrap(std::move(o));
  PyObject* y = THPVariable_Wrap(std::move(l));
  PyObject* r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

bool tables_of(Args& a, zl_page_tables_t* t, c10::Device* dev, const at::Tensor** like) {
  const at::Tensor* table = a.t();
  const at::Tensor* lens = a.t();
  const at::Tensor* refs = a.t();
  if (!a.ok || table->dim() != 2 || lens->dim() != 1 || refs->dim() != 1 || !current(table->device())) return false;
  *dev = table->device();
  *like = lens;
  if (!ints(*table, *dev) || !ints(*lens, *dev) || !ints(*refs, *dev) || lens->size(0) != table->size(0)) return false;
  for (const int64_t x : {table->size(0), table->size(1), refs->size(0)})
    if (x > INT32_MAX) return false;
  *t = zl_page_tables_t{table->data_ptr<int32_t>(), lens->data_ptr<int32_t>(), refs->data_ptr<int32_t>(),
                        static_cast<int32_t>(table->size(0)), static_cast<int32_t>(table->size(1)),
                        static_cast<int32_t>(refs->size(0)), 0};
  return true;
}

bool pool_of(const at::Tensor* cache, const zl_page_tables_t& t, c10::Device dev, zl_page_pool_t* p, int32_t* page) {
  if (!cache || cache->dim() < 4 || cache->device() != dev || !cache->is_contiguous()) return false;
  const int64_t d = cache->dim();
  if (cache->size(d - 4) != t.num_pages || cache->size(d - 2) > INT32_MAX) return false;
  const int64_t elems = cache->size(d - 3) * cache->size(d - 2) * cache->size(d - 1);
  if (elems == 0 || t.num_pages == 0) return false;
  const int64_t bytes = elems * cache->element_size(), groups = cache->numel() / (elems * t.num_pages);
  if (groups > INT32_MAX) return false;
  *p = zl_page_pool_t{cache->data_ptr(), bytes, bytes * t.num_pages, static_cast<int32_t>(groups), t.num_pages};
  *page = static_cast<int32_t>(cache->size(d - 2));
  return true;
}

bool list_of(const at::Tensor* t, c10::Device dev, int64_t n) {
  return t && t->dim() == 1 && ints(*t, dev) && t->size(0) == n;
}

// the tables, counts, page size
PyObject* extend(Args& a) {
  zl_page_tables_t t;
  c10::Device dev(c10::kCPU);
  const at::Tensor* like = nullptr;
  if (!tables_of(a, &t, &dev, &like)) return none();
  const at::Tensor* counts = a.t();
  t.page_size = a.int32();
  if (!a.done() || !list_of(counts, dev, t.slots)) return none();
  at::Tensor out;
  zl_status st;
  {
    Unlocked u;
    out = fresh(*like, {1}, at::kInt);
    st = zl_pages_extend(&t, counts->data_ptr<int32_t>(), out.data_ptr<int32_t>(), stream_of(dev));
  }
  return st != ZL_OK ? status(st) : THPVariable_Wrap(std::move(out));
}

// the cache, the tables, parents, children, workspace | None
PyObject* fork(Args& a) {
  const at::Tensor* cache = a.t();
  zl_page_tables_t t;
  zl_page_pool_t p;
  c10::Device dev(c10::kCPU);
  const at::Tensor* like = nullptr;
  if (!tables_of(a, &t, &dev, &like) || !pool_of(cache, t, dev, &p, &t.page_size)) return none();
  const at::Tensor* parents = a.t();
  const at::Tensor* children = a.t();
  const at::Tensor* ws = a.t();
  if (!a.done() || parents->dim() != 1) return none();
  const int64_t n = parents->size(0);
  const Scratch scratch(ws, dev);
  if (!list_of(parents, dev, n) || !list_of(children, dev, n) || n > INT32_MAX || !scratch.ok) return none();
  at::Tensor out;
  zl_status st;
  {
    Unlocked u;
    out = fresh(*like, {1}, at::kInt);
    st = zl_pages_fork(&p, &t, parents->data_ptr<int32_t>(), children->data_ptr<int32_t>(),
                       static_cast<int32_t>(n), out.data_ptr<int32_t>(), scratch.p, scratch.bytes,
                       stream_of(dev));
  }
  return st != ZL_OK ? status(st) : THPVariable_Wrap(std::move(out));
}

// the cache, the tables, workspace
PyObject* compact(Args& a) {
  const at::Tensor* cache = a.t();
  zl_page_tables_t t;
  zl_page_pool_t p;
  c10::Device dev(c10::kCPU);
  const at::Tensor* like = nullptr;
  if (!tables_of(a, &t, &dev, &like) || !pool_of(cache, t, dev, &p, &t.page_size)) return none();
  const at::Tensor* ws = a.t();
  if (!a.done()) return none();
  const Scratch scratch(ws, dev);
  if (!scratch.ok) return none();
  at::Tensor out;
  zl_status st;
  {
    Unlocked u;
    out = fresh(*like, {1}, at::kInt);
    st = zl_pages_compact(&p, &t, out.data_ptr<int32_t>(), scratch.p, scratch.bytes, stream_of(dev));
  }
  return st != ZL_OK ? status(st) : THPVariable_Wrap(std::move(out));
}

template <PyObject* (*F)(Args&)>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    Args a{args, n};
    return F(a);
  } catch (...) {
    // Only what comes before a launch throws (no memory, a tensor without
    // storage): the long way meets it again and raises it as PyTorch does.
    return PyErr_Occurred() ? nullptr : none();
  }
}

template <PyObject* (*F)(Args&)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<F>));
}

PyMethodDef methods[] = {
    {"rope", fast<rope>(), METH_FASTCALL, nullptr},       {"append", fast<append<false>>(), METH_FASTCALL, nullptr},
    {"append_after", fast<append<true>>(), METH_FASTCALL, nullptr},
    {"attn", fast<attn>(), METH_FASTCALL, nullptr},       {"extend", fast<extend>(), METH_FASTCALL, nullptr},
    {"fork", fast<fork>(), METH_FASTCALL, nullptr},       {"compact", fast<compact>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// It lays tensors out as the PyTorch did that it was compiled against.
PyMODINIT_FUNC PyInit__bind() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", ZL_TORCH_VERSION) != 0) {
    Py_DECREF(m);
    m = nullptr;
  }
  return m;
}
