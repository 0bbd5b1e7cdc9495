// torch_calls.cpp -- the Python calls of the latent, sampling, tree and row operators, compiled (module _calls).
//
// A decode step's kernels take 3 to 20 us, and the same calls through ctypes took 15 to 19 us of
// host time: the output's allocation and the checks of a dozen tensors run cold after every
// launch, an attribute at a time.  Here a call reads its tensors directly, allocates its
// output and enters the C ABI (whose addresses bind() is given).  A call that is not
// of the plain form (tensors of the documented types and shapes on the current device, host
// lengths as a list, ...) returns None, and the Python function takes it from there, with its
// messages: nothing is decided here that it would not decide the same way.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <vector>

#include "pskv.h"

namespace {

decltype(&::kv_prep_append_latent) g_append = nullptr;
decltype(&::decode_attn_latent) g_decode = nullptr;
decltype(&::prefill_attn_expanded) g_prefill = nullptr;
decltype(&::verify_drafts) g_verify = nullptr;
decltype(&::decode_attn_latent_tree) g_tree = nullptr;
decltype(&::sample_tokens) g_sample = nullptr;
decltype(&::verify_tree) g_walk = nullptr;
decltype(&::kv_keep_tokens) g_keep = nullptr;
decltype(&::kv_fork_rows) g_fork = nullptr;

constexpr auto kBf16 = at::kBFloat16;
constexpr auto kI32 = at::kInt;

using Shape = std::initializer_list<int64_t>;

const at::Tensor *tensor(PyObject *o) {
  return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}

bool on(const at::Tensor &t, at::ScalarType kind, int dev, Shape shape) {
  return t.is_cuda() && t.layout() == at::kStrided && t.get_device() == dev && t.scalar_type() == kind &&
         t.sizes() == at::IntArrayRef(shape);
}

// The address of a contiguous tensor of this kind and shape; false: not that.
bool whole(PyObject *o, at::ScalarType kind, int dev, Shape shape, void **p) {
  const at::Tensor *t = tensor(o);
  if (!t || !on(*t, kind, dev, shape) || !t->is_contiguous()) return false;
  *p = t->data_ptr();
  return true;
}

// The same where None stands for a null pointer.
bool maybe(PyObject *o, at::ScalarType kind, int dev, Shape shape, void **p) {
  *p = nullptr;
  return o == Py_None || whole(o, kind, dev, shape, p);
}

// bf16 rows: only the last dimension has to be contiguous.
const at::Tensor *rows(PyObject *o, int dev, Shape shape) {
  const at::Tensor *t = tensor(o);
  return t && on(*t, kBf16, dev, shape) && t->stride(-1) == 1 ? t : nullptr;
}

bool whole_numbers(PyObject *o, std::vector<int32_t> &v) {
  if (!PyList_CheckExact(o)) return false;
  const Py_ssize_t n = PyList_GET_SIZE(o);
  v.resize((size_t)n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject *x = PyList_GET_ITEM(o, i);
    if (!PyLong_CheckExact(x)) return false;
    int over = 0;
    const long long y = PyLong_AsLongLongAndOverflow(x, &over);
    if (over || y < INT32_MIN || y > INT32_MAX) return false;
    v[(size_t)i] = (int32_t)y;
  }
  return true;
}

bool number(PyObject *o, double *x) {
  if (PyFloat_CheckExact(o)) {
    *x = PyFloat_AS_DOUBLE(o);
    return true;
  }
  if (!PyLong_CheckExact(o)) return false;
  *x = PyLong_AsDouble(o);
  if (!PyErr_Occurred()) return true;
  PyErr_Clear();
  return false;
}

bool integer(PyObject *o, long long lo, long long hi, long long *x) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  *x = PyLong_AsLongLongAndOverflow(o, &over);
  return !over && *x >= lo && *x <= hi;
}

// A stream's address, or None for the current one.
bool stream_of(PyObject *o, int dev, pskv_stream_t *s) {
  if (o == Py_None) {
    *s = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    return true;
  }
  if (!PyLong_CheckExact(o)) return false;
  *s = static_cast<pskv_stream_t>(PyLong_AsVoidPtr(o));
  if (!PyErr_Occurred()) return true;
  PyErr_Clear();
  return false;
}

// New memory on the tensor's device; it belongs to the stream of the call (`given`: its argument).
at::Tensor fresh(const at::Tensor &like, at::ScalarType kind, Shape shape, PyObject *given, pskv_stream_t s, int dev) {
  c10::cuda::OptionalCUDAStreamGuard guard;
  if (given != Py_None) {
    // (0 and 1 name the default stream)
    cudaStream_t raw = reinterpret_cast<cudaStream_t>(s);
    guard.reset_stream(reinterpret_cast<uintptr_t>(raw) <= 1
                           ? c10::cuda::getDefaultCUDAStream((c10::DeviceIndex)dev)
                           : c10::cuda::getStreamFromExternal(raw, (c10::DeviceIndex)dev));
  }
  // (through the dispatcher, as torch.empty: its modes see the tensor, and deterministic mode fills it.  Straight from the
  // allocator three of them took 0.6 to 1.1 us less)
  return at::empty(shape, like.options().dtype(kind));
}

// The output: the given tensor, or a new one of `code`'s type (-1: the caller's to refuse).
bool output(PyObject *given, long long code, const at::Tensor &like, int dev, Shape shape, PyObject *stream,
            pskv_stream_t s, at::Tensor *out, int32_t *dtype) {
  if (given != Py_None) {
    const at::Tensor *t = tensor(given);
    if (!t || !(on(*t, kBf16, dev, shape) || on(*t, at::kFloat, dev, shape)) || !t->is_contiguous())
      return false;
    *dtype = t->scalar_type() == kBf16 ? PSKV_DTYPE_BF16 : PSKV_DTYPE_F32;
    *out = *t;
    return true;
  }
  if (code != PSKV_DTYPE_BF16 && code != PSKV_DTYPE_F32) return false;
  *dtype = (int32_t)code;
  *out = fresh(like, code == PSKV_DTYPE_BF16 ? kBf16 : at::kFloat, shape, stream, s, dev);
  return true;
}

// None where the arguments are not plain, or where the tensor library throws (out of memory, no
// device: the Python form then raises what belongs there).
template <typename F>
PyObject *guarded(F f) {
  try {
    PyObject *r = f();
    if (r || PyErr_Occurred()) return r;
  } catch (...) {
    PyErr_Clear();
  }
  Py_RETURN_NONE;
}

PyObject *result(int rc, PyObject *kept, const at::Tensor &out) {
  if (rc != PSKV_OK) return PyLong_FromLong(rc);
  if (kept != Py_None) {
    Py_INCREF(kept);
    return kept;
  }
  return THPVariable_Wrap(out);
}

#define NEED(c) \
  if (!(c)) return nullptr

// (layout address, its device, head_dim_k, head_dim_v), as the four first arguments.
struct Pool {
  void *layout;
  long long dev, dk, dv;
  bool read(PyObject *const *a) {
    if (!PyLong_CheckExact(a[0])) return false;
    layout = PyLong_AsVoidPtr(a[0]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return false;
    }
    return integer(a[1], 0, 1 << 20, &dev) && integer(a[2], 1, 1 << 20, &dk) &&
           integer(a[3], 1, 1 << 20, &dv) && dev == c10::cuda::current_device();
  }
};

// A window's ancestor masks: 64-bit integers, signed or not.
bool masks(PyObject *o, int dev, Shape shape, void **p) {
  return whole(o, at::kLong, dev, shape, p) || whole(o, at::kUInt64, dev, shape, p);
}

// q, page_tables, seq_lens, seq_lens_host, scale, num_splits, workspace, out, code, stream[, tree_mask]
PyObject *decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Pool pool;
    NEED((n == 14 || n == 15) && pool.read(a));
    const int dev = (int)pool.dev;
    const at::Tensor *q = tensor(a[4]), *table = tensor(a[5]);
    NEED(q && table && q->dim() == 4 && table->dim() == 2);
    const int64_t batch = q->size(0), tokens = q->size(1), heads = q->size(2), stride = table->size(1);
    std::vector<int32_t> lens;
    void *qp, *tp, *lp;
    pskv_stream_t s;
    double scale;
    long long splits, code;
    NEED(whole(a[4], kBf16, dev, {batch, tokens, heads, pool.dk}, &qp));
    NEED(whole(a[5], kI32, dev, {batch, stride}, &tp) && whole(a[6], kI32, dev, {batch}, &lp));
    NEED(whole_numbers(a[7], lens) && (int64_t)lens.size() == batch && number(a[8], &scale));
    NEED(integer(a[9], INT32_MIN, INT32_MAX, &splits) && integer(a[12], -1, 1 << 20, &code));
    void *mp = nullptr;
    NEED(n == 14 || masks(a[14], dev, {batch, tokens}, &mp));
    void *wp = nullptr;  // without a workspace: for plans that need none
    size_t bytes = 0;
    if (a[10] != Py_None) {
      const at::Tensor *ws = tensor(a[10]);
      NEED(ws && ws->is_cuda() && ws->get_device() == dev && ws->is_contiguous());
      wp = ws->data_ptr();
      bytes = ws->nbytes();
    }
    NEED(batch <= INT32_MAX && tokens <= INT32_MAX && heads <= INT32_MAX && stride <= INT32_MAX);
    NEED(stream_of(a[13], dev, &s));
    at::Tensor out;
    int32_t dtype;
    NEED(output(a[11], code, *q, dev, {batch, tokens, heads, pool.dv}, a[13], s, &out, &dtype));
    void *op = out.data_ptr();
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = n == 14 ? g_decode(static_cast<const pskv_layout *>(pool.layout), qp, (const int32_t *)tp, (int32_t)stride,
                            lens.data(), (const int32_t *)lp, (int32_t)batch, (int32_t)tokens, (int32_t)heads,
                            (float)scale, (int32_t)splits, wp, bytes, op, dtype, nullptr, s)
                 : g_tree(static_cast<const pskv_layout *>(pool.layout), qp, (const int32_t *)tp, (int32_t)stride,
                          lens.data(), (const int32_t *)lp, (const uint64_t *)mp, (int32_t)batch, (int32_t)tokens,
                          (int32_t)heads, (float)scale, (int32_t)splits, wp, bytes, op, dtype, nullptr, s);
    Py_END_ALLOW_THREADS
    NEED(wp || rc != PSKV_ERR_WORKSPACE_TOO_SMALL);
    return result(rc, a[11], out);
  });
}

// x, row_of, pos_of, page_tables, pages_of_row, eps, w, cos, sin, adjacent, first_pos, q, q_out, dense, stream
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    Pool pool;
    NEED(n == 19 && pool.read(a));
    const int dev = (int)pool.dev;
    const at::Tensor *row_of = tensor(a[5]), *table = tensor(a[7]), *cos = tensor(a[11]);
    NEED(row_of && table && cos && table->dim() == 2 && cos->dim() == 2);
    const int64_t t = row_of->numel(), batch = table->size(0), stride = table->size(1), d = pool.dk;
    const at::Tensor *x = rows(a[4], dev, {t, d});
    pskv_latent_prep_desc p = {};
    double eps;
    long long adjacent;
    void *rp, *pp, *tp, *gp, *w, *c, *s, *fp, *dp;
    pskv_stream_t st;
    NEED(x && number(a[9], &eps) && integer(a[13], 0, 1, &adjacent));
    NEED(whole(a[5], kI32, dev, {t}, &rp) && whole(a[6], kI32, dev, {t}, &pp));
    NEED(whole(a[7], kI32, dev, {batch, stride}, &tp) && whole(a[8], kI32, dev, {batch}, &gp));
    NEED(maybe(a[10], at::kFloat, dev, {d - PSKV_LATENT_ROT}, &w));
    const int64_t angles = cos->size(0);
    NEED(whole(a[11], at::kFloat, dev, {angles, PSKV_LATENT_ROT / 2}, &c));
    NEED(whole(a[12], at::kFloat, dev, {angles, PSKV_LATENT_ROT / 2}, &s));
    NEED(maybe(a[14], kI32, dev, {batch}, &fp) && maybe(a[17], kBf16, dev, {t, d}, &dp));
    NEED(t <= INT32_MAX && batch <= INT32_MAX && stride <= INT32_MAX && angles <= INT32_MAX);
    p.eps = (float)eps;
    p.pairs = adjacent ? PSKV_PAIRS_ADJACENT : PSKV_PAIRS_HALVES;
    p.w = (const float *)w;
    p.rope_cos = (const float *)c;
    p.rope_sin = (const float *)s;
    p.max_pos = (int32_t)angles;
    NEED((a[15] == Py_None) == (a[16] == Py_None));
    if (a[15] != Py_None) {
      const at::Tensor *q0 = tensor(a[15]);
      NEED(q0 && q0->dim() == 3);
      const int64_t heads = q0->size(1);
      const at::Tensor *q = rows(a[15], dev, {t, heads, PSKV_LATENT_ROT});
      const at::Tensor *o = rows(a[16], dev, {t, heads, PSKV_LATENT_ROT});
      NEED(q && o && heads >= 1 && heads <= INT32_MAX);
      p.num_q_heads = (int32_t)heads;
      p.q = q->data_ptr();
      // (a stride over a single row says nothing)
      auto step = [](const at::Tensor *r, int64_t dim) { return r->size(dim) > 1 ? r->stride(dim) : PSKV_LATENT_ROT; };
      p.q_token = step(q, 0);
      p.q_head = step(q, 1);
      p.q_out = o->data_ptr();
      p.q_out_token = step(o, 0);
      p.q_out_head = step(o, 1);
      NEED(p.q_out_token >= PSKV_LATENT_ROT && p.q_out_head >= PSKV_LATENT_ROT);
    }
    NEED(stream_of(a[18], dev, &st));
    void *xp = x->data_ptr();
    const int64_t x_token = t > 1 ? x->stride(0) : d;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_append(static_cast<const pskv_layout *>(pool.layout), &p, xp, x_token, (int32_t)t,
                  (const int32_t *)rp, (const int32_t *)pp, (const int32_t *)fp, (const int32_t *)tp,
                  (int32_t)stride, (const int32_t *)gp, (int32_t)batch, nullptr, nullptr, nullptr, dp, st);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
  });
}

// q, kv, k_rot, cu_q, cu_q_host, cu_k, cu_k_host, scale, out, code, status, stream
PyObject *prefill(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    NEED(n == 12);
    const int dev = c10::cuda::current_device();
    const at::Tensor *q = tensor(a[0]);
    std::vector<int32_t> cq, ck;
    NEED(q && q->dim() == 3 && whole_numbers(a[4], cq) && whole_numbers(a[6], ck));
    NEED(cq.size() >= 2 && cq.size() == ck.size() && cq.size() <= INT32_MAX);
    const int64_t batch = (int64_t)cq.size() - 1, tq = cq.back(), tk = ck.back(), heads = q->size(1);
    void *qp, *kp, *cqp, *ckp, *sp = nullptr;
    pskv_stream_t s;
    double scale;
    long long code;
    NEED(whole(a[0], kBf16, dev, {tq, heads, PSKV_EXPANDED_NOPE + PSKV_LATENT_ROT}, &qp));
    NEED(whole(a[1], kBf16, dev, {tk, heads, PSKV_EXPANDED_NOPE + PSKV_EXPANDED_V}, &kp));
    const at::Tensor *rot = rows(a[2], dev, {tk, PSKV_LATENT_ROT});
    NEED(rot && whole(a[3], kI32, dev, {batch + 1}, &cqp) && whole(a[5], kI32, dev, {batch + 1}, &ckp));
    NEED(number(a[7], &scale) && integer(a[9], -1, 1 << 20, &code) && heads <= INT32_MAX);
    if (a[10] != Py_None) {
      const at::Tensor *st = tensor(a[10]);
      NEED(st && st->is_cuda() && st->get_device() == dev && st->scalar_type() == kI32 && st->is_contiguous());
      sp = st->data_ptr();
    }
    NEED(stream_of(a[11], dev, &s));
    at::Tensor out;
    int32_t dtype;
    NEED(output(a[8], code, *q, dev, {tq, heads, PSKV_EXPANDED_V}, a[11], s, &out, &dtype));
    void *op = out.data_ptr(), *rp = rot->data_ptr();
    const int64_t r_token = tk > 1 ? rot->stride(0) : PSKV_LATENT_ROT;
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_prefill(qp, kp, rp, r_token, cq.data(), (const int32_t *)cqp, ck.data(), (const int32_t *)ckp,
                   (int32_t)batch, (int32_t)heads, (float)scale, op, dtype, (int32_t *)sp, s);
    Py_END_ALLOW_THREADS
    return result(rc, a[8], out);
  });
}

// target, draft, drafts, u, num_drafts, tokens, accepted, status, stream
PyObject *verify(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    NEED(n == 9);
    const int dev = c10::cuda::current_device();
    const at::Tensor *target = tensor(a[0]);
    NEED(target && target->dim() == 3 && target->size(1) >= 1);
    const at::ScalarType kind = target->scalar_type();
    const int64_t batch = target->size(0), t1 = target->size(1), t = t1 - 1, vocab = target->size(2);
    NEED((kind == kBf16 || kind == at::kFloat) && batch <= INT32_MAX && t1 <= INT32_MAX && vocab <= INT32_MAX);
    void *tp, *qp, *dp, *up, *np, *sp = nullptr, *kp, *ap;
    pskv_stream_t s;
    NEED(whole(a[0], kind, dev, {batch, t1, vocab}, &tp) && maybe(a[1], kind, dev, {batch, t, vocab}, &qp));
    NEED(whole(a[2], kI32, dev, {batch, t}, &dp) && whole(a[3], at::kFloat, dev, {batch, t1}, &up));
    NEED(maybe(a[4], kI32, dev, {batch}, &np));
    if (a[7] != Py_None) {
      const at::Tensor *st = tensor(a[7]);
      NEED(st && st->is_cuda() && st->get_device() == dev && st->scalar_type() == kI32 && st->is_contiguous());
      sp = st->data_ptr();
    }
    NEED(stream_of(a[8], dev, &s));
    at::Tensor tokens, accepted;
    if (a[5] == Py_None) {
      tokens = fresh(*target, kI32, {batch, t1}, a[8], s, dev);
      kp = tokens.data_ptr();
    } else {
      NEED(whole(a[5], kI32, dev, {batch, t1}, &kp));
    }
    if (a[6] == Py_None) {
      accepted = fresh(*target, kI32, {batch}, a[8], s, dev);
      ap = accepted.data_ptr();
    } else {
      NEED(whole(a[6], kI32, dev, {batch}, &ap));
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_verify(tp, qp, kind == kBf16 ? PSKV_DTYPE_BF16 : PSKV_DTYPE_F32, (const int32_t *)dp,
                  (const int32_t *)np, (const float *)up, (int32_t)batch, (int32_t)t, (int32_t)vocab,
                  (int32_t *)kp, (int32_t *)ap, (int32_t *)sp, s);
    Py_END_ALLOW_THREADS
    if (rc != PSKV_OK) return PyLong_FromLong(rc);
    PyObject *x = result(rc, a[5], tokens), *y = result(rc, a[6], accepted), *r = nullptr;
    if (x && y) r = PyTuple_Pack(2, x, y);
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
  });
}

// A fault word, or None.
bool fault_word(PyObject *o, int dev, void **p) {
  *p = nullptr;
  if (o == Py_None) return true;
  const at::Tensor *t = tensor(o);
  if (!t || !t->is_cuda() || t->get_device() != dev || t->scalar_type() != kI32 || !t->is_contiguous()) return false;
  *p = t->data_ptr();
  return true;
}

// A given int32 tensor of this shape, or a new one: its address, and the Python object that the call returns.
bool result_i32(PyObject *given, const at::Tensor &like, int dev, Shape shape, PyObject *stream, pskv_stream_t s,
                at::Tensor *made, void **p) {
  if (given != Py_None) return whole(given, kI32, dev, shape, p);
  *made = fresh(like, kI32, shape, stream, s, dev);
  *p = made->data_ptr();
  return true;
}

// logits, u, temperature, top_k, top_p, min_p, tokens, probs, status, stream
PyObject *sample(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    NEED(n == 10);
    const int dev = c10::cuda::current_device();
    const at::Tensor *l = tensor(a[0]);
    NEED(l && (l->dim() == 2 || l->dim() == 3) && l->is_cuda() && l->layout() == at::kStrided && l->get_device() == dev);
    const at::ScalarType kind = l->scalar_type();
    const bool three = l->dim() == 3;
    const int64_t batch = l->size(0), each = three ? l->size(1) : 1, vocab = l->size(three ? 2 : 1);
    NEED((kind == kBf16 || kind == at::kFloat) && batch >= 1 && each >= 1 && vocab >= 1);
    NEED(batch <= INT32_MAX && each <= INT32_MAX && vocab <= INT32_MAX && (vocab == 1 || l->stride(-1) == 1));
    // one step from row to row (a stride over a single one says nothing)
    int64_t step = vocab;
    if (each > 1) step = l->stride(1);
    if (batch > 1) {
      NEED(l->stride(0) % each == 0 && (each == 1 || l->stride(0) / each == step));
      step = l->stride(0) / each;
    }
    NEED(step >= vocab);
    const bool draw = a[1] != Py_None;  // (else only the distribution is asked for)
    void *up = nullptr, *kp = nullptr, *hp, *tp, *pp, *mp, *sp, *qp = nullptr;
    pskv_stream_t s;
    auto head = [&](PyObject *o, at::ScalarType t, void **p) {
      return three ? whole(o, t, dev, {batch, each}, p) : whole(o, t, dev, {batch}, p);
    };
    NEED((!draw || head(a[1], at::kFloat, &up)) && maybe(a[2], at::kFloat, dev, {batch}, &hp) && maybe(a[3], kI32, dev, {batch}, &tp));
    NEED(maybe(a[4], at::kFloat, dev, {batch}, &pp) && maybe(a[5], at::kFloat, dev, {batch}, &mp));
    NEED(fault_word(a[8], dev, &sp) && stream_of(a[9], dev, &s));
    int32_t code = PSKV_DTYPE_F32;
    if (a[7] != Py_None) {
      const at::Tensor *q = tensor(a[7]);
      NEED(q && (q->scalar_type() == kBf16 || q->scalar_type() == at::kFloat));
      NEED(three ? whole(a[7], q->scalar_type(), dev, {batch, each, vocab}, &qp)
                 : whole(a[7], q->scalar_type(), dev, {batch, vocab}, &qp));
      code = q->scalar_type() == kBf16 ? PSKV_DTYPE_BF16 : PSKV_DTYPE_F32;
    }
    at::Tensor tokens;
    if (a[6] != Py_None) {
      NEED(head(a[6], kI32, &kp));
    } else if (draw) {
      tokens = three ? fresh(*l, kI32, {batch, each}, a[9], s, dev) : fresh(*l, kI32, {batch}, a[9], s, dev);
      kp = tokens.data_ptr();
    }
    const pskv_sample_desc f = {(const float *)hp, (const int32_t *)tp, (const float *)pp, (const float *)mp};
    void *lp = l->data_ptr();
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_sample(lp, kind == kBf16 ? PSKV_DTYPE_BF16 : PSKV_DTYPE_F32, step, (int32_t)batch, (int32_t)each,
                  (int32_t)vocab, &f, (const float *)up, (int32_t *)kp, qp, code, (int32_t *)sp, s);
    Py_END_ALLOW_THREADS
    return draw ? result(rc, a[6], tokens) : PyLong_FromLong(rc);
  });
}

// drafts, tree_mask, sampled, tokens, path, kept, status, stream
PyObject *walk(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    NEED(n == 8);
    const int dev = c10::cuda::current_device();
    const at::Tensor *drafts = tensor(a[0]);
    NEED(drafts && drafts->dim() == 2);
    const int64_t batch = drafts->size(0), t = drafts->size(1);
    void *dp, *mp, *sp, *kp, *pp, *np, *fp;
    pskv_stream_t s;
    NEED(batch <= INT32_MAX && t <= INT32_MAX);
    NEED(whole(a[0], kI32, dev, {batch, t}, &dp) && masks(a[1], dev, {batch, t}, &mp) && whole(a[2], kI32, dev, {batch, t}, &sp));
    NEED(fault_word(a[6], dev, &fp) && stream_of(a[7], dev, &s));
    at::Tensor tokens, path, kept;
    NEED(result_i32(a[3], *drafts, dev, {batch, t}, a[7], s, &tokens, &kp));
    NEED(result_i32(a[4], *drafts, dev, {batch, t}, a[7], s, &path, &pp));
    NEED(result_i32(a[5], *drafts, dev, {batch}, a[7], s, &kept, &np));
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_walk((const int32_t *)dp, (const uint64_t *)mp, (const int32_t *)sp, (int32_t)batch, (int32_t)t,
                (int32_t *)kp, (int32_t *)pp, (int32_t *)np, (int32_t *)fp, s);
    Py_END_ALLOW_THREADS
    if (rc != PSKV_OK) return PyLong_FromLong(rc);
    PyObject *x = result(rc, a[3], tokens), *y = result(rc, a[4], path), *z = result(rc, a[5], kept), *r = nullptr;
    if (x && y && z) r = PyTuple_Pack(3, x, y, z);
    Py_XDECREF(x);
    Py_XDECREF(y);
    Py_XDECREF(z);
    return r;
  });
}

// Layout addresses of a tuple that Python made of the layouts.
bool layouts_of(PyObject *o, std::vector<const pskv_layout *> &v) {
  if (!PyTuple_CheckExact(o)) return false;
  const Py_ssize_t n = PyTuple_GET_SIZE(o);
  v.resize((size_t)n);
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject *x = PyTuple_GET_ITEM(o, i);
    if (!PyLong_CheckExact(x)) return false;
    v[(size_t)i] = static_cast<const pskv_layout *>(PyLong_AsVoidPtr(x));
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return false;
    }
  }
  return n >= 1 && n <= INT32_MAX;
}

// layouts (all on device), device, page_tables, seq_lens, path, kept, new_lens, stream
PyObject *keep(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    std::vector<const pskv_layout *> layouts;
    long long dev64;
    NEED(n == 8 && layouts_of(a[0], layouts) && integer(a[1], 0, 1 << 20, &dev64) && dev64 == c10::cuda::current_device());
    const int dev = (int)dev64;
    const at::Tensor *table = tensor(a[2]), *path = tensor(a[4]);
    NEED(table && path && table->dim() == 2 && path->dim() == 2);
    const int64_t batch = path->size(0), t = path->size(1), stride = table->size(1);
    void *tp, *lp, *pp, *kp, *np;
    pskv_stream_t s;
    NEED(batch <= INT32_MAX && t <= INT32_MAX && stride <= INT32_MAX);
    NEED(whole(a[2], kI32, dev, {batch, stride}, &tp) && whole(a[3], kI32, dev, {batch}, &lp));
    NEED(whole(a[4], kI32, dev, {batch, t}, &pp) && whole(a[5], kI32, dev, {batch}, &kp) && stream_of(a[7], dev, &s));
    at::Tensor lens;
    NEED(result_i32(a[6], *path, dev, {batch}, a[7], s, &lens, &np));
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_keep(layouts.data(), (int32_t)layouts.size(), (const int32_t *)tp, (int32_t)stride, (const int32_t *)lp,
                (const int32_t *)pp, (const int32_t *)kp, (int32_t)batch, (int32_t)t, (int32_t *)np, s);
    Py_END_ALLOW_THREADS
    return result(rc, a[6], lens);
  });
}

// layouts, device, src, dst, new_pages, page_tables, seq_lens, pages_of_row, stream
PyObject *fork_rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    std::vector<const pskv_layout *> layouts;
    long long dev64;
    NEED(n == 9 && layouts_of(a[0], layouts) && integer(a[1], 0, 1 << 20, &dev64) && dev64 == c10::cuda::current_device());
    const int dev = (int)dev64;
    const at::Tensor *src = tensor(a[2]), *table = tensor(a[5]);
    NEED(src && table && src->dim() == 1 && table->dim() == 2);
    const int64_t k = src->size(0), batch = table->size(0), stride = table->size(1);
    void *sp, *dp, *np, *tp, *lp, *gp;
    pskv_stream_t s;
    NEED(k <= INT32_MAX && batch <= INT32_MAX && stride <= INT32_MAX);
    NEED(whole(a[2], kI32, dev, {k}, &sp) && whole(a[3], kI32, dev, {k}, &dp) && whole(a[4], kI32, dev, {k}, &np));
    NEED(whole(a[5], kI32, dev, {batch, stride}, &tp) && whole(a[6], kI32, dev, {batch}, &lp));
    NEED(whole(a[7], kI32, dev, {batch}, &gp) && stream_of(a[8], dev, &s));
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_fork(layouts.data(), (int32_t)layouts.size(), (const int32_t *)sp, (const int32_t *)dp, (const int32_t *)np,
                (int32_t)k, (int32_t *)tp, (int32_t)stride, (int32_t *)lp, (int32_t *)gp, (int32_t)batch, s);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
  });
}

// Addresses of the C entry points: kv_prep_append_latent, decode_attn_latent, prefill_attn_expanded,
// verify_drafts, decode_attn_latent_tree, sample_tokens, verify_tree, kv_keep_tokens, kv_fork_rows.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  void *p[9];
  if (n != 9) {
    PyErr_SetString(PyExc_TypeError, "nine addresses");
    return nullptr;
  }
  for (int i = 0; i < 9; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_append = reinterpret_cast<decltype(g_append)>(p[0]);
  g_decode = reinterpret_cast<decltype(g_decode)>(p[1]);
  g_prefill = reinterpret_cast<decltype(g_prefill)>(p[2]);
  g_verify = reinterpret_cast<decltype(g_verify)>(p[3]);
  g_tree = reinterpret_cast<decltype(g_tree)>(p[4]);
  g_sample = reinterpret_cast<decltype(g_sample)>(p[5]);
  g_walk = reinterpret_cast<decltype(g_walk)>(p[6]);
  g_keep = reinterpret_cast<decltype(g_keep)>(p[7]);
  g_fork = reinterpret_cast<decltype(g_fork)>(p[8]);
  Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef methods[] = {{"bind", fast<bind>(), METH_FASTCALL, nullptr},
                         {"append", fast<append>(), METH_FASTCALL, nullptr},
                         {"decode", fast<decode>(), METH_FASTCALL, nullptr},
                         {"prefill", fast<prefill>(), METH_FASTCALL, nullptr},
                         {"verify", fast<verify>(), METH_FASTCALL, nullptr},
                         {"sample", fast<sample>(), METH_FASTCALL, nullptr},
                         {"walk", fast<walk>(), METH_FASTCALL, nullptr},
                         {"keep", fast<keep>(), METH_FASTCALL, nullptr},
                         {"fork", fast<fork_rows>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
