// lm_torch.cpp -- the 8-bit operators' binding for torch tensors, as a CPython module.
//
// One of these calls is a few microseconds of GPU time, and marshalling it in Python costs several
// times that.  Each function here takes the regular case: tensors of the right types, shapes and
// strides on the current device.  It returns None for anything else, and the caller in binding.py
// then goes its own way, which names what is wrong or deals with what is unusual.  A status other
// than VOC_OK comes back as an int.  The entry points of libvocoder.so are handed over by address.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "vocoder.h"

namespace {

decltype(&vocoder_lm_rows_fp8) g_rows;
decltype(&vocoder_lm_linear_fp8) g_linear;
decltype(&vocoder_lm_kv_append) g_append;
decltype(&vocoder_lm_attention) g_attention;
decltype(&vocoder_lm_attention_ws_bytes) g_attention_ws;
decltype(&vocoder_lm_rotate) g_rotate;
decltype(&vocoder_lm_adapters) g_adapters;
decltype(&vocoder_lm_logprobs) g_logprobs;

constexpr at::ScalarType kF8 = at::kFloat8_e4m3fn;

// The tensor behind an argument; null for None and for anything else.
const at::Tensor *tensor(PyObject *o) {
  return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}
bool none(PyObject *o) { return o == Py_None; }

// VOC_LM_* of a type, -1 for the others.
int code_of(at::ScalarType t) {
  return t == at::kBFloat16 ? VOC_LM_BF16 : t == at::kHalf ? VOC_LM_F16 : t == at::kFloat ? VOC_LM_F32 : -1;
}

bool on(const at::Tensor &t, int dev) { return t.is_cuda() && t.get_device() == dev; }

// Row stride of a [rows, width] operand of the given type, or -1.
long long rows_of(const at::Tensor &t, int64_t rows, int64_t width, at::ScalarType type, int dev) {
  if (t.dim() != 2 || t.scalar_type() != type || t.size(0) != rows || t.size(1) != width ||
      !on(t, dev) || (width > 1 && t.stride(1) != 1))
    return -1;
  return rows > 1 ? t.stride(0) : std::max<int64_t>(width, t.stride(0));
}
bool vector_of(const at::Tensor &t, int64_t n, at::ScalarType type, int dev) {
  return t.dim() == 1 && t.scalar_type() == type && t.size(0) == n && on(t, dev) &&
         (n <= 1 || t.stride(0) == 1);
}

at::Tensor make(at::IntArrayRef size, at::ScalarType type, int dev) {
  return at::Tensor(at::detail::empty_cuda(size, type, c10::Device(c10::kCUDA, dev), std::nullopt));
}
voc_stream_t stream_of(int dev) {
  return reinterpret_cast<voc_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream());
}
int current() { return c10::cuda::current_device(); }

PyObject *wrap(PyObject *given, const at::Tensor &made) {
  if (!none(given)) return Py_NewRef(given);
  return THPVariable_Wrap(made);
}
PyObject *status(voc_status st) { return PyLong_FromLong(st); }

// A call of the library without the interpreter's lock: with VOC_FLAG_SYNC it waits for the stream, and
// a launch may wait for room in the queue, both possibly for what another Python thread has yet to do.
template <typename F, typename... Args>
voc_status unlocked(F call, Args... args) {
  PyThreadState *state = PyEval_SaveThread();
  const voc_status st = call(args...);
  PyEval_RestoreThread(state);
  return st;
}

// rows(x, mode, weight, residual, eps, sum_out, out, scale, flags)
PyObject *rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9) Py_RETURN_NONE;
  const at::Tensor *x = tensor(a[0]), *w = tensor(a[2]), *r = tensor(a[3]), *s = tensor(a[5]),
                   *o = tensor(a[6]), *sc = tensor(a[7]);
  const long mode = PyLong_AsLong(a[1]);
  const double eps = PyFloat_AsDouble(a[4]);
  const long flags = PyLong_AsLong(a[8]);
  if (PyErr_Occurred()) return nullptr;
  if (!x || x->dim() != 2 || !x->is_cuda() || (!w && !none(a[2])) || (!r && !none(a[3])) ||
      (!s && !none(a[5])) || (!o && !none(a[6])) || (!sc && !none(a[7])) || (s && !r))
    Py_RETURN_NONE;
  const int dev = x->get_device();
  const at::ScalarType type = x->scalar_type();
  const int code = code_of(type);
  const int64_t count = x->size(0), width = x->size(1);
  if (dev != current() || code < 0 || (mode == VOC_LM_GATED && width % 2)) Py_RETURN_NONE;
  const int64_t d = mode == VOC_LM_GATED ? width / 2 : width, ldq = (d + 15) / 16 * 16;
  const long long ldx = rows_of(*x, count, width, type, dev);
  const long long ldr = r ? rows_of(*r, count, d, type, dev) : 0;
  long long lds = s ? rows_of(*s, count, d, type, dev) : r ? d : 0;
  const long long ldo = o ? rows_of(*o, count, d, kF8, dev) : ldq;
  if (ldx < 0 || ldr < 0 || lds < 0 || ldo < 0 || d > 0x7fffffff ||
      (w && !vector_of(*w, d, type, dev)) || (sc && !vector_of(*sc, count, at::kFloat, dev)))
    Py_RETURN_NONE;
  at::Tensor sum, out, scale;
  if (r && !s) sum = make({count, d}, type, dev);
  if (!o) {
    out = make({count, ldq}, kF8, dev);
    if (ldq != d) out = out.narrow(1, 0, d);
  }
  if (!sc) scale = make({count}, at::kFloat, dev);
  const voc_status st =
      unlocked(g_rows, x->data_ptr(), ldx, r ? r->data_ptr() : nullptr, ldr,
               w ? w->data_ptr() : nullptr, code, static_cast<int>(mode), count, static_cast<int>(d),
               static_cast<float>(eps), s ? s->data_ptr() : r ? sum.data_ptr() : nullptr, lds,
               o ? o->data_ptr() : out.data_ptr(), ldo,
               static_cast<float *>(sc ? sc->data_ptr() : scale.data_ptr()), stream_of(dev),
               static_cast<unsigned>(flags));
  if (st != VOC_OK) return status(st);
  PyObject *res = PyTuple_New(3);
  if (!res) return nullptr;
  PyTuple_SET_ITEM(res, 0, wrap(a[6], out));
  PyTuple_SET_ITEM(res, 1, wrap(a[7], scale));
  PyTuple_SET_ITEM(res, 2, r && !s ? THPVariable_Wrap(sum) : Py_NewRef(a[5]));
  return res;
  END_HANDLE_TH_ERRORS
}

// linear(x, x_scale, w, w_scale, bias, out_dtype code, out, flags)
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) Py_RETURN_NONE;
  const at::Tensor *x = tensor(a[0]), *xs = tensor(a[1]), *w = tensor(a[2]), *ws = tensor(a[3]),
                   *b = tensor(a[4]), *o = tensor(a[6]);
  long code = PyLong_AsLong(a[5]);
  const long flags = PyLong_AsLong(a[7]);
  if (PyErr_Occurred()) return nullptr;
  if (!x || !xs || !w || !ws || (!b && !none(a[4])) || (!o && !none(a[6])) || x->dim() != 2 ||
      w->dim() != 2 || !x->is_cuda())
    Py_RETURN_NONE;
  const int dev = x->get_device();
  const int64_t M = x->size(0), K = x->size(1), N = w->size(0);
  constexpr int64_t kMost = 1 << 28;
  if (dev != current() || M > kMost || N > kMost || K > kMost) Py_RETURN_NONE;
  long long ldx = rows_of(*x, M, K, kF8, dev), ldw = rows_of(*w, N, K, kF8, dev);
  if (ldx < 0 || ldw < 0 || !vector_of(*xs, M, at::kFloat, dev) ||
      !vector_of(*ws, N, at::kFloat, dev) || (b && !vector_of(*b, N, at::kFloat, dev)))
    Py_RETURN_NONE;
  if (M == 1) ldx = (ldx + 15) / 16 * 16;
  if (N == 1) ldw = (ldw + 15) / 16 * 16;
  at::Tensor out;
  long long ldo = N;
  if (o) {
    if (code >= 0 && code != code_of(o->scalar_type())) Py_RETURN_NONE;
    code = code_of(o->scalar_type());
    ldo = rows_of(*o, M, N, o->scalar_type(), dev);
    if (code < 0 || ldo < 0) Py_RETURN_NONE;
  } else {
    if (code < 0) code = VOC_LM_BF16;
    out = make({M, N},
               code == VOC_LM_BF16 ? at::kBFloat16 : code == VOC_LM_F16 ? at::kHalf : at::kFloat,
               dev);
  }
  const voc_status st = unlocked(
      g_linear, x->data_ptr(), ldx, static_cast<float *>(xs->data_ptr()), w->data_ptr(), ldw,
      static_cast<float *>(ws->data_ptr()), b ? static_cast<float *>(b->data_ptr()) : nullptr,
      static_cast<int>(M), static_cast<int>(N), static_cast<int>(K),
      o ? o->data_ptr() : out.data_ptr(), ldo, static_cast<int>(code), stream_of(dev),
      static_cast<unsigned>(flags));
  if (st != VOC_OK) return status(st);
  return wrap(a[6], out);
  END_HANDLE_TH_ERRORS
}

// What append and attention take of a cache: cache(k, v, k_scale, v_scale) ->
// (k, v, k_scale, v_scale addresses, pages, heads, head_dim, device)
PyObject *cache(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4) Py_RETURN_NONE;
  const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]), *ks = tensor(a[2]), *vs = tensor(a[3]);
  if (!k || !v || !ks || !vs || k->dim() != 4 || v->dim() != 4 || ks->dim() != 2 || vs->dim() != 2)
    Py_RETURN_NONE;
  const int64_t pages = k->size(0), heads = k->size(1), d = k->size(3);
  const int dev = k->get_device();
  if (k->scalar_type() != kF8 || v->scalar_type() != kF8 || ks->scalar_type() != at::kFloat ||
      vs->scalar_type() != at::kFloat || k->size(2) != VOC_LM_BLOCK || v->size(0) != pages ||
      v->size(1) != heads || v->size(2) != d || v->size(3) != VOC_LM_BLOCK ||
      ks->size(0) != pages || ks->size(1) != heads || vs->size(0) != pages ||
      vs->size(1) != heads || !k->is_contiguous() || !v->is_contiguous() ||
      !ks->is_contiguous() || !vs->is_contiguous() || v->get_device() != dev ||
      ks->get_device() != dev || vs->get_device() != dev)
    Py_RETURN_NONE;
  return Py_BuildValue("(KKKKLLLi)", reinterpret_cast<unsigned long long>(k->data_ptr()),
                       reinterpret_cast<unsigned long long>(v->data_ptr()),
                       reinterpret_cast<unsigned long long>(ks->data_ptr()),
                       reinterpret_cast<unsigned long long>(vs->data_ptr()),
                       static_cast<long long>(pages), static_cast<long long>(heads),
                       static_cast<long long>(d), dev);
  END_HANDLE_TH_ERRORS
}

struct CacheArgs {
  unsigned long long p[4];
  long long pages, heads, d;
  long dev;
  bool read(PyObject *t) {
    if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) != 8) return false;
    for (int i = 0; i < 4; ++i) p[i] = PyLong_AsUnsignedLongLong(PyTuple_GET_ITEM(t, i));
    pages = PyLong_AsLongLong(PyTuple_GET_ITEM(t, 4));
    heads = PyLong_AsLongLong(PyTuple_GET_ITEM(t, 5));
    d = PyLong_AsLongLong(PyTuple_GET_ITEM(t, 6));
    dev = PyLong_AsLong(PyTuple_GET_ITEM(t, 7));
    return !PyErr_Occurred() && pages <= 0x7fffffff;
  }
  template <typename T>
  T *at(int i) const { return reinterpret_cast<T *>(p[i]); }
};

struct BatchArgs {
  const int *table, *lens, *cu;
  long long ldt;
  int cols, n_seq;
  bool read(PyObject *table_o, PyObject *lens_o, PyObject *cu_o, int dev) {
    const at::Tensor *t = tensor(table_o), *l = tensor(lens_o), *c = tensor(cu_o);
    if (!t || !l || (!c && !none(cu_o)) || t->dim() != 2 || t->size(0) > 65535 ||
        t->size(1) > 0x3ffffff)
      return false;
    ldt = rows_of(*t, t->size(0), t->size(1), at::kInt, dev);
    n_seq = static_cast<int>(t->size(0)), cols = static_cast<int>(t->size(1));
    if (ldt < 0 || !vector_of(*l, n_seq, at::kInt, dev) ||
        (c && !vector_of(*c, n_seq + 1, at::kInt, dev)))
      return false;
    table = static_cast<const int *>(t->data_ptr()), lens = static_cast<const int *>(l->data_ptr());
    cu = c ? static_cast<const int *>(c->data_ptr()) : nullptr;
    return true;
  }
};

// append(cache, k, v, page_table, kv_lens, cu_q, max_q, flags)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) Py_RETURN_NONE;
  CacheArgs c;
  BatchArgs b;
  const at::Tensor *k = tensor(a[1]), *v = tensor(a[2]);
  const long max_q = PyLong_AsLong(a[6]), flags = PyLong_AsLong(a[7]);
  if (PyErr_Occurred()) return nullptr;
  if (!c.read(a[0]) || !k || !v || k->dim() != 3 || v->dim() != 3 || !k->is_cuda()) Py_RETURN_NONE;
  const int dev = k->get_device(), code = code_of(k->scalar_type());
  if (dev != c.dev || dev != current() || code < 0 || v->scalar_type() != k->scalar_type() ||
      !on(*v, dev) || k->sizes() != v->sizes() || k->size(1) != c.heads || k->size(2) != c.d ||
      k->stride(2) != 1 || v->stride(2) != 1 || k->size(0) > 0x7fffffff || max_q > 0x7fffffff ||
      max_q < 0 || !b.read(a[3], a[4], a[5], dev))
    Py_RETURN_NONE;
  const voc_status st = unlocked(
      g_append, c.at<void>(0), c.at<void>(1), c.at<float>(2), c.at<float>(3), static_cast<int>(c.pages),
      static_cast<int>(c.heads), static_cast<int>(c.d), k->data_ptr(), k->stride(0), k->stride(1),
      v->data_ptr(), v->stride(0), v->stride(1), code, b.table, b.ldt, b.cols, b.lens, b.cu, b.n_seq,
      static_cast<int>(k->size(0)), static_cast<int>(max_q), stream_of(dev),
      static_cast<unsigned>(flags));
  return status(st);
  END_HANDLE_TH_ERRORS
}

// attention(q, cache, page_table, kv_lens, cu_q, max_q, max_kv, softmax_scale, causal, window, out,
//           ws, flags); max_kv < 0 and softmax_scale None stand for the defaults
PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 13) Py_RETURN_NONE;
  CacheArgs c;
  BatchArgs b;
  const at::Tensor *q = tensor(a[0]), *o = tensor(a[10]), *ws = tensor(a[11]);
  const long max_q = PyLong_AsLong(a[5]);
  long max_kv = PyLong_AsLong(a[6]);
  const int causal = PyObject_IsTrue(a[8]);
  const long window = PyLong_AsLong(a[9]), flags = PyLong_AsLong(a[12]);
  double scale = none(a[7]) ? 0. : PyFloat_AsDouble(a[7]);
  if (PyErr_Occurred()) return nullptr;
  if (!c.read(a[1]) || !q || q->dim() != 3 || !q->is_cuda() || (!o && !none(a[10])) ||
      (!ws && !none(a[11])))
    Py_RETURN_NONE;
  const int dev = q->get_device(), code = code_of(q->scalar_type());
  constexpr long kMost = 0x7fffffff;
  if (dev != c.dev || dev != current() || code < 0 || q->size(2) != c.d || q->stride(2) != 1 ||
      q->size(0) > kMost || q->size(1) > kMost || max_q < 0 || max_q > kMost || window < 0 ||
      window > kMost || max_kv > kMost || !b.read(a[2], a[3], a[4], dev))
    Py_RETURN_NONE;
  if (o && (o->sizes() != q->sizes() || o->scalar_type() != q->scalar_type() || !on(*o, dev) ||
            o->stride(2) != 1))
    Py_RETURN_NONE;
  if (ws && (ws->scalar_type() != at::kByte || !ws->is_contiguous() || !on(*ws, dev)))
    Py_RETURN_NONE;
  const int heads = static_cast<int>(q->size(1));
  if (max_kv < 0) max_kv = static_cast<long>(b.cols) * VOC_LM_BLOCK;
  if (none(a[7])) scale = 1. / std::sqrt(static_cast<double>(c.d));
  at::Tensor out, work;
  if (!o) out = make(q->sizes(), q->scalar_type(), dev);
  void *wp = ws ? ws->data_ptr() : nullptr;
  size_t wb = ws ? ws->numel() : 0;
  if (!ws) {
    wb = g_attention_ws(b.n_seq, static_cast<int>(max_q), heads, static_cast<int>(c.heads),
                        static_cast<int>(c.d), static_cast<int>(max_kv), static_cast<int>(window));
    if (wb) {
      work = make({static_cast<int64_t>(wb)}, at::kByte, dev);
      wp = work.data_ptr();
    }
  }
  const at::Tensor &dst = o ? *o : out;
  const voc_status st = unlocked(
      g_attention, q->data_ptr(), q->stride(0), q->stride(1), code, heads, c.at<void>(0), c.at<void>(1),
      c.at<float>(2), c.at<float>(3), static_cast<int>(c.pages), static_cast<int>(c.heads),
      static_cast<int>(c.d), b.table, b.ldt, b.cols, b.lens, b.cu, b.n_seq,
      static_cast<int>(q->size(0)), static_cast<int>(max_q), static_cast<int>(max_kv),
      static_cast<float>(scale), causal, static_cast<int>(window), dst.data_ptr(), dst.stride(0),
      dst.stride(1), wp, wb, stream_of(dev), static_cast<unsigned>(flags));
  if (st != VOC_OK) return status(st);
  return wrap(a[10], out);
  END_HANDLE_TH_ERRORS
}

// One of the tensors of rotate: [tokens][heads][d] with head_dim contiguous.
bool heads_of(const at::Tensor &t, int64_t tokens, int64_t d, at::ScalarType type, int dev) {
  return t.dim() == 3 && t.scalar_type() == type && t.size(0) == tokens && t.size(2) == d && on(t, dev) &&
         t.stride(2) == 1 && t.size(1) <= 65536;
}

// rotate(q, k, positions, turns, axis, q_weight, k_weight, eps, neighbours, q_out, k_out, flags)
PyObject *rotate(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 12) Py_RETURN_NONE;
  const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]), *pos = tensor(a[2]), *turns = tensor(a[3]),
                   *axis = tensor(a[4]), *qw = tensor(a[5]), *kw = tensor(a[6]), *qo = tensor(a[9]),
                   *ko = tensor(a[10]);
  const double eps = PyFloat_AsDouble(a[7]);
  const int near = PyObject_IsTrue(a[8]);
  const long flags = PyLong_AsLong(a[11]);
  if (PyErr_Occurred()) return nullptr;
  if (!q || !pos || !turns || (!k && !none(a[1])) || (!axis && !none(a[4])) || (!qw && !none(a[5])) ||
      (!kw && !none(a[6])) || (!qo && !none(a[9])) || (!ko && !none(a[10])) || q->dim() != 3 ||
      !q->is_cuda() || (!k && (kw || ko)) || pos->dim() < 1 || pos->dim() > 2 || turns->dim() != 1)
    Py_RETURN_NONE;
  const int dev = q->get_device(), code = code_of(q->scalar_type());
  const at::ScalarType type = q->scalar_type();
  const int64_t tokens = q->size(0), d = q->size(2), pairs = turns->size(0);
  const int64_t axes = pos->dim() == 2 ? pos->size(0) : 1;
  if (dev != current() || code < 0 || d > 65536 || pairs > 65536 || axes > 65536 ||
      !heads_of(*q, tokens, d, type, dev) || (k && !heads_of(*k, tokens, d, type, dev)) ||
      (qo && (qo->sizes() != q->sizes() || !heads_of(*qo, tokens, d, type, dev))) ||
      (ko && (ko->sizes() != k->sizes() || !heads_of(*ko, tokens, d, type, dev))) ||
      (qw && !vector_of(*qw, d, type, dev)) || (kw && !vector_of(*kw, d, type, dev)) ||
      !vector_of(*turns, pairs, at::kLong, dev) || (axis && !vector_of(*axis, pairs, at::kInt, dev)))
    Py_RETURN_NONE;
  long long ldp = tokens;
  if (pos->dim() == 1 ? !vector_of(*pos, tokens, at::kInt, dev)
                      : (ldp = rows_of(*pos, axes, tokens, at::kInt, dev)) < 0)
    Py_RETURN_NONE;
  at::Tensor q_made, k_made;
  if (!qo) q_made = make(q->sizes(), type, dev);
  if (k && !ko) k_made = make(k->sizes(), type, dev);
  const at::Tensor &qd = qo ? *qo : q_made, &kd = !k ? *q : ko ? *ko : k_made, &ks = k ? *k : *q;
  const voc_status st = unlocked(
      g_rotate, q->data_ptr(), q->stride(0), q->stride(1), static_cast<int>(q->size(1)),
      k ? k->data_ptr() : nullptr, k ? ks.stride(0) : 0, k ? ks.stride(1) : 0,
      k ? static_cast<int>(k->size(1)) : 0, static_cast<int>(d), code, qw ? qw->data_ptr() : nullptr,
      kw ? kw->data_ptr() : nullptr, static_cast<float>(eps), static_cast<const int *>(pos->data_ptr()),
      ldp, static_cast<int>(axes), static_cast<const long long *>(turns->data_ptr()),
      axis ? static_cast<const int *>(axis->data_ptr()) : nullptr, static_cast<int>(pairs), near, tokens,
      qd.data_ptr(), qd.stride(0), qd.stride(1), k ? kd.data_ptr() : nullptr, k ? kd.stride(0) : 0,
      k ? kd.stride(1) : 0, stream_of(dev), static_cast<unsigned>(flags));
  if (st != VOC_OK) return status(st);
  PyObject *res = PyTuple_New(2);
  if (!res) return nullptr;
  PyTuple_SET_ITEM(res, 0, wrap(a[9], q_made));
  PyTuple_SET_ITEM(res, 1, k ? wrap(a[10], k_made) : Py_NewRef(Py_None));
  return res;
  END_HANDLE_TH_ERRORS
}

// A pool of adapters' matrices [pool][rows][width], rows contiguous: its row stride, or -1.
long long pool_of(const at::Tensor &t, int64_t pool, int64_t rows, int64_t width, at::ScalarType type,
                  int dev) {
  if (t.dim() != 3 || t.scalar_type() != type || t.size(0) != pool || t.size(1) != rows ||
      t.size(2) != width || !on(t, dev) || (width > 1 && t.stride(2) != 1))
    return -1;
  return rows > 1 ? t.stride(1) : (std::max<int64_t>(width, t.stride(1)) + 7) / 8 * 8;
}

// adapters(y, x, x_scale, a, b, scale, ids, ranks, out, flags)
PyObject *adapters(PyObject *, PyObject *const *o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 10) Py_RETURN_NONE;
  const at::Tensor *y = tensor(o[0]), *x = tensor(o[1]), *xs = tensor(o[2]), *a = tensor(o[3]),
                   *b = tensor(o[4]), *scale = tensor(o[5]), *ids = tensor(o[6]), *ranks = tensor(o[7]),
                   *out = tensor(o[8]);
  const long flags = PyLong_AsLong(o[9]);
  if (PyErr_Occurred()) return nullptr;
  if (!y || !x || !xs || !a || !b || !scale || !ids || (!ranks && !none(o[7])) ||
      (!out && !none(o[8])) || x->dim() != 2 || y->dim() != 2 || a->dim() != 3 || !x->is_cuda())
    Py_RETURN_NONE;
  const int dev = x->get_device();
  const int64_t M = x->size(0), K = x->size(1), N = y->size(1), pool = a->size(0), rank = a->size(1);
  const at::ScalarType type = a->scalar_type();
  const int code = code_of(type), y_code = code_of(y->scalar_type());
  constexpr int64_t kMost = 1 << 28;
  if (dev != current() || code < 0 || y_code < 0 || M > kMost || N > kMost || K > kMost ||
      pool > kMost || rank > kMost)
    Py_RETURN_NONE;
  long long ldx = rows_of(*x, M, K, kF8, dev);
  const long long ldy = rows_of(*y, M, N, y->scalar_type(), dev);
  const long long lda = pool_of(*a, pool, rank, K, type, dev), ldb = pool_of(*b, pool, N, rank, type, dev);
  const long long ldo = out ? rows_of(*out, M, N, y->scalar_type(), dev) : N;
  if (ldx < 0 || ldy < 0 || lda < 0 || ldb < 0 || ldo < 0 || !vector_of(*xs, M, at::kFloat, dev) ||
      !vector_of(*scale, pool, at::kFloat, dev) || !vector_of(*ids, M, at::kInt, dev) ||
      (ranks && !vector_of(*ranks, pool, at::kInt, dev)))
    Py_RETURN_NONE;
  if (M == 1) ldx = (ldx + 15) / 16 * 16;
  at::Tensor made;
  if (!out) made = make({M, N}, y->scalar_type(), dev);
  const voc_status st = unlocked(
      g_adapters, x->data_ptr(), ldx, static_cast<const float *>(xs->data_ptr()), y->data_ptr(), ldy,
      y_code, a->data_ptr(), lda, pool > 1 ? a->stride(0) : 0, b->data_ptr(), ldb,
      pool > 1 ? b->stride(0) : 0, code, static_cast<const float *>(scale->data_ptr()),
      ranks ? static_cast<const int *>(ranks->data_ptr()) : nullptr, static_cast<int>(rank),
      static_cast<int>(pool), static_cast<const int *>(ids->data_ptr()), static_cast<int>(M),
      static_cast<int>(N), static_cast<int>(K), out ? out->data_ptr() : made.data_ptr(), ldo,
      stream_of(dev), static_cast<unsigned>(flags));
  if (st != VOC_OK) return status(st);
  return wrap(o[8], made);
  END_HANDLE_TH_ERRORS
}

// logprobs(logits, tokens, top, temperature, entropy, flags)
PyObject *logprobs(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 6) Py_RETURN_NONE;
  const at::Tensor *x = tensor(a[0]), *tokens = tensor(a[1]);
  const long top = PyLong_AsLong(a[2]);
  const double temperature = PyFloat_AsDouble(a[3]);
  const int entropy = PyObject_IsTrue(a[4]);
  const long flags = PyLong_AsLong(a[5]);
  if (PyErr_Occurred()) return nullptr;
  if (!x || (!tokens && !none(a[1])) || x->dim() != 2 || !x->is_cuda() || top < 0 ||
      top > x->size(1))
    Py_RETURN_NONE;
  const int dev = x->get_device(), code = code_of(x->scalar_type());
  const int64_t rows = x->size(0), vocab = x->size(1);
  if (dev != current() || code < 0 || vocab > 0x7fffffff) Py_RETURN_NONE;
  const long long ldl = rows_of(*x, rows, vocab, x->scalar_type(), dev);
  if (ldl < 0 || (tokens && !vector_of(*tokens, rows, at::kLong, dev))) Py_RETURN_NONE;
  at::Tensor made[4];
  if (tokens) made[0] = make({rows}, at::kFloat, dev);
  if (entropy) made[1] = make({rows}, at::kFloat, dev);
  if (top) made[2] = make({rows, top}, at::kFloat, dev), made[3] = make({rows, top}, at::kLong, dev);
  auto at = [&](int i) { return made[i].defined() ? made[i].data_ptr() : nullptr; };
  const voc_status st = unlocked(
      g_logprobs, x->data_ptr(), ldl, code, rows, static_cast<int>(vocab), static_cast<float>(temperature),
      tokens ? static_cast<const long long *>(tokens->data_ptr()) : nullptr, static_cast<float *>(at(0)),
      static_cast<float *>(at(1)), static_cast<int>(top), static_cast<float *>(at(2)),
      static_cast<long long *>(at(3)), stream_of(dev), static_cast<unsigned>(flags));
  if (st != VOC_OK) return status(st);
  PyObject *res = PyTuple_New(4);
  if (!res) return nullptr;
  for (int i = 0; i < 4; ++i)
    PyTuple_SET_ITEM(res, i, made[i].defined() ? THPVariable_Wrap(made[i]) : Py_NewRef(Py_None));
  return res;
  END_HANDLE_TH_ERRORS
}

// init(addresses of rows, linear, append, attention, attention_ws, rotate, adapters, logprobs)
PyObject *init(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "init takes eight addresses");
    return nullptr;
  }
  void *p[8];
  for (int i = 0; i < 8; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
      return nullptr;
    }
  }
  g_rows = reinterpret_cast<decltype(g_rows)>(p[0]);
  g_linear = reinterpret_cast<decltype(g_linear)>(p[1]);
  g_append = reinterpret_cast<decltype(g_append)>(p[2]);
  g_attention = reinterpret_cast<decltype(g_attention)>(p[3]);
  g_attention_ws = reinterpret_cast<decltype(g_attention_ws)>(p[4]);
  g_rotate = reinterpret_cast<decltype(g_rotate)>(p[5]);
  g_adapters = reinterpret_cast<decltype(g_adapters)>(p[6]);
  g_logprobs = reinterpret_cast<decltype(g_logprobs)>(p[7]);
  Py_RETURN_NONE;
}

template <typename F>
PyMethodDef method(const char *name, F f) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {method("init", init),         method("rows", rows),
                           method("linear", linear),     method("cache", cache),
                           method("append", append),     method("attention", attention),
                           method("rotate", rotate),     method("adapters", adapters),
                           method("logprobs", logprobs), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "lm_torch", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_lm_torch(void) { return PyModule_Create(&g_module); }
