// The verify step's calls on torch tensors: checks their arguments, reads the
// addresses and strides out of them and calls the C ABI (include/qgemv.h).
//
// A call of these operators takes the GPU 3 to 10 us for one request.  The same
// checks in Python, with ctypes, take 5 to 10 us a call; here they take less
// than one, so that the GPU is what is waited for.
//
// The library is loaded by the Python module, which hands over the addresses of
// its functions (bind); nothing here depends on where it lies.

#include <Python.h>

#include <climits>
#include <cmath>

#include <ATen/ATen.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include "qgemv.h"

namespace {

struct Library {
  decltype(&qgemv_kv_append) append;
  decltype(&qgemv_kv_attend_workspace) attend_workspace;
  decltype(&qgemv_kv_attend) attend;
  decltype(&qgemv_verify_drafts_workspace) verify_workspace;
  decltype(&qgemv_verify_drafts) verify;
  decltype(&qgemv_kv_attend_shared_workspace) attend_shared_workspace;
  decltype(&qgemv_kv_attend_shared) attend_shared;
  decltype(&qgemv_kv_append_rotated) append_rotated;
  decltype(&qgemv_route) route;
  decltype(&qgemv_adapt_workspace) adapt_workspace;
  decltype(&qgemv_adapt) adapt;
} lib;

PyObject *current_stream;  // of a device: index -> address

#define REFUSE(...) throw c10::ValueError({__func__, __FILE__, __LINE__}, c10::str(__VA_ARGS__))

const at::Tensor &tensor(const char *name, PyObject *o) {
  if (!THPVariable_Check(o)) {
    throw c10::TypeError({__func__, __FILE__, __LINE__},
                         c10::str(name, " must be a tensor, not ", Py_TYPE(o)->tp_name));
  }
  return THPVariable_Unpack(o);
}

int64_t integer(const char *name, PyObject *o, int64_t lo, int64_t hi) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  if (v < lo || v > hi) REFUSE(name, " is out of range: ", v);
  return v;
}
int int32(const char *name, PyObject *o) { return (int)integer(name, o, INT_MIN, INT_MAX); }

double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

int type_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return QGEMV_F32;
    case at::kBFloat16: return QGEMV_BF16;
    case at::kHalf: return QGEMV_F16;
    case at::kFloat8_e4m3fn: return QGEMV_E4M3;
    default: return -1;
  }
}

// A [T][heads][dim] operand.  A dimension of one element has no stride of its
// own: it gets a packed one.
struct Operand {
  void *p;
  int64_t row, head;
};
Operand operand(const char *name, const at::Tensor &t, int64_t T, int64_t heads, int64_t dim, int64_t type,
                const at::Device &on) {
  if (t.dim() != 3 || t.size(0) != T || t.size(1) != heads || t.size(2) != dim || type_of(t.scalar_type()) != type ||
      t.device() != on)
    REFUSE(name, " must be a [", T, ", ", heads, ", ", dim, "] tensor of the right type on ", on);
  if (t.stride(2) != 1) REFUSE(name, " must have a contiguous last dimension");
  Operand o;
  o.p = t.data_ptr();
  o.head = heads > 1 ? t.stride(1) : dim;
  o.row = T > 1 ? t.stride(0) : heads * o.head;
  return o;
}

template <class X>
X *flat(const char *name, const at::Tensor &t, int64_t n, const at::Device &on) {
  constexpr at::ScalarType type = std::is_same_v<X, float> ? at::kFloat : std::is_same_v<X, uint8_t> ? at::kByte : at::kInt;
  if (t.scalar_type() != type || t.device() != on || !t.is_contiguous() || (n >= 0 && (t.dim() != 1 || t.size(0) != n)))
    REFUSE(name, " must be a contiguous ", type, " [", n >= 0 ? std::to_string(n) : "bytes", "] tensor on ", on);
  return static_cast<X *>(t.data_ptr());
}

// The raw stream of a call on `on`, which has to be the current device.
void *stream_of(const at::Device &on, PyObject *stream) {
  if (!on.is_cuda()) REFUSE("tensors must be on the GPU, not on ", on);
  const c10::impl::VirtualGuardImpl guard(on.type());
  const at::Device current = guard.getDevice();
  if (current != on) REFUSE("tensors are on ", on, ", the current device is ", current);
  THPObjectPtr got;
  if (stream == Py_None) {
    THPObjectPtr index(PyLong_FromLong(on.index()));
    if (!index) throw python_error();
    got = PyObject_CallOneArg(current_stream, index.get());
  } else if (PyLong_Check(stream)) {
    Py_INCREF(stream);
    got = stream;
  } else {
    got = PyObject_GetAttrString(stream, "cuda_stream");
  }
  if (!got) throw python_error();
  const unsigned long long v = PyLong_AsUnsignedLongLong(got.get());
  if (v == (unsigned long long)-1 && PyErr_Occurred()) throw python_error();
  return reinterpret_cast<void *>(v);
}

// The cache's description and its device, as KvCache keeps them.
struct Cache {
  const qgemv_kv_cache *c;
  at::Device on;
};
Cache cache_of(PyObject *address, PyObject *k) {
  return {static_cast<const qgemv_kv_cache *>(PyLong_AsVoidPtr(address)), tensor("k", k).device()};
}

// A status below 0 goes back to Python, which raises it by name.
PyObject *status_of(int64_t s) { return PyLong_FromLongLong(s); }

void expect(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) throw c10::TypeError({__func__, __FILE__, __LINE__}, c10::str("expected ", want, " arguments, got ", n));
}

template <class F>
int unlocked(F call) {
  Py_BEGIN_ALLOW_THREADS
  const int s = call();
  Py_BLOCK_THREADS
  return s;
  Py_END_ALLOW_THREADS
}

// What a call returns: the given output, or its own.
PyObject *given_or(PyObject *given, const at::Tensor &own) {
  if (given == Py_None) return THPVariable_Wrap(own);
  Py_INCREF(given);
  return given;
}

// append(cache, k, new_k, new_v, start, len, stream) -> status
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 7);
  const Cache cache = cache_of(a[0], a[1]);
  const at::Tensor &nk = tensor("new_k", a[2]), &nv = tensor("new_v", a[3]);
  const int src = type_of(nk.scalar_type());
  if (src < 0 || src == QGEMV_E4M3 || nv.scalar_type() != nk.scalar_type())
    REFUSE("new_k and new_v must be float32, bfloat16 or float16, got ", nk.scalar_type(), ", ", nv.scalar_type());
  if (nk.dim() != 3) REFUSE("new_k must be [T, heads, dim]");
  const int64_t T = nk.size(0);
  const Operand k = operand("new_k", nk, T, cache.c->heads, cache.c->dim, src, cache.on);
  const Operand v = operand("new_v", nv, T, cache.c->heads, cache.c->dim, src, cache.on);
  const int32_t *start = flat<int32_t>("start", tensor("start", a[4]), cache.c->batch + 1, cache.on);
  const int32_t *len = flat<int32_t>("len", tensor("len", a[5]), cache.c->batch, cache.on);
  if (T == 0) return status_of(QGEMV_OK);
  if (T > INT_MAX) REFUSE("too many rows: ", T);
  void *const stream = stream_of(cache.on, a[6]);
  return status_of(unlocked([&] {
    return lib.append(cache.c, k.p, k.row, k.head, v.p, v.row, v.head, src, start, len, (int)T, stream);
  }));
  END_HANDLE_TH_ERRORS
}

// attend(cache, k, q, start, len, M, window, sinks, scale, out, lse, workspace, stream) -> out or status;
// with a common prefix of `common` tokens, attend_shared
PyObject *attend_over(const Cache &cache, PyObject *const *a, PyObject *common) {
  const int32_t *const shared = common ? flat<int32_t>("shared", tensor("shared", common), 1, cache.on) : nullptr;
  const at::Tensor &q = tensor("q", a[2]);
  const int type = type_of(q.scalar_type()), dim = cache.c->dim;
  if ((type != QGEMV_BF16 && type != QGEMV_F16) || (cache.c->dtype != type && cache.c->dtype != QGEMV_E4M3))
    REFUSE("q of ", q.scalar_type(), " over this cache is not supported");
  if (q.dim() != 3) REFUSE("q must be [T, heads, ", dim, "]");
  const int64_t T = q.size(0), heads = q.size(1);
  if (T > INT_MAX || heads > INT_MAX) REFUSE("q is too large");
  const Operand x = operand("q", q, T, heads, dim, type, cache.on);
  const int32_t *start = flat<int32_t>("start", tensor("start", a[3]), cache.c->batch + 1, cache.on);
  const int32_t *len = flat<int32_t>("len", tensor("len", a[4]), cache.c->batch, cache.on);
  const int M = int32("M", a[5]), window = int32("window", a[6]), sinks = int32("sinks", a[7]);
  const float scale = a[8] == Py_None ? (float)(1.0 / std::sqrt((double)dim)) : (float)number(a[8]);
  const at::Tensor out = a[9] == Py_None ? at::empty({T, heads, dim}, q.options()) : tensor("out", a[9]);
  const Operand o = operand("out", out, T, heads, dim, type, cache.on);
  float *lse = nullptr;
  if (a[10] != Py_None) {
    const at::Tensor &t = tensor("lse", a[10]);
    if (t.dim() != 2 || t.size(0) != T || t.size(1) != heads) REFUSE("lse must be [", T, ", ", heads, "]");
    lse = flat<float>("lse", t, -1, cache.on);
  }
  at::Tensor work;
  if (a[11] == Py_None) {
    const int64_t need = (shared ? lib.attend_shared_workspace : lib.attend_workspace)(cache.c, M, (int)heads, (int)T);
    if (need < 0) return status_of(need);
    work = at::empty({need}, q.options().dtype(at::kByte));
  } else {
    work = tensor("workspace", a[11]);
  }
  uint8_t *const w = flat<uint8_t>("workspace", work, -1, cache.on);
  if (T > 0) {
    void *const stream = stream_of(cache.on, a[12]);
    const int s = unlocked([&] {
      return shared ? lib.attend_shared(cache.c, x.p, x.row, x.head, o.p, o.row, o.head, type, lse, start, len, shared,
                                        (int)T, M, (int)heads, window, sinks, scale, w, work.numel(), stream)
                    : lib.attend(cache.c, x.p, x.row, x.head, o.p, o.row, o.head, type, lse, start, len, (int)T, M,
                                 (int)heads, window, sinks, scale, w, work.numel(), stream);
    });
    if (s < 0) return status_of(s);
  }
  return given_or(a[9], out);
}

PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 13);
  return attend_over(cache_of(a[0], a[1]), a, nullptr);
  END_HANDLE_TH_ERRORS
}

// attend_shared(cache, k, q, start, len, shared, M, window, sinks, scale, out, lse, workspace, stream) -> out or status
PyObject *attend_shared(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 14);
  PyObject *const rest[] = {a[0], a[1], a[2], a[3], a[4], a[6], a[7], a[8], a[9], a[10], a[11], a[12], a[13]};
  return attend_over(cache_of(a[0], a[1]), rest, a[5]);
  END_HANDLE_TH_ERRORS
}

// append_rotated(cache, k, q, new_k, new_v, start, len, freq, position, axes, interleaved, out, stream) -> out or status
PyObject *append_rotated(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 13);
  const Cache cache = cache_of(a[0], a[1]);
  const at::Tensor &q = tensor("q", a[2]), &nk = tensor("new_k", a[3]), &nv = tensor("new_v", a[4]);
  const int src = type_of(q.scalar_type()), dim = cache.c->dim;
  if (src < 0 || src == QGEMV_E4M3 || nk.scalar_type() != q.scalar_type() || nv.scalar_type() != q.scalar_type())
    REFUSE("q, new_k and new_v must be of one type, float32, bfloat16 or float16, got ", q.scalar_type(), ", ",
           nk.scalar_type(), ", ", nv.scalar_type());
  if (q.dim() != 3) REFUSE("q must be [T, heads, ", dim, "]");
  const int64_t T = q.size(0), heads = q.size(1);
  if (T > INT_MAX || heads > INT_MAX) REFUSE("q is too large");
  const Operand x = operand("q", q, T, heads, dim, src, cache.on);
  const Operand k = operand("new_k", nk, T, cache.c->heads, dim, src, cache.on);
  const Operand v = operand("new_v", nv, T, cache.c->heads, dim, src, cache.on);
  const int32_t *start = flat<int32_t>("start", tensor("start", a[5]), cache.c->batch + 1, cache.on);
  const int32_t *len = flat<int32_t>("len", tensor("len", a[6]), cache.c->batch, cache.on);
  const at::Tensor &freq = tensor("freq", a[7]);
  if (freq.dim() != 1) REFUSE("freq must be [pairs]");
  const int64_t pairs = freq.size(0);
  if (pairs > dim) REFUSE("freq has ", pairs, " pairs for heads of ", dim);
  const float *f = flat<float>("freq", freq, pairs, cache.on);
  const int32_t *position = nullptr, *axis = nullptr;
  int64_t axes = 0;
  if (a[8] != Py_None) {
    const at::Tensor &p = tensor("position", a[8]);
    if (p.dim() != 2 || p.size(0) < 1 || p.size(0) > INT_MAX || p.size(1) != T) REFUSE("position must be [axes, ", T, "]");
    position = flat<int32_t>("position", p, -1, cache.on);
    axes = p.size(0);
  }
  if (a[9] != Py_None) {
    if (!position) REFUSE("axes belong to given positions");
    axis = flat<int32_t>("axes", tensor("axes", a[9]), pairs, cache.on);
  }
  const int interleaved = PyObject_IsTrue(a[10]);
  if (interleaved < 0) throw python_error();
  const at::ScalarType kind = cache.c->dtype == QGEMV_F16 ? at::kHalf : at::kBFloat16;
  const at::Tensor out = a[11] == Py_None ? at::empty({T, heads, dim}, q.options().dtype(kind)) : tensor("out", a[11]);
  const int out_type = type_of(out.scalar_type());
  if (out_type != QGEMV_BF16 && out_type != QGEMV_F16) REFUSE("out must be bfloat16 or float16, got ", out.scalar_type());
  const Operand o = operand("out", out, T, heads, dim, out_type, cache.on);
  if (T > 0) {
    void *const stream = stream_of(cache.on, a[12]);
    const int s = unlocked([&] {
      return lib.append_rotated(cache.c, x.p, x.row, x.head, (int)heads, o.p, o.row, o.head, out_type, k.p, k.row,
                                k.head, v.p, v.row, v.head, src, start, len, (int)T, f, (int)pairs, position, T,
                                (int)axes, axis, interleaved, stream);
    });
    if (s < 0) return status_of(s);
  }
  return given_or(a[11], out);
  END_HANDLE_TH_ERRORS
}

// route(logits, k, score, bias, groups, keep, best, renormalise, scale, stream) -> (experts, weights) or status
PyObject *route(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 10);
  const at::Tensor &x = tensor("logits", a[0]);
  const at::Device on = x.device();
  const int type = type_of(x.scalar_type());
  if (type < 0 || type == QGEMV_E4M3 || x.dim() != 2 || x.size(1) < 1)
    REFUSE("logits must be a float32, bfloat16 or float16 [T, E] tensor");
  const int64_t T = x.size(0), E = x.size(1);
  if (T > INT_MAX || E > INT_MAX) REFUSE("logits are too large");
  if (E > 1 && x.stride(1) != 1) REFUSE("logits must have contiguous rows");
  const int64_t row = T > 1 ? x.stride(0) : E;
  const int k = (int)integer("k", a[1], 1, E);
  const int score = int32("score", a[2]), groups = int32("groups", a[4]), keep = int32("keep", a[5]);
  const int best = int32("best", a[6]), renormalise = PyObject_IsTrue(a[7]);
  if (renormalise < 0) throw python_error();
  const float scale = (float)number(a[8]);
  const float *bias = a[3] == Py_None ? nullptr : flat<float>("bias", tensor("bias", a[3]), E, on);
  const at::Tensor experts = at::empty({T, k}, x.options().dtype(at::kInt));
  const at::Tensor weights = at::empty({T, k}, x.options().dtype(at::kFloat));
  if (T > 0) {
    void *const stream = stream_of(on, a[9]);
    const int s = unlocked([&] {
      return lib.route(x.data_ptr(), row, type, bias, static_cast<int32_t *>(experts.data_ptr()),
                       static_cast<float *>(weights.data_ptr()), (int)T, (int)E, k, score, groups, keep, best,
                       renormalise, scale, stream);
    });
    if (s < 0) return status_of(s);
  }
  THPObjectPtr e(THPVariable_Wrap(experts)), w(THPVariable_Wrap(weights));
  if (!e || !w) throw python_error();
  return PyTuple_Pack(2, e.get(), w.get());
  END_HANDLE_TH_ERRORS
}

// adapt(y, x, a, b, adapter, scales, out, workspace, stream) -> out or status
PyObject *adapt(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 9);
  const at::Tensor &y = tensor("y", a[0]), &x = tensor("x", a[1]), &down = tensor("a", a[2]), &up = tensor("b", a[3]);
  const at::Device on = y.device();
  if (y.dim() != 2 || y.scalar_type() != at::kFloat || y.size(1) < 1) REFUSE("y must be a float32 [T, N] tensor");
  const int64_t T = y.size(0), N = y.size(1);
  const int type = type_of(x.scalar_type());
  if ((type != QGEMV_BF16 && type != QGEMV_F16) || x.dim() != 2 || x.size(0) != T || x.size(1) < 1 || x.device() != on)
    REFUSE("x must be a bfloat16 or float16 [", T, ", K] tensor on ", on);
  const int64_t K = x.size(1);
  if (down.dim() != 3 || down.size(0) < 1 || down.size(2) != K || down.scalar_type() != x.scalar_type() ||
      down.device() != on || !down.is_contiguous())
    REFUSE("a must be a contiguous ", x.scalar_type(), " [n, r, ", K, "] tensor on ", on);
  const int64_t count = down.size(0), r = down.size(1);
  if (up.dim() != 3 || up.size(0) != count || up.size(1) != N || up.size(2) != r || up.scalar_type() != x.scalar_type() ||
      up.device() != on || !up.is_contiguous())
    REFUSE("b must be a contiguous ", x.scalar_type(), " [", count, ", ", N, ", ", r, "] tensor on ", on);
  if (T > INT_MAX || N > INT_MAX || K > INT_MAX || count > INT_MAX || r > INT_MAX) REFUSE("an operand is too large");
  auto row_of = [](const char *name, const at::Tensor &t) {
    if (t.size(1) > 1 && t.stride(1) != 1) REFUSE(name, " must have contiguous rows");
    return t.size(0) > 1 ? t.stride(0) : t.size(1);
  };
  const int64_t y_row = row_of("y", y);
  int64_t x_row = row_of("x", x);
  const int32_t *adapter = flat<int32_t>("adapter", tensor("adapter", a[4]), T, on);
  const float *scales = a[5] == Py_None ? nullptr : flat<float>("scales", tensor("scales", a[5]), count, on);
  const at::Tensor out = a[6] == Py_None ? at::empty({T, N}, y.options()) : tensor("out", a[6]);
  if (out.dim() != 2 || out.size(0) != T || out.size(1) != N || out.scalar_type() != at::kFloat || out.device() != on)
    REFUSE("out must be a float32 [", T, ", ", N, "] tensor on ", on);
  const int64_t out_row = row_of("out", out);
  const int64_t need = lib.adapt_workspace((int)T, (int)r);
  if (need < 0) return status_of(need);
  at::Tensor work = a[7] == Py_None ? at::empty({need}, y.options().dtype(at::kByte)) : tensor("workspace", a[7]);
  uint8_t *const w = flat<uint8_t>("workspace", work, -1, on);
  if (T > 0) {
    void *const stream = stream_of(on, a[8]);
    const int s = unlocked([&] {
      return lib.adapt(static_cast<const float *>(y.data_ptr()), y_row, static_cast<float *>(out.data_ptr()), out_row,
                       x.data_ptr(), x_row, down.data_ptr(), up.data_ptr(), type, adapter, scales, (int)T, (int)count,
                       (int)r, (int)K, (int)N, w, work.numel(), stream);
    });
    if (s < 0) return status_of(s);
  }
  return given_or(a[6], out);
  END_HANDLE_TH_ERRORS
}

// verify(p, q, tokens, u, start, M, workspace, stream) -> (out, count) or status
PyObject *verify(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 8);
  const at::Tensor &p = tensor("p", a[0]);
  const at::Device on = p.device();
  const int type = type_of(p.scalar_type());
  if (type < 0 || type == QGEMV_E4M3 || p.dim() != 2 || p.size(1) < 1)
    REFUSE("p must be a float32, bfloat16 or float16 [T, V] tensor");
  const int64_t T = p.size(0), V = p.size(1);
  if (T > INT_MAX || V > INT_MAX) REFUSE("p is too large");
  const void *qp = nullptr;
  int64_t p_row = T > 1 ? p.stride(0) : V, q_row = 0;
  if (V > 1 && p.stride(1) != 1) REFUSE("p must have contiguous rows");
  if (a[1] != Py_None) {
    const at::Tensor &q = tensor("q", a[1]);
    if (q.sizes() != p.sizes() || q.scalar_type() != p.scalar_type() || q.device() != on || (V > 1 && q.stride(1) != 1))
      REFUSE("q must be a ", p.scalar_type(), " [", T, ", ", V, "] tensor on ", on, " with contiguous rows");
    qp = q.data_ptr();
    q_row = T > 1 ? q.stride(0) : V;
  }
  const at::Tensor &starts = tensor("start", a[4]);
  if (starts.dim() != 1 || starts.size(0) < 2) REFUSE("start must have at least two entries");
  const int64_t B = starts.size(0) - 1;
  if (B > INT_MAX) REFUSE("too many sequences: ", B);
  const int32_t *start = flat<int32_t>("start", starts, B + 1, on);
  const at::Tensor &tokens = tensor("tokens", a[2]);
  const int32_t *tok = flat<int32_t>("tokens", tokens, T, on);
  const float *u = flat<float>("u", tensor("u", a[3]), T, on);
  const int M = int32("M", a[5]);
  const at::Tensor out = at::empty({T}, tokens.options()), count = at::empty({B}, tokens.options());
  int32_t *const o = static_cast<int32_t *>(out.data_ptr()), *const c = static_cast<int32_t *>(count.data_ptr());
  if (T == 0) {
    count.zero_();
  } else {
    at::Tensor work;
    if (a[6] == Py_None) {
      const int64_t need = lib.verify_workspace((int)B, (int)V);
      if (need < 0) return status_of(need);
      work = at::zeros({need}, p.options().dtype(at::kByte));
    } else {
      work = tensor("workspace", a[6]);
    }
    uint8_t *const w = flat<uint8_t>("workspace", work, -1, on);
    void *const stream = stream_of(on, a[7]);
    const int s = unlocked([&] {
      return lib.verify(p.data_ptr(), p_row, qp, q_row, type, tok, u, start, o, c, (int)B, (int)T, M, (int)V, w,
                        work.numel(), stream);
    });
    if (s < 0) return status_of(s);
  }
  THPObjectPtr x(THPVariable_Wrap(out)), y(THPVariable_Wrap(count));
  if (!x || !y) throw python_error();
  return PyTuple_Pack(2, x.get(), y.get());
  END_HANDLE_TH_ERRORS
}

// bind(the functions of Library in its order, current_stream)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  constexpr int N = 11;
  expect(n, N + 1);
  void *f[N];
  for (int i = 0; i < N; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (!f[i]) REFUSE("no function");
  }
  lib.append = reinterpret_cast<decltype(lib.append)>(f[0]);
  lib.attend_workspace = reinterpret_cast<decltype(lib.attend_workspace)>(f[1]);
  lib.attend = reinterpret_cast<decltype(lib.attend)>(f[2]);
  lib.verify_workspace = reinterpret_cast<decltype(lib.verify_workspace)>(f[3]);
  lib.verify = reinterpret_cast<decltype(lib.verify)>(f[4]);
  lib.attend_shared_workspace = reinterpret_cast<decltype(lib.attend_shared_workspace)>(f[5]);
  lib.attend_shared = reinterpret_cast<decltype(lib.attend_shared)>(f[6]);
  lib.append_rotated = reinterpret_cast<decltype(lib.append_rotated)>(f[7]);
  lib.route = reinterpret_cast<decltype(lib.route)>(f[8]);
  lib.adapt_workspace = reinterpret_cast<decltype(lib.adapt_workspace)>(f[9]);
  lib.adapt = reinterpret_cast<decltype(lib.adapt)>(f[10]);
  Py_INCREF(a[N]);
  Py_XDECREF(current_stream);
  current_stream = a[N];
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind), FAST(append), FAST(attend), FAST(attend_shared), FAST(append_rotated),
                         FAST(verify), FAST(route), FAST(adapt), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qgemv_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qgemv_torch(void) { return PyModule_Create(&module); }
