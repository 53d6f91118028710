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

// attend(cache, k, q, start, len, M, window, sinks, scale, out, lse, workspace, stream) -> out or status
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 13);
  const Cache cache = cache_of(a[0], a[1]);
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
    const int64_t need = lib.attend_workspace(cache.c, M, (int)heads, (int)T);
    if (need < 0) return status_of(need);
    work = at::empty({need}, q.options().dtype(at::kByte));
  } else {
    work = tensor("workspace", a[11]);
  }
  uint8_t *const w = flat<uint8_t>("workspace", work, -1, cache.on);
  if (T > 0) {
    void *const stream = stream_of(cache.on, a[12]);
    const int s = unlocked([&] {
      return lib.attend(cache.c, x.p, x.row, x.head, o.p, o.row, o.head, type, lse, start, len, (int)T, M, (int)heads,
                        window, sinks, scale, w, work.numel(), stream);
    });
    if (s < 0) return status_of(s);
  }
  if (a[9] != Py_None) {
    Py_INCREF(a[9]);
    return a[9];
  }
  return THPVariable_Wrap(out);
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

// bind(append, attend_workspace, attend, verify_workspace, verify, current_stream)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 6);
  void *f[5];
  for (int i = 0; i < 5; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (!f[i]) REFUSE("no function");
  }
  lib.append = reinterpret_cast<decltype(lib.append)>(f[0]);
  lib.attend_workspace = reinterpret_cast<decltype(lib.attend_workspace)>(f[1]);
  lib.attend = reinterpret_cast<decltype(lib.attend)>(f[2]);
  lib.verify_workspace = reinterpret_cast<decltype(lib.verify_workspace)>(f[3]);
  lib.verify = reinterpret_cast<decltype(lib.verify)>(f[4]);
  Py_INCREF(a[5]);
  Py_XDECREF(current_stream);
  current_stream = a[5];
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind), FAST(append), FAST(attend), FAST(verify), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qgemv_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qgemv_torch(void) { return PyModule_Create(&module); }
