// The Python side of the calls that a decode loop makes for every token: kvs_rope,
// kvs_append_paged and kvs_attn_decode, and around drafted tokens kvs_attn_tree,
// kvs_accept_paged, kvs_fork_paged and kvs_reclaim_paged.  The kernels of the first three take 2 to
// 10 us for a token of a batch, and up to 25 arguments checked and converted in Python took longer:
// calls back to back are one per 6.8 us (rotation of 64 tokens), 13.2 (their append) and 8.7
// (attention of a short sequence) that way, and 2.9, 5.0 and 5.9 through this file, launches
// included.  The drafting calls take 3 to 15 us on small batches (accepted paths 3, forks 7,
// reclaimed pages 10, a short tree 12) and come the same way.  Arguments are those of the C
// functions; a tensor is checked for its type, size, device and layout, an int is taken as an
// address and None as NULL.
#define PY_SSIZE_T_CLEAN
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "../../include/kvs.h"

namespace {

struct PythonError {};  // set, and to be raised

int64_t times(int64_t a, int64_t b) {
  int64_t y;
  return __builtin_mul_overflow(a, b, &y) ? ((a < 0) == (b < 0) ? INT64_MAX : INT64_MIN) : y;
}
template <class... T>
int64_t times(int64_t a, int64_t b, T... rest) { return times(times(a, b), rest...); }

int64_t integer(PyObject* o, const char* name, int64_t lo, int64_t hi) {
  int overflow = 0;
  const long long x = PyLong_AsLongLongAndOverflow(o, &overflow);
  if (x == -1 && PyErr_Occurred()) throw PythonError();
  if (overflow || x < lo || x > hi) {
    PyErr_Format(PyExc_OverflowError, "kvs: %s = %S is out of range", name, o);
    throw PythonError();
  }
  return x;
}
int32_t int32(PyObject* o, const char* name) {
  return (int32_t)integer(o, name, INT32_MIN, INT32_MAX);
}

const kvs_dims& dims(PyObject* o, kvs_dims* to) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE)) throw PythonError();
  const bool whole = b.len == (Py_ssize_t)sizeof(kvs_dims);
  if (whole) memcpy(to, b.buf, sizeof(kvs_dims));
  PyBuffer_Release(&b);
  if (!whole) {
    PyErr_SetString(PyExc_TypeError, "kvs: the first argument must be a Dims");
    throw PythonError();
  }
  return *to;
}

// The current device, where the library launches, and the stream of a call.
struct Place {
  int device = -2;  // no tensor's
  void* stream = nullptr;

  explicit Place(PyObject* s) {
    static bool ready = false;  // once torch's CUDA state is set up it stays
    if (!ready) {
      PyObject* cuda = PyImport_ImportModule("torch.cuda");
      PyObject* yes = cuda ? PyObject_CallMethod(cuda, "is_initialized", nullptr) : nullptr;
      ready = yes == Py_True;
      Py_XDECREF(yes);
      if (yes && !ready && s == Py_None) {  // sets it up, or raises
        PyObject* current = PyObject_CallMethod(cuda, "current_stream", nullptr);
        ready = current != nullptr;
        Py_XDECREF(current);
      }
      Py_XDECREF(cuda);
      if (PyErr_Occurred()) throw PythonError();
    }
    if (ready) device = c10::cuda::current_device();
    if (s == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    } else if (PyLong_Check(s)) {
      stream = address(s);
    } else {
      PyObject* raw = PyObject_GetAttrString(s, "cuda_stream");
      if (!raw) throw PythonError();
      stream = PyLong_AsVoidPtr(raw);
      Py_DECREF(raw);
      if (PyErr_Occurred()) throw PythonError();
    }
  }

  static void* address(PyObject* o) {
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw PythonError();
    return p;
  }

  // Device pointer of an argument that must hold at least n elements of a type.
  template <class T>
  T* arg(PyObject* o, at::ScalarType type, int64_t n, const char* name) const {
    if (o == Py_None) return nullptr;
    if (PyLong_CheckExact(o)) return static_cast<T*>(address(o));
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "kvs: %s must be a tensor, an address or None, got %R", name,
                   (PyObject*)Py_TYPE(o));
      throw PythonError();
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != type || t.numel() < n) {
      PyObject* dtype = PyObject_GetAttrString(o, "dtype");
      PyErr_Format(PyExc_ValueError, "kvs: %s must hold at least %lld elements of %s, got %lld of %S",
                   name, (long long)n,
                   type == at::kBFloat16 ? "torch.bfloat16" : type == at::kInt ? "torch.int32"
                   : type == at::kFloat  ? "torch.float32"  : "torch.uint8",
                   (long long)t.numel(), dtype);
      Py_XDECREF(dtype);
      throw PythonError();
    }
    if (!t.is_cuda() || t.get_device() != device) {
      PyObject* where = PyObject_GetAttrString(o, "device");
      PyErr_Format(PyExc_ValueError, "kvs: tensor arguments must be CUDA tensors on the current "
                   "device (%s is on %S)", name, where);
      Py_XDECREF(where);
      throw PythonError();
    }
    if (!t.is_contiguous()) {
      PyErr_Format(PyExc_ValueError, "kvs: tensor arguments must be contiguous (%s is not)", name);
      throw PythonError();
    }
    return static_cast<T*>(t.data_ptr());
  }
  kvs_bf16* bf16(PyObject* o, int64_t n, const char* name) const {
    return arg<kvs_bf16>(o, at::kBFloat16, n, name);
  }
  int32_t* i32(PyObject* o, int64_t n, const char* name) const {
    return arg<int32_t>(o, at::kInt, n, name);
  }
};

// The rotation frequencies in host memory: a contiguous float64 CPU tensor's own, another CPU
// tensor of real numbers converted whole (64 of float32: 0.1 us a call, number by number 59),
// or a copy of any sequence of numbers.  A tensor elsewhere is refused: reading it would wait
// for the device, and fail in a capture.
struct Freqs {
  const double* p = nullptr;
  at::Tensor as_double;
  std::vector<double> own;

  Freqs(PyObject* o, int32_t rot_dim) {
    if (o == Py_None || rot_dim <= 0) return;
    int64_t n = 0;
    if (THPVariable_Check(o)) {
      const at::Tensor& t = THPVariable_Unpack(o);
      if (!t.is_cpu()) {
        PyObject* where = PyObject_GetAttrString(o, "device");
        PyErr_Format(PyExc_ValueError, "kvs: inv_freq must be in host memory (it is on %S)", where);
        Py_XDECREF(where);
        throw PythonError();
      }
      if (!at::isFloatingType(t.scalar_type()) && !at::isIntegralType(t.scalar_type(), true)) {
        PyErr_SetString(PyExc_TypeError, "kvs: inv_freq must hold real numbers");
        throw PythonError();
      }
      n = t.numel();
      if (t.scalar_type() == at::kFloat && t.is_contiguous()) {  // as models keep them
        const float* x = static_cast<const float*>(t.data_ptr());
        own.assign(x, x + n);
        own.push_back(0);
        p = own.data();
      } else {
        const bool as_it_is = t.scalar_type() == at::kDouble && t.is_contiguous();
        as_double = as_it_is ? t : t.detach().to(at::kDouble).contiguous();
        p = static_cast<const double*>(as_double.data_ptr());
      }
    } else {
      PyObject* all = PySequence_Fast(o, "kvs: inv_freq must be a sequence of numbers");
      if (!all) throw PythonError();
      n = PySequence_Fast_GET_SIZE(all);
      own.resize(n + 1);
      for (int64_t i = 0; i < n; ++i) {
        own[i] = PyFloat_AsDouble(PySequence_Fast_GET_ITEM(all, i));
        if (own[i] == -1.0 && PyErr_Occurred()) break;
      }
      Py_DECREF(all);
      if (PyErr_Occurred()) throw PythonError();
      p = own.data();
    }
    if (n < rot_dim / 2) {
      PyErr_Format(PyExc_ValueError, "kvs: inv_freq holds %lld frequencies, %d needed", (long long)n,
                   rot_dim / 2);
      throw PythonError();
    }
  }
};

void expect(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return;
  PyErr_Format(PyExc_TypeError, "kvs: %zd arguments, %zd needed", got, want);
  throw PythonError();
}

template <class F>
PyObject* guarded(F f) {
  try {
    return PyLong_FromLong(f());
  } catch (const PythonError&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* rope(PyObject*, PyObject* const* x, Py_ssize_t nx) {
  return guarded([&] {
    expect(nx, 11);
    kvs_dims dm;
    dims(x[0], &dm);
    const int32_t N = int32(x[1], "N"), rot = int32(x[3], "rot_dim");
    const Freqs f(x[4], rot);
    const int il = PyObject_IsTrue(x[5]);
    if (il < 0) throw PythonError();
    const Place at(x[10]);
    const int64_t nq = times(dm.L, dm.d, N, dm.H_q), nk = times(dm.L, dm.d, N, dm.H_kv);
    const int32_t* pos = at.i32(x[2], N, "pos");
    const kvs_bf16 *q = at.bf16(x[6], nq, "q"), *k = at.bf16(x[8], nk, "k");
    kvs_bf16 *qo = at.bf16(x[7], nq, "q_out"), *ko = at.bf16(x[9], nk, "k_out");
    kvs_status st;
    Py_BEGIN_ALLOW_THREADS
    st = kvs_rope(&dm, N, pos, rot, f.p, il, q, qo, k, ko, at.stream);
    Py_END_ALLOW_THREADS
    return st;
  });
}

PyObject* append_paged(PyObject*, PyObject* const* x, Py_ssize_t nx) {
  return guarded([&] {
    expect(nx, 25);
    kvs_dims dm;
    dims(x[0], &dm);
    const int32_t B = int32(x[1], "B"), N = int32(x[2], "N"), rot = int32(x[5], "rot_dim");
    const Freqs f(x[6], rot);
    const int il = PyObject_IsTrue(x[7]);
    if (il < 0) throw PythonError();
    const int32_t ps = int32(x[12], "page_size"), cap = int32(x[15], "capacity_pages");
    const int32_t mp = int32(x[19], "max_pages");
    const int64_t ws_bytes = integer(x[23], "ws_bytes", 0, INT64_MAX);
    const Place at(x[24]);
    const int64_t rows = times(dm.L, dm.H_kv, B), nq = times(dm.L, dm.H_q, N, dm.d);
    const int64_t nk = times(dm.L, dm.H_kv, N, dm.d), pool = times(cap, ps, dm.d);
    const int32_t *tok = at.i32(x[3], (int64_t)B + 1, "tok_start"), *pos = at.i32(x[4], N, "pos");
    const kvs_bf16* q = at.bf16(x[8], nq, "q");
    kvs_bf16* qo = at.bf16(x[9], nq, "q_out");
    const kvs_bf16 *k = at.bf16(x[10], nk, "k"), *v = at.bf16(x[11], nk, "v");
    kvs_bf16 *kp = at.bf16(x[13], pool, "k_pages"), *vp = at.bf16(x[14], pool, "v_pages");
    const int32_t* next = at.i32(x[16], 1, "next_page");
    int32_t* next_out = at.i32(x[17], 1, "next_page_out");
    int32_t* bt = at.i32(x[18], times(rows, mp), "block_table");
    const int32_t* sl = at.i32(x[20], rows, "seq_lens");
    int32_t* sl_out = at.i32(x[21], rows, "seq_lens_out");
    void* ws = at.arg<void>(x[22], at::kByte, ws_bytes, "ws");
    kvs_status st;
    Py_BEGIN_ALLOW_THREADS
    st = kvs_append_paged(&dm, B, N, tok, pos, rot, f.p, il, q, qo, k, v, ps, kp, vp, cap, next,
                          next_out, bt, mp, sl, sl_out, ws, (size_t)ws_bytes, at.stream);
    Py_END_ALLOW_THREADS
    return st;
  });
}

PyObject* attn_decode(PyObject*, PyObject* const* x, Py_ssize_t nx) {
  return guarded([&] {
    expect(nx, 19);
    kvs_dims dm;
    dims(x[0], &dm);
    const int32_t B = int32(x[1], "B"), ps = int32(x[3], "page_size");
    const int32_t cap = int32(x[6], "capacity_pages"), mp = int32(x[8], "max_pages");
    const int32_t w = int32(x[10], "w");
    const int64_t ws_bytes = integer(x[17], "ws_bytes", 0, INT64_MAX);
    const Place at(x[18]);
    const int64_t rows = times(dm.L, dm.H_kv, B), heads = times(dm.L, dm.H_q, B);
    const int64_t nq = times(heads, dm.d), pool = times(cap, ps, dm.d), ring = times(rows, w, dm.d);
    const kvs_bf16* q = at.bf16(x[2], nq, "q");
    const kvs_bf16 *kp = at.bf16(x[4], pool, "k_pages"), *vp = at.bf16(x[5], pool, "v_pages");
    const int32_t* bt = at.i32(x[7], times(rows, mp), "block_table");
    const int32_t *sl = at.i32(x[9], rows, "seq_lens"), *pos = at.i32(x[11], w ? B : 0, "pos");
    const kvs_bf16 *rk = at.bf16(x[12], ring, "ring_k"), *rv = at.bf16(x[13], ring, "ring_v");
    kvs_bf16* o = at.bf16(x[14], nq, "o");
    float* lse = at.arg<float>(x[15], at::kFloat, heads, "lse");
    void* ws = at.arg<void>(x[16], at::kByte, ws_bytes, "ws");
    kvs_status st;
    Py_BEGIN_ALLOW_THREADS
    st = kvs_attn_decode(&dm, B, q, ps, kp, vp, cap, bt, mp, sl, w, pos, rk, rv, o, lse, ws,
                         (size_t)ws_bytes, at.stream);
    Py_END_ALLOW_THREADS
    return st;
  });
}

PyObject* attn_tree(PyObject*, PyObject* const* x, Py_ssize_t nx) {
  return guarded([&] {
    expect(nx, 23);
    kvs_dims dm;
    dims(x[0], &dm);
    const int32_t B = int32(x[1], "B"), N = int32(x[2], "N"), md = int32(x[3], "max_draft");
    const int32_t ps = int32(x[7], "page_size"), cap = int32(x[10], "capacity_pages");
    const int32_t mp = int32(x[12], "max_pages"), w = int32(x[14], "w");
    const int64_t ws_bytes = integer(x[21], "ws_bytes", 0, INT64_MAX);
    const Place at(x[22]);
    const int64_t rows = times(dm.L, dm.H_kv, B), heads = times(dm.L, dm.H_q, N);
    const int64_t nq = times(heads, dm.d), pool = times(cap, ps, dm.d), ring = times(rows, w, dm.d);
    const int32_t *tok = at.i32(x[4], (int64_t)B + 1, "tok_start"), *up = at.i32(x[5], N, "parent");
    const kvs_bf16* q = at.bf16(x[6], nq, "q");
    const kvs_bf16 *kp = at.bf16(x[8], pool, "k_pages"), *vp = at.bf16(x[9], pool, "v_pages");
    const int32_t* bt = at.i32(x[11], times(rows, mp), "block_table");
    const int32_t *sl = at.i32(x[13], rows, "seq_lens"), *pos = at.i32(x[15], w ? B : 0, "pos");
    const kvs_bf16 *rk = at.bf16(x[16], ring, "ring_k"), *rv = at.bf16(x[17], ring, "ring_v");
    kvs_bf16* o = at.bf16(x[18], nq, "o");
    float* lse = at.arg<float>(x[19], at::kFloat, heads, "lse");
    void* ws = at.arg<void>(x[20], at::kByte, ws_bytes, "ws");
    kvs_status st;
    Py_BEGIN_ALLOW_THREADS
    st = kvs_attn_tree(&dm, B, N, md, tok, up, q, ps, kp, vp, cap, bt, mp, sl, w, pos, rk, rv, o, lse,
                       ws, (size_t)ws_bytes, at.stream);
    Py_END_ALLOW_THREADS
    return st;
  });
}

PyObject* accept_paged(PyObject*, PyObject* const* x, Py_ssize_t nx) {
  return guarded([&] {
    expect(nx, 15);
    kvs_dims dm;
    dims(x[0], &dm);
    const int32_t B = int32(x[1], "B"), N = int32(x[2], "N"), ps = int32(x[6], "page_size");
    const int32_t cap = int32(x[9], "capacity_pages"), mp = int32(x[11], "max_pages");
    const Place at(x[14]);
    const int64_t rows = times(dm.L, dm.H_kv, B), pool = times(cap, ps, dm.d);
    const int32_t *tok = at.i32(x[3], (int64_t)B + 1, "tok_start"), *n = at.i32(x[4], B, "n_accept");
    const int32_t* path = at.i32(x[5], N, "accept");
    kvs_bf16 *kp = at.bf16(x[7], pool, "k_pages"), *vp = at.bf16(x[8], pool, "v_pages");
    const int32_t* bt = at.i32(x[10], times(rows, mp), "block_table");
    const int32_t* sl = at.i32(x[12], rows, "seq_lens");
    int32_t* sl_out = at.i32(x[13], rows, "seq_lens_out");
    kvs_status st;
    Py_BEGIN_ALLOW_THREADS
    st = kvs_accept_paged(&dm, B, N, tok, n, path, ps, kp, vp, cap, bt, mp, sl, sl_out, at.stream);
    Py_END_ALLOW_THREADS
    return st;
  });
}

PyObject* fork_paged(PyObject*, PyObject* const* x, Py_ssize_t nx) {
  return guarded([&] {
    expect(nx, 22);
    kvs_dims dm;
    dims(x[0], &dm);
    const int32_t B = int32(x[1], "B"), forks = int32(x[2], "n_forks"), ps = int32(x[5], "page_size");
    const int32_t cap = int32(x[8], "capacity_pages"), mp = int32(x[12], "max_pages");
    const int32_t w = int32(x[14], "w");
    const int64_t ws_bytes = integer(x[20], "ws_bytes", 0, INT64_MAX);
    const Place at(x[21]);
    const int64_t rows = times(dm.L, dm.H_kv, B), pool = times(cap, ps, dm.d), ring = times(rows, w);
    const int32_t *src = at.i32(x[3], forks, "src"), *dst = at.i32(x[4], forks, "dst");
    kvs_bf16 *kp = at.bf16(x[6], pool, "k_pages"), *vp = at.bf16(x[7], pool, "v_pages");
    const int32_t* next = at.i32(x[9], 1, "next_page");
    int32_t* next_out = at.i32(x[10], 1, "next_page_out");
    int32_t* bt = at.i32(x[11], times(rows, mp), "block_table");
    int32_t *sl = at.i32(x[13], rows, "seq_lens"), *pos = at.i32(x[15], w ? B : 0, "pos");
    float* score = at.arg<float>(x[16], at::kFloat, ring, "ring_score");
    kvs_bf16* rk = at.bf16(x[17], times(ring, dm.d), "ring_k");
    kvs_bf16* rv = at.bf16(x[18], times(ring, dm.d), "ring_v");
    void* ws = at.arg<void>(x[19], at::kByte, ws_bytes, "ws");
    kvs_status st;
    Py_BEGIN_ALLOW_THREADS
    st = kvs_fork_paged(&dm, B, forks, src, dst, ps, kp, vp, cap, next, next_out, bt, mp, sl, w, pos,
                        score, rk, rv, ws, (size_t)ws_bytes, at.stream);
    Py_END_ALLOW_THREADS
    return st;
  });
}

PyObject* reclaim_paged(PyObject*, PyObject* const* x, Py_ssize_t nx) {
  return guarded([&] {
    expect(nx, 15);
    kvs_dims dm;
    dims(x[0], &dm);
    const int32_t B = int32(x[1], "B"), ps = int32(x[2], "page_size");
    const int32_t cap = int32(x[5], "capacity_pages"), mp = int32(x[10], "max_pages");
    const int64_t ws_bytes = integer(x[13], "ws_bytes", 0, INT64_MAX);
    const Place at(x[14]);
    const int64_t rows = times(dm.L, dm.H_kv, B), pool = times(cap, ps, dm.d);
    kvs_bf16 *kp = at.bf16(x[3], pool, "k_pages"), *vp = at.bf16(x[4], pool, "v_pages");
    const int32_t* next = at.i32(x[6], 1, "next_page");
    int32_t* next_out = at.i32(x[7], 1, "next_page_out");
    const int32_t* bt = at.i32(x[8], times(rows, mp), "block_table");
    int32_t* bt_out = at.i32(x[9], times(rows, mp), "block_table_out");
    const int32_t* sl = at.i32(x[11], rows, "seq_lens");
    void* ws = at.arg<void>(x[12], at::kByte, ws_bytes, "ws");
    kvs_status st;
    Py_BEGIN_ALLOW_THREADS
    st = kvs_reclaim_paged(&dm, B, ps, kp, vp, cap, next, next_out, bt, bt_out, mp, sl, ws,
                           (size_t)ws_bytes, at.stream);
    Py_END_ALLOW_THREADS
    return st;
  });
}

PyMethodDef methods[] = {
    {"rope", (PyCFunction)(void (*)())rope, METH_FASTCALL, nullptr},
    {"append_paged", (PyCFunction)(void (*)())append_paged, METH_FASTCALL, nullptr},
    {"attn_decode", (PyCFunction)(void (*)())attn_decode, METH_FASTCALL, nullptr},
    {"attn_tree", (PyCFunction)(void (*)())attn_tree, METH_FASTCALL, nullptr},
    {"accept_paged", (PyCFunction)(void (*)())accept_paged, METH_FASTCALL, nullptr},
    {"fork_paged", (PyCFunction)(void (*)())fork_paged, METH_FASTCALL, nullptr},
    {"reclaim_paged", (PyCFunction)(void (*)())reclaim_paged, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "kvs_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_kvs_binding() {
  return PyModule_Create(&module);
}
