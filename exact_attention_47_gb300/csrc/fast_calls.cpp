// The usual case of the rotary, append and 4-bit-cache calls, marshalled in
// C++: a decode step's kernels take 3 to 8 us each, and checking and passing
// their tensors from Python took 15 to 20.
//
// Each function here takes the positional arguments of its namesake in
// _binding.py, checks what that checks, allocates the outputs that are not
// given and calls the C entry point of the library (whose addresses `bind`
// receives), with the GIL released for the last two.  Whatever is not the
// usual case (tensors of another device, type or layout than wanted, another
// current device, arguments that the library refuses) makes it return None, and
// the Python function goes its own, longer way, which raises the errors.  A
// status that may come after a launch is returned as a number, for the Python
// function to raise: the call is not made again (a rotation in place would turn
// twice).
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>

#include "attn47.h"

namespace {

// No GIL while this lives: a launch may have to wait for the GPU, and an
// allocation may free blocks.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

decltype(&rope_fwd) g_rope_fwd = nullptr;
decltype(&rope_bwd) g_rope_bwd = nullptr;
decltype(&rope_append_paged) g_append = nullptr;
decltype(&rope_append_paged_kv4) g_append_kv4 = nullptr;
decltype(&kv4_record_bytes) g_record_bytes = nullptr;
decltype(&kv4_read_paged) g_read = nullptr;
decltype(&attn_decode_paged_kv4_workspace_size) g_workspace_size = nullptr;
decltype(&attn_decode_paged_kv4) g_decode = nullptr;

constexpr int kBlock = 16;   // cached tokens of a block

// The tensor of an argument, or nullptr: not one, not on the GPU `device` (any
// if -1), not of `type`.
const at::Tensor* tensor(PyObject* o, at::ScalarType type, int device) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || !t.is_cuda() || t.scalar_type() != type || (device >= 0 && t.get_device() != device))
    return nullptr;
  return &t;
}
const at::Tensor* packed(PyObject* o, at::ScalarType type, int device, int dim) {
  const at::Tensor* t = tensor(o, type, device);
  return t && t->dim() == dim && t->is_contiguous() ? t : nullptr;
}
template <class T>
T* data(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}
template <class T>
T* data(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
bool small(int64_t v) { return v >= 0 && v <= 0x7fffffff; }
bool integer(PyObject* o, int* out) {
  if (!PyLong_CheckExact(o)) return false;
  int overflow = 0;
  const long v = PyLong_AsLongAndOverflow(o, &overflow);
  if (overflow || v < 0 || v > 0x7fffffff) return false;
  *out = static_cast<int>(v);
  return true;
}
bool truth(PyObject* o, int* out) {
  if (!PyBool_Check(o)) return false;
  *out = o == Py_True;
  return true;
}

int64_t step(const at::Tensor& t, int i) { return t.size(i) > 1 ? t.stride(i) : 0; }

// attn_heads_t of [B, H, N, d] or [T, H, d].
bool heads(const at::Tensor& t, attn_heads_t* h) {
  const int dim = static_cast<int>(t.dim());
  if (t.stride(dim - 1) != 1 && t.size(dim - 1) > 1) return false;
  if (!small(t.size(1))) return false;
  h->data = t.data_ptr();
  h->stride_batch = dim == 4 ? step(t, 0) : 0;
  h->stride_token = dim == 4 ? step(t, 2) : step(t, 0);
  h->stride_head = step(t, 1);
  h->heads = static_cast<int>(t.size(1));
  return true;
}

// attn_rope_t; `lead` (`dims` sizes) is the shape that a position axis may
// have, or its last size alone.
struct Rope {
  attn_rope_t r;
  uint8_t axis[64];
  bool fill(PyObject* inv_freq, PyObject* positions, const int64_t* lead, int dims, PyObject* pair_axis,
            PyObject* interleaved, int device) {
    const at::Tensor* f = packed(inv_freq, at::kFloat, device, 1);
    int il = 0;
    if (!f || f->size(0) > 64 || !truth(interleaved, &il)) return false;
    const int pairs = static_cast<int>(f->size(0));
    r = attn_rope_t{data<float>(f), 2 * pairs, il, nullptr, 1, 0, 0, nullptr};
    const bool table = pair_axis != Py_None;
    if (table) {
      if (PyBytes_CheckExact(pair_axis) && PyBytes_GET_SIZE(pair_axis) == pairs) {
        std::memcpy(axis, PyBytes_AS_STRING(pair_axis), pairs);
      } else if ((PyList_CheckExact(pair_axis) || PyTuple_CheckExact(pair_axis)) &&
                 PySequence_Fast_GET_SIZE(pair_axis) == pairs) {
        PyObject** item = PySequence_Fast_ITEMS(pair_axis);
        for (int i = 0; i < pairs; ++i) {
          int a = 0;
          if (!integer(item[i], &a) || a > 255) return false;
          axis[i] = static_cast<uint8_t>(a);
        }
      } else {
        return false;
      }
      r.pair_axis = axis;
    }
    if (positions == Py_None) return !table;
    const at::Tensor* p = tensor(positions, at::kInt, device);
    if (!p) return false;
    const int64_t skip = table ? 1 : 0, left = p->dim() - skip;
    if (left < 1 || left > dims) return false;
    for (int64_t i = 0; i < left; ++i)
      if (p->size(skip + i) != lead[dims - left + i]) return false;
    if (p->size(p->dim() - 1) > 1 && p->stride(p->dim() - 1) != 1) return false;
    if (table) {
      if (!small(p->size(0))) return false;
      r.axes = static_cast<int>(p->size(0));
      r.stride_axis = step(*p, 0);
    }
    if (left == 2) r.stride_batch = step(*p, static_cast<int>(skip));
    r.positions = data<int32_t>(p);
    return true;
  }
};

// A new tensor, past torch's dispatcher: an `at::empty` takes 1.45 us here,
// this 0.9, and a decode call makes two.
at::Tensor make(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor& like) {
  return at::detail::empty_cuda(sizes, type, like.device(), std::nullopt);
}
void* stream_of(int device) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }
bool current(int device) { return c10::cuda::current_device() == device; }

// This thread's call has reached the library.
thread_local bool t_called = false;

// For a status other than ATTN_OK: None where nothing was launched.
PyObject* not_done(attn_status_t st) {
  if (st == ATTN_ERR_INVALID_ARG || st == ATTN_ERR_UNSUPPORTED || st == ATTN_ERR_WORKSPACE) Py_RETURN_NONE;
  return PyLong_FromLong(st);
}

PyObject* pair(const at::Tensor& a, const at::Tensor* b) {
  PyObject* t = PyTuple_New(2);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(t, 1, b ? THPVariable_Wrap(*b) : Py_NewRef(Py_None));
  return t;
}

// A caller-given output (null: none was given, one has to be made), or false.
bool output(PyObject* o, at::IntArrayRef sizes, at::ScalarType type, int device, bool any_strides,
            const at::Tensor** given) {
  *given = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o, type, device);
  if (!t || t->sizes() != sizes || (!any_strides && !t->is_contiguous())) return false;
  *given = t;
  return true;
}

// rope(back, q, k, positions, inv_freq, pair_axis, interleaved, q_out, k_out)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  int back = 0;
  if (n != 9 || !g_rope_fwd || !truth(a[0], &back)) Py_RETURN_NONE;
  const at::Tensor* q = tensor(a[1], at::kBFloat16, -1);
  if (!q || q->dim() != 4) Py_RETURN_NONE;
  const int dev = static_cast<int>(q->get_device());
  const at::Tensor* k = nullptr;
  const int64_t B = q->size(0), N = q->size(2), d = q->size(3);
  if (a[2] != Py_None) {
    k = tensor(a[2], at::kBFloat16, dev);
    if (!k || k->dim() != 4 || k->size(0) != B || k->size(2) != N || k->size(3) != d) Py_RETURN_NONE;
  } else if (a[8] != Py_None) {
    Py_RETURN_NONE;
  }
  const int64_t lead[2] = {B, N};
  attn_heads_t hq, hk, ho, hko;
  Rope r;
  if (!small(B) || !small(N) || !small(d) || !current(dev) || !heads(*q, &hq) || (k && !heads(*k, &hk)) ||
      !r.fill(a[4], a[3], lead, 2, a[5], a[6], dev))
    Py_RETURN_NONE;
  const at::Tensor *q_given, *k_given = nullptr;
  if (!output(a[7], q->sizes(), at::kBFloat16, dev, true, &q_given) || (q_given && !heads(*q_given, &ho))) Py_RETURN_NONE;
  if (k && (!output(a[8], k->sizes(), at::kBFloat16, dev, true, &k_given) || (k_given && !heads(*k_given, &hko))))
    Py_RETURN_NONE;
  at::Tensor qo, ko;
  attn_status_t st;
  {
    Unlocked unlocked;
    qo = q_given ? *q_given : make(q->sizes(), at::kBFloat16, *q);
    heads(qo, &ho);
    if (k) {
      ko = k_given ? *k_given : make(k->sizes(), at::kBFloat16, *k);
      heads(ko, &hko);
    }
    t_called = true;
    st = (back ? g_rope_bwd : g_rope_fwd)(&hq, k ? &hk : nullptr, &ho, k ? &hko : nullptr, &r.r, static_cast<int>(B),
                                          static_cast<int>(N), static_cast<int>(d), stream_of(dev));
  }
  if (st != ATTN_OK) return not_done(st);
  return pair(qo, k ? &ko : nullptr);
}

// append(q, k, v, k_cache, v_cache, block_table, seq_ids, positions, group, inv_freq, rope_positions, pair_axis,
// interleaved, q_out); a 4-bit cache comes as k_cache with v_cache None.  Returns (q_out or None,).
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  int group = 0;
  if (n != 14 || !g_append || !integer(a[8], &group)) Py_RETURN_NONE;
  const at::Tensor* k = tensor(a[1], at::kBFloat16, -1);
  if (!k || k->dim() != 3) Py_RETURN_NONE;
  const int dev = static_cast<int>(k->get_device());
  const at::Tensor* v = tensor(a[2], at::kBFloat16, dev);
  if (!v || v->sizes() != k->sizes()) Py_RETURN_NONE;
  const int64_t T = k->size(0), Hkv = k->size(1), d = k->size(2);
  const at::Tensor* table = packed(a[5], at::kInt, dev, 2);
  const at::Tensor* ids = packed(a[6], at::kInt, dev, 1);
  const at::Tensor* pos = packed(a[7], at::kInt, dev, 1);
  if (!table || !ids || !pos || ids->size(0) != T || pos->size(0) != T || !small(T) || !small(Hkv) || !small(d) ||
      !small(table->size(0)) || !small(table->size(1)) || !current(dev))
    Py_RETURN_NONE;
  const bool kv4 = a[4] == Py_None;
  const at::Tensor *kc, *vc = nullptr;
  int block = kBlock;
  if (kv4) {
    kc = packed(a[3], at::kByte, dev, 3);
    const size_t rec = kc ? g_record_bytes(static_cast<int>(d), group) : 0;
    if (!kc || rec == 0 || kc->size(1) != Hkv || kc->size(2) != static_cast<int64_t>(rec)) Py_RETURN_NONE;
  } else {
    kc = packed(a[3], at::kBFloat16, dev, 4);
    vc = packed(a[4], at::kBFloat16, dev, 4);
    if (!kc || !vc || kc->sizes() != vc->sizes() || kc->size(1) != Hkv || kc->size(3) != d || !small(kc->size(2)))
      Py_RETURN_NONE;
    block = static_cast<int>(kc->size(2));
  }
  if (!small(kc->size(0))) Py_RETURN_NONE;
  attn_heads_t hq, hk, hv, ho;
  if (!heads(*k, &hk) || !heads(*v, &hv)) Py_RETURN_NONE;
  const at::Tensor* q = nullptr;
  if (a[0] != Py_None) {
    q = tensor(a[0], at::kBFloat16, dev);
    if (!q || q->dim() != 3 || q->size(0) != T || q->size(2) != d || !heads(*q, &hq)) Py_RETURN_NONE;
  } else if (a[13] != Py_None) {
    Py_RETURN_NONE;
  }
  Rope r;
  const bool turn = a[9] != Py_None;
  if (turn ? !r.fill(a[9], a[10], &T, 1, a[11], a[12], dev) : (a[10] != Py_None || a[11] != Py_None)) Py_RETURN_NONE;
  const at::Tensor* q_given = nullptr;
  if (q && (!output(a[13], q->sizes(), at::kBFloat16, dev, true, &q_given) || (q_given && !heads(*q_given, &ho))))
    Py_RETURN_NONE;
  const int t = static_cast<int>(T), S = static_cast<int>(table->size(0)), mb = static_cast<int>(table->size(1)),
            nb = static_cast<int>(kc->size(0)), dd = static_cast<int>(d);
  const attn_heads_t *pq = q ? &hq : nullptr, *po = q ? &ho : nullptr;
  const attn_rope_t* pr = turn ? &r.r : nullptr;
  at::Tensor qo;
  attn_status_t st;
  {
    Unlocked unlocked;
    if (q) {
      qo = q_given ? *q_given : make(q->sizes(), at::kBFloat16, *q);
      heads(qo, &ho);
    }
    t_called = true;
    st = kv4 ? g_append_kv4(pq, &hk, &hv, po, pr, data<void>(kc), group, data<int32_t>(table), data<int32_t>(ids),
                            data<int32_t>(pos), t, S, dd, block, mb, nb, stream_of(dev))
             : g_append(pq, &hk, &hv, po, pr, data<void>(kc), data<void>(vc), data<int32_t>(table),
                        data<int32_t>(ids), data<int32_t>(pos), t, S, dd, block, mb, nb, stream_of(dev));
  }
  if (st != ATTN_OK) return not_done(st);
  PyObject* out = PyTuple_New(1);
  if (out) PyTuple_SET_ITEM(out, 0, q ? THPVariable_Wrap(qo) : Py_NewRef(Py_None));
  return out;
}

// read(kv_cache, block_table, seq_ids, positions, d, group, k, v)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  int d = 0, group = 0;
  if (n != 8 || !g_read || !integer(a[4], &d) || !integer(a[5], &group)) Py_RETURN_NONE;
  const at::Tensor* kv = packed(a[0], at::kByte, -1, 3);
  if (!kv) Py_RETURN_NONE;
  const int dev = static_cast<int>(kv->get_device());
  const size_t rec = g_record_bytes(d, group);
  const at::Tensor* table = packed(a[1], at::kInt, dev, 2);
  const at::Tensor* ids = packed(a[2], at::kInt, dev, 1);
  const at::Tensor* pos = packed(a[3], at::kInt, dev, 1);
  if (rec == 0 || kv->size(2) != static_cast<int64_t>(rec) || !table || !ids || !pos || pos->size(0) != ids->size(0) ||
      !small(ids->size(0)) || !small(kv->size(0)) || !small(kv->size(1)) || !small(table->size(0)) ||
      !small(table->size(1)) || !current(dev))
    Py_RETURN_NONE;
  const int64_t sizes[3] = {ids->size(0), kv->size(1), d};
  const at::Tensor *k_given, *v_given;
  if (!output(a[6], sizes, at::kBFloat16, dev, false, &k_given) ||
      !output(a[7], sizes, at::kBFloat16, dev, false, &v_given))
    Py_RETURN_NONE;
  at::Tensor k, v;
  attn_status_t st;
  {
    Unlocked unlocked;
    k = k_given ? *k_given : make(sizes, at::kBFloat16, *kv);
    v = v_given ? *v_given : make(sizes, at::kBFloat16, *kv);
    t_called = true;
    st = g_read(data<void>(kv), group, data<int32_t>(table), data<int32_t>(ids), data<int32_t>(pos), data<void>(k),
                data<void>(v), static_cast<int>(sizes[0]), static_cast<int>(table->size(0)),
                static_cast<int>(sizes[1]), d, kBlock, static_cast<int>(table->size(1)), static_cast<int>(kv->size(0)),
                stream_of(dev));
  }
  if (st != ATTN_OK) return not_done(st);
  return pair(k, &v);
}

// decode(q, kv_cache, block_table, seq_lens, group, scale, o, lse, workspace, return_lse)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  int group = 0, want_lse = 0;
  if (n != 10 || !g_decode || !integer(a[4], &group) || !truth(a[9], &want_lse)) Py_RETURN_NONE;
  const at::Tensor* q = packed(a[0], at::kBFloat16, -1, 3);
  if (!q) Py_RETURN_NONE;
  const int dev = static_cast<int>(q->get_device());
  const int64_t S = q->size(0), Hq = q->size(1), d = q->size(2);
  const at::Tensor* kv = packed(a[1], at::kByte, dev, 3);
  const at::Tensor* table = packed(a[2], at::kInt, dev, 2);
  const at::Tensor* lens = packed(a[3], at::kInt, dev, 1);
  if (!kv || !table || !lens || table->size(0) != S || lens->size(0) != S || !small(S) || !small(Hq) || !small(d) ||
      !small(kv->size(0)) || !small(kv->size(1)) || !small(table->size(1)) || !current(dev))
    Py_RETURN_NONE;
  const size_t rec = g_record_bytes(static_cast<int>(d), group);
  if (rec == 0 || kv->size(2) != static_cast<int64_t>(rec)) Py_RETURN_NONE;
  float scale;
  if (a[5] == Py_None)
    scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
  else if (PyFloat_CheckExact(a[5]))
    scale = static_cast<float>(PyFloat_AS_DOUBLE(a[5]));
  else
    Py_RETURN_NONE;
  const int Hkv = static_cast<int>(kv->size(1));
  const int64_t lse_sizes[2] = {S, Hq};
  const bool has_lse = a[7] != Py_None || want_lse;
  const size_t need = g_workspace_size(static_cast<int>(S), static_cast<int>(Hq), Hkv, static_cast<int>(d));
  const at::Tensor *o_given, *lse_given = nullptr, *ws_given = nullptr;
  if (!output(a[6], q->sizes(), at::kBFloat16, dev, false, &o_given) ||
      (has_lse && !output(a[7], lse_sizes, at::kFloat, dev, false, &lse_given)))
    Py_RETURN_NONE;
  if (a[8] != Py_None) {
    if (!THPVariable_Check(a[8])) Py_RETURN_NONE;
    ws_given = &THPVariable_Unpack(a[8]);
    if (!ws_given->defined() || !ws_given->is_cuda() || ws_given->get_device() != dev || !ws_given->is_contiguous() ||
        ws_given->nbytes() < need)
      Py_RETURN_NONE;
  }
  at::Tensor o, lse, ws;
  attn_status_t st;
  {
    Unlocked unlocked;
    o = o_given ? *o_given : make(q->sizes(), at::kBFloat16, *q);
    if (has_lse) lse = lse_given ? *lse_given : make(lse_sizes, at::kFloat, *q);
    ws = ws_given ? *ws_given : make({static_cast<int64_t>(need < 16 ? 16 : need)}, at::kByte, *q);
    t_called = true;
    st = g_decode(data<void>(q), data<void>(kv), data<int32_t>(table), data<int32_t>(lens), static_cast<int>(S),
                  static_cast<int>(Hq), Hkv, static_cast<int>(d), group, kBlock, static_cast<int>(table->size(1)),
                  static_cast<int>(kv->size(0)), scale, data<void>(o), has_lse ? data<float>(lse) : nullptr,
                  data<void>(ws), ws.nbytes(), stream_of(dev));
  }
  if (st != ATTN_OK) return not_done(st);
  return pair(o, has_lse ? &lse : nullptr);
}

// C++ exceptions (an allocation that failed, say) become "not handled": the
// Python function meets the same and raises it.  Not so once the library has
// been called.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  t_called = false;
  try {
    return F(self, a, n);
  } catch (...) {
    if (t_called) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "the call was made, but its results could not be returned");
      return nullptr;
    }
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "bind takes 8 addresses");
    return nullptr;
  }
  void* p[8];
  for (int i = 0; i < 8; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  g_rope_fwd = reinterpret_cast<decltype(g_rope_fwd)>(p[0]);
  g_rope_bwd = reinterpret_cast<decltype(g_rope_bwd)>(p[1]);
  g_append = reinterpret_cast<decltype(g_append)>(p[2]);
  g_append_kv4 = reinterpret_cast<decltype(g_append_kv4)>(p[3]);
  g_record_bytes = reinterpret_cast<decltype(g_record_bytes)>(p[4]);
  g_read = reinterpret_cast<decltype(g_read)>(p[5]);
  g_workspace_size = reinterpret_cast<decltype(g_workspace_size)>(p[6]);
  g_decode = reinterpret_cast<decltype(g_decode)>(p[7]);
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef methods[] = {{"bind", FAST(bind), METH_FASTCALL, nullptr},
                         {"rope", FAST(guarded<rope>), METH_FASTCALL, nullptr},
                         {"append", FAST(guarded<append>), METH_FASTCALL, nullptr},
                         {"read", FAST(guarded<read>), METH_FASTCALL, nullptr},
                         {"decode", FAST(guarded<decode>), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn47_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn47_fast() { return PyModule_Create(&module); }
