// The short way from Python into libpa.so for the calls whose launch takes a
// few microseconds: checks a call's tensors and passes their pointers, which
// through ctypes costs several times the launch itself. Whatever it does not
// take — a wrong type, shape or layout, another device, an explicit stream —
// it leaves alone by returning None, and the Python binding goes the long
// way, which says what is wrong. Otherwise it returns the call's status.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>

#include "pa.h"

namespace {

// The tensors of one call: all on one CUDA device, the current one.
struct Call {
  PyObject *const *args;
  int device = -1;
  bool fine = true;

  const at::Tensor *tensor(int i, int dims, bool contiguous = true) {
    static const at::Tensor none;
    if (!fine || !THPVariable_Check(args[i])) {
      fine = false;
      return &none;
    }
    const at::Tensor &t = THPVariable_Unpack(args[i]);
    if (!t.defined() || !t.is_cuda() || t.dim() != dims || (contiguous && !t.is_contiguous())) fine = false;
    for (const int64_t n : t.sizes()) fine = fine && n <= INT32_MAX;  // sizes are passed as int
    if (fine && device < 0) device = t.get_device();
    if (fine && t.get_device() != device) fine = false;
    return fine ? &t : &none;
  }
  const at::Tensor *typed(int i, int dims, at::ScalarType type) {
    const at::Tensor *t = tensor(i, dims);
    if (fine && t->scalar_type() != type) fine = false;
    return t;
  }
  // a token's heads contiguous, any distance between tokens
  const at::Tensor *rows(int i, int64_t *stride) {
    const at::Tensor *t = tensor(i, 3, false);
    if (fine && (t->scalar_type() != at::kBFloat16 || t->stride(2) != 1 ||
                 (t->stride(1) != t->size(2) && t->size(1) != 1)))
      fine = false;
    if (fine) *stride = t->size(0) > 1 ? t->stride(0) : t->size(1) * t->size(2);
    return t;
  }
  const at::Tensor *cache(int i, pa_kv_dtype *kv) {
    const at::Tensor *t = tensor(i, 4);
    if (!fine) return t;
    if (t->scalar_type() == at::kBFloat16)
      *kv = PA_KV_BF16;
    else if (t->scalar_type() == at::kFloat8_e4m3fn || t->scalar_type() == at::kByte)
      *kv = PA_KV_FP8_E4M3;
    else
      fine = false;
    return t;
  }
  // numbers as ctypes takes them; sizes beyond an int go the long way
  int integer(int i) {
    const long v = fine ? PyLong_AsLong(args[i]) : 0;
    return number(v >= INT32_MIN && v <= INT32_MAX) ? static_cast<int>(v) : 0;
  }
  float real(int i) {
    const double v = fine ? PyFloat_AsDouble(args[i]) : 0.0;
    return number(true) ? static_cast<float>(v) : 0.f;
  }
  bool number(bool in_range) {
    if (fine && PyErr_Occurred()) {
      PyErr_Clear();
      fine = false;
    }
    if (!in_range) fine = false;
    return fine;
  }
  bool ready() {
    if (fine && c10::cuda::current_device() != device) fine = false;
    return fine;
  }
  void *stream() const { return c10::cuda::getCurrentCUDAStream(device).stream(); }
};

// The library's status as a Python number, its launch made without the
// interpreter's lock (a full launch queue blocks).
template <typename F>
PyObject *status_of(F &&launch) {
  pa_status rc;
  Py_BEGIN_ALLOW_THREADS
  rc = launch();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

// A method that never throws into the interpreter.
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *, PyObject *const *args, Py_ssize_t n) {
  try {
    return F(args, n);
  } catch (const std::exception &) {  // a tensor without storage, no memory: the long way says so
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

template <typename T>
T *ptr(const at::Tensor *t) {
  return static_cast<T *>(t->data_ptr());
}
int len(const at::Tensor *t, int d) { return static_cast<int>(t->size(d)); }

// (block_tables, context_lens, new_lens, free_blocks, free_count,
// context_lens_out, free_count_out, slot_mapping, positions, query_start,
// num_blocks or None)
PyObject *extend_tables(PyObject *const *args, Py_ssize_t n) {
  if (n != 11) Py_RETURN_NONE;
  Call c{args};
  const at::Tensor *bt = c.typed(0, 2, at::kInt), *lens = c.typed(1, 1, at::kInt), *more = c.typed(2, 1, at::kInt),
                   *free = c.typed(3, 1, at::kInt), *count = c.typed(4, 1, at::kInt),
                   *lens_out = c.typed(5, 1, at::kInt), *count_out = c.typed(6, 1, at::kInt),
                   *slots = c.typed(7, 1, at::kLong), *pos = c.typed(8, 1, at::kInt), *qs = c.typed(9, 1, at::kInt);
  const bool whole = args[10] == Py_None;  // the pool is as large as the stack
  int nb = whole ? 0 : c.integer(10);
  if (!c.ready()) Py_RETURN_NONE;
  const int64_t S = bt->size(0);
  if (lens->size(0) != S || more->size(0) != S || lens_out->size(0) != S || count->size(0) != 1 ||
      count_out->size(0) != 1 || pos->size(0) != slots->size(0) || qs->size(0) != S + 1)
    Py_RETURN_NONE;
  if (whole) nb = len(free, 0);
  return status_of([&] {
    return pa_extend_tables(ptr<int32_t>(bt), len(bt, 1), ptr<int32_t>(lens), ptr<int32_t>(more), ptr<int32_t>(free),
                            len(free, 0), ptr<int32_t>(count), ptr<int32_t>(lens_out), ptr<int32_t>(count_out),
                            ptr<int64_t>(slots), ptr<int32_t>(pos), ptr<int32_t>(qs), static_cast<int>(S),
                            len(slots, 0), 16, nb, c.stream());
  });
}

// (block_tables, context_lens, release, free_blocks, free_count,
// context_lens_out, free_count_out, keep_blocks, num_blocks or None)
PyObject *release_tables(PyObject *const *args, Py_ssize_t n) {
  if (n != 9) Py_RETURN_NONE;
  Call c{args};
  const at::Tensor *bt = c.typed(0, 2, at::kInt), *lens = c.typed(1, 1, at::kInt), *rel = c.typed(2, 1, at::kInt),
                   *free = c.typed(3, 1, at::kInt), *count = c.typed(4, 1, at::kInt),
                   *lens_out = c.typed(5, 1, at::kInt), *count_out = c.typed(6, 1, at::kInt);
  const int keep = c.integer(7);
  const bool whole = args[8] == Py_None;
  int nb = whole ? 0 : c.integer(8);
  if (!c.ready()) Py_RETURN_NONE;
  const int64_t S = bt->size(0);
  if (lens->size(0) != S || rel->size(0) != S || lens_out->size(0) != S || count->size(0) != 1 ||
      count_out->size(0) != 1)
    Py_RETURN_NONE;
  if (whole) nb = len(free, 0);
  return status_of([&] {
    return pa_release_tables(ptr<int32_t>(bt), len(bt, 1), ptr<int32_t>(lens), ptr<int32_t>(rel), ptr<int32_t>(free),
                             len(free, 0), ptr<int32_t>(count), ptr<int32_t>(lens_out), ptr<int32_t>(count_out), keep,
                             static_cast<int>(S), 16, nb, c.stream());
  });
}

// (q_out, q, key, value, k_cache, v_cache, slot_mapping, positions, inv_freq,
// interleaved, rope_scale, k_scale, v_scale)
PyObject *rope_and_cache(PyObject *const *args, Py_ssize_t n) {
  if (n != 13) Py_RETURN_NONE;
  Call c{args};
  int64_t qs = 0, ks = 0, vs = 0;
  pa_kv_dtype kv = PA_KV_BF16, kv2 = PA_KV_BF16;
  const at::Tensor *out = c.typed(0, 3, at::kBFloat16), *q = c.rows(1, &qs), *k = c.rows(2, &ks), *v = c.rows(3, &vs),
                   *kc = c.cache(4, &kv), *vc = c.cache(5, &kv2), *slots = c.typed(6, 1, at::kLong),
                   *pos = c.typed(7, 1, at::kInt), *inv = c.typed(8, 1, at::kDouble);
  const int il = c.fine ? PyObject_IsTrue(args[9]) : 0;
  const float scale = c.real(10), k_scale = c.real(11), v_scale = c.real(12);
  if (il < 0) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  if (!c.ready()) Py_RETURN_NONE;
  const int64_t T = q->size(0), D = q->size(2), Hkv = kc->size(1);
  if (out->sizes() != q->sizes() || kc->size(3) != D || vc->sizes() != kc->sizes() ||
      vc->scalar_type() != kc->scalar_type() || k->size(0) != T || k->size(1) != Hkv || k->size(2) != D ||
      v->sizes() != k->sizes() || slots->size(0) != T || pos->size(0) != T)
    Py_RETURN_NONE;
  return status_of([&] {
    return pa_rope_and_cache(ptr<void>(out), ptr<void>(q), ptr<void>(k), ptr<void>(v), ptr<void>(kc), ptr<void>(vc),
                             ptr<int64_t>(slots), ptr<int32_t>(pos), ptr<double>(inv), 2 * len(inv, 0), il, scale, qs,
                             ks, vs, static_cast<int>(T), len(q, 1), static_cast<int>(Hkv), static_cast<int>(D),
                             len(kc, 2), len(kc, 0), kv, k_scale, v_scale, c.stream());
  });
}

// (out, q, k_cache, v_cache, block_tables, context_lens, max_context_len,
// group_start, prefix_blocks, max_prefix_blocks, max_suffix_len, sm_scale,
// k_scale, v_scale); the workspace is allocated on the current stream.
PyObject *decode_shared_prefix(PyObject *const *args, Py_ssize_t n) {
  if (n != 14) Py_RETURN_NONE;
  Call c{args};
  pa_kv_dtype kv = PA_KV_BF16, kv2 = PA_KV_BF16;
  const at::Tensor *out = c.typed(0, 3, at::kFloat), *q = c.typed(1, 3, at::kBFloat16), *kc = c.cache(2, &kv),
                   *vc = c.cache(3, &kv2), *bt = c.typed(4, 2, at::kInt), *lens = c.typed(5, 1, at::kInt),
                   *start = c.typed(7, 1, at::kInt), *blocks = c.typed(8, 1, at::kInt);
  const int max_len = c.integer(6), max_prefix = c.integer(9), max_suffix = c.integer(10);
  const float sm_scale = c.real(11), k_scale = c.real(12), v_scale = c.real(13);
  if (!c.ready()) Py_RETURN_NONE;
  const int64_t S = q->size(0), G = blocks->size(0);
  if (out->sizes() != q->sizes() || kc->size(3) != q->size(2) || vc->sizes() != kc->sizes() ||
      vc->scalar_type() != kc->scalar_type() || bt->size(0) != S || lens->size(0) != S || start->size(0) != G + 1)
    Py_RETURN_NONE;
  const int Hq = len(q, 1), Hkv = len(kc, 1), D = len(q, 2);
  const size_t bytes = pa_decode_shared_prefix_workspace_size(static_cast<int>(S), Hq, Hkv, D, static_cast<int>(G),
                                                              max_prefix, max_suffix);
  const at::Tensor ws = at::empty({static_cast<int64_t>(bytes)}, q->options().dtype(at::kByte));
  return status_of([&] {
    return pa_decode_shared_prefix(ptr<float>(out), ptr<void>(q), ptr<void>(kc), ptr<void>(vc), kv, k_scale, v_scale,
                                   ptr<int32_t>(bt), len(bt, 1), ptr<int32_t>(lens), max_len, ptr<int32_t>(start),
                                   ptr<int32_t>(blocks), static_cast<int>(G), max_prefix, max_suffix,
                                   static_cast<int>(S), Hq, Hkv, D, len(kc, 2), len(kc, 0), sm_scale, ws.data_ptr(),
                                   bytes, c.stream());
  });
}

PyMethodDef kMethods[] = {
    {"extend_tables", reinterpret_cast<PyCFunction>(guarded<extend_tables>), METH_FASTCALL, nullptr},
    {"release_tables", reinterpret_cast<PyCFunction>(guarded<release_tables>), METH_FASTCALL, nullptr},
    {"rope_and_cache", reinterpret_cast<PyCFunction>(guarded<rope_and_cache>), METH_FASTCALL, nullptr},
    {"decode_shared_prefix", reinterpret_cast<PyCFunction>(guarded<decode_shared_prefix>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
