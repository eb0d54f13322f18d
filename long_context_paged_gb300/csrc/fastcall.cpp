// The binding's fast path: the calls that a serving step makes, marshalled in one C++ function each.
//
// A small call's time is its host time: checking a dozen tensors through Python attributes and
// converting two dozen arguments through ctypes takes up to 15 us, the launch 2-3 us, the kernel often
// less. Measured, one call after another, through ctypes and through this file: decode of one sequence
// of 1,000 keys 18.9 and 4.7 us, 375 prefill rows 21.1 and 14.4 (14.3 of it the kernel's), 31 rotary rows
// 12.7 and 3.0, a plan for 32 requests 10.8 and 5.4 (5.3 of it the kernel's), a release of 512 requests'
// pages with a copy of the table 15.9 and 10.3.
//
// These functions take the same arguments as the Python wrappers, make the same checks on the tensors
// themselves, and call the C ABI. They decide nothing else: whatever is not plainly right (a wrong
// type, shape, device or layout, an argument of another kind, a refusal of the C ABI) returns False,
// and the wrapper's own path then makes the call or names the error; the C ABI refuses before its first
// launch, so nothing runs twice. A CUDA error may come from a later launch of the call: it is raised
// from here. No computation happens here, and the binding works without this module, only slower.
#include <Python.h>

#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "pagedattn.h"

namespace {

using at::ScalarType;

// The arguments of one call, read in order; `good` turns false at the first that does not fit.
struct Reader {
  PyObject* const* a;
  Py_ssize_t n, i = 0;
  int dev;
  bool good = true;

  Reader(PyObject* const* args, Py_ssize_t count) : a(args), n(count), dev(c10::cuda::current_device()) {}

  PyObject* next() {
    if (i >= n) {
      good = false;
      return Py_None;
    }
    return a[i++];
  }
  const at::Tensor* tensor_of(PyObject* o, ScalarType type) {
    if (good && THPVariable_Check(o)) {
      const at::Tensor& t = THPVariable_Unpack(o);
      if (t.defined() && t.is_cuda() && t.get_device() == dev && t.scalar_type() == type) return &t;
    }
    good = false;
    return nullptr;
  }
  // A contiguous tensor of this type and number of dims on the current device.
  const at::Tensor* tensor(ScalarType type, int dims) {
    const at::Tensor* t = tensor_of(next(), type);
    if (good && (t->dim() != dims || !t->is_contiguous())) good = false;
    return good ? t : nullptr;
  }
  const at::Tensor* tensor_or_none(ScalarType type, int dims) {
    if (i < n && a[i] == Py_None) {
      ++i;
      return nullptr;
    }
    return tensor(type, dims);
  }
  // A status word: any contiguous int32 tensor, or None.
  void* status() {
    PyObject* o = next();
    if (o == Py_None) return nullptr;
    const at::Tensor* t = tensor_of(o, ScalarType::Int);
    if (good && !t->is_contiguous()) good = false;
    return good ? t->data_ptr() : nullptr;
  }
  // A workspace: bytes on the device, or None.
  const at::Tensor* bytes_or_none() {
    if (i < n && a[i] == Py_None) {
      ++i;
      return nullptr;
    }
    return tensor(ScalarType::Byte, 1);
  }
  long long integer() {
    PyObject* o = next();
    if (!PyLong_Check(o)) {
      good = false;
      return 0;
    }
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      good = false;
    }
    return v;
  }
  int32_t int32() {
    const long long v = integer();
    if (v < INT32_MIN || v > INT32_MAX) good = false;
    return static_cast<int32_t>(v);
  }
  double number() {
    PyObject* o = next();
    if (!PyFloat_Check(o) && !PyLong_Check(o)) {
      good = false;
      return 0.0;
    }
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      good = false;
    }
    return v;
  }
  // None: the current stream; else its handle.
  cudaStream_t stream() {
    PyObject* o = next();
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    --i;
    return reinterpret_cast<cudaStream_t>(integer());
  }
  // None: the decoder's shape; else a tuple of four ints that the library supports.
  pa_dims dims() {
    pa_dims d{16, 8, 128, 16};
    PyObject* o = next();
    if (o == Py_None) return d;
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) {
      good = false;
      return d;
    }
    int32_t v[4];
    for (int k = 0; k < 4; ++k) {
      PyObject* x = PyTuple_GET_ITEM(o, k);
      const long n = PyLong_Check(x) ? PyLong_AsLong(x) : -1;
      if (n < 0 || n > 4096) {
        PyErr_Clear();
        good = false;
        return d;
      }
      v[k] = static_cast<int32_t>(n);
    }
    d = pa_dims{v[0], v[1], v[2], v[3]};
    const int h = d.num_kv_heads;
    if (!(h == 1 || h == 2 || h == 4 || h == 8) || d.num_q_heads != 2 * h || d.head_dim != 128 || d.page_size != 16)
      good = false;
    return d;
  }
  void shape(const at::Tensor* t, int64_t d0) { if (good && t && t->size(0) != d0) good = false; }
  void shape(const at::Tensor* t, int64_t d0, int64_t d1) {
    if (good && t && (t->size(0) != d0 || t->size(1) != d1)) good = false;
  }
  void shape(const at::Tensor* t, int64_t d0, int64_t d1, int64_t d2) {
    if (good && t && (t->size(0) != d0 || t->size(1) != d1 || t->size(2) != d2)) good = false;
  }
  void shape(const at::Tensor* t, int64_t d0, int64_t d1, int64_t d2, int64_t d3) {
    if (good && t && (t->size(0) != d0 || t->size(1) != d1 || t->size(2) != d2 || t->size(3) != d3)) good = false;
  }
  void at_least(const at::Tensor* t, int64_t rows) { if (good && t && t->size(0) < rows) good = false; }
  void require(bool b) { good = good && b; }
  bool done() { return good && i == n; }
};

template <class T = void>
T* ptr(const at::Tensor* t) { return t == nullptr ? nullptr : static_cast<T*>(t->data_ptr()); }

// The library's calls run without the interpreter's lock: a launch waits while the device's queue is
// full, and what it waits for may need the lock (a host callback).
struct Unlocked {
  PyThreadState* state;
  Unlocked() : state(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state); }
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;
};

// A call's workspace: the caller's, or memory of the stream for the length of the call, given back as
// soon as the call is launched, to be handed out again only to later work of the same stream.
struct Scratch {
  void* p = nullptr;
  size_t bytes = 0;
  bool own = false;
  Scratch(const at::Tensor* given, size_t need, cudaStream_t st) {
    if (given != nullptr) {
      p = given->data_ptr();
      bytes = given->nbytes();
      return;
    }
    bytes = need < 256 ? 256 : need;
    p = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(bytes, st);
    own = true;
  }
  ~Scratch() { if (own) c10::cuda::CUDACachingAllocator::raw_delete(p); }
  Scratch(const Scratch&) = delete;
  Scratch& operator=(const Scratch&) = delete;
};

// The score options, in the order softcap, alibi_slopes, window, prefix_lens, max_prefix_len (None:
// max_seq_len), row_start. Returns whether any is set.
bool score_options(Reader& r, pa_score_opts& s, int hq, int64_t batch, int64_t rows, int32_t max_seq_len) {
  s.softcap = static_cast<float>(r.number());
  const at::Tensor* slopes = r.tensor_or_none(ScalarType::Float, 1);
  s.window = r.int32();
  const at::Tensor* prefix = r.tensor_or_none(ScalarType::Int, 1);
  if (r.i < r.n && r.a[r.i] == Py_None) {
    ++r.i;
    s.max_prefix_len = max_seq_len;
  } else {
    s.max_prefix_len = r.int32();
  }
  const at::Tensor* start = r.tensor_or_none(ScalarType::Int, 1);
  r.shape(slopes, hq);
  r.at_least(prefix, batch);
  r.at_least(start, rows);
  if (prefix == nullptr) s.max_prefix_len = 0;
  s.alibi_slopes = ptr<const float>(slopes);
  s.prefix_lens = ptr<const int32_t>(prefix);
  s.row_start = ptr<const int32_t>(start);
  return s.softcap != 0.f || slopes != nullptr || s.window != 0 || prefix != nullptr || start != nullptr;
}

// max_ctas: None or an int >= 0.
const pa_launch_opts* launch_options(Reader& r, pa_launch_opts& o) {
  PyObject* x = r.next();
  if (x == Py_None) return nullptr;
  --r.i;
  o.max_ctas = r.int32();
  r.require(o.max_ctas >= 0);
  return &o;
}

// The binding's error class, called with a call's name and its status code (set_error).
PyObject* error_class = nullptr;

// What became of a call: not made, or made under this name with this status code.
struct Made {
  const char* name = nullptr;
  pa_status code = PA_OK;
};

// f(): makes the call or not. What it throws comes from before the call (a machine without a GPU, a
// tensor without strides or storage, the allocator): the wrapper meets it again and raises its error.
template <class F>
PyObject* guarded(F f) {
  Made made;
  try {
    made = f();
  } catch (const std::exception&) {
    PyErr_Clear();
  }
  if (made.name != nullptr && made.code == PA_ERR_CUDA && error_class != nullptr) {
    PyObject* e = PyObject_CallFunction(error_class, "si", made.name, static_cast<int>(made.code));
    if (e != nullptr) {
      PyErr_SetObject(error_class, e);
      Py_DECREF(e);
    }
    return nullptr;
  }
  return PyBool_FromLong(made.name != nullptr && made.code == PA_OK);
}

// (q, k_pool, v_pool, block_table, seq_lens, max_seq_len, scale, split_tokens, out, lse,
//  workspace, status, stream, dims, max_ctas, options)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> Made {
    Reader r(a, n);
    const at::Tensor* q = r.tensor(ScalarType::BFloat16, 3);
    const at::Tensor* k = r.tensor(ScalarType::BFloat16, 4);
    const at::Tensor* v = r.tensor(ScalarType::BFloat16, 4);
    const at::Tensor* table = r.tensor(ScalarType::Int, 2);
    const at::Tensor* lens = r.tensor(ScalarType::Int, 1);
    const int32_t max_len = r.int32();
    const float scale = static_cast<float>(r.number());
    const int32_t split = r.int32();
    const at::Tensor* out = r.tensor(ScalarType::BFloat16, 3);
    const at::Tensor* lse = r.tensor_or_none(ScalarType::Float, 2);
    const at::Tensor* workspace = r.bytes_or_none();
    void* status = r.status();
    cudaStream_t st = r.stream();
    const pa_dims d = r.dims();
    pa_launch_opts lo{};
    const pa_launch_opts* opts = launch_options(r, lo);
    if (!r.good) return {};
    const int64_t B = q->size(0), hq = d.num_q_heads, hkv = d.num_kv_heads;
    pa_score_opts so{};
    const bool scored = score_options(r, so, static_cast<int>(hq), B, B, max_len);
    r.shape(q, B, hq, 128);
    r.shape(k, k->size(0), 16, hkv, 128);
    r.shape(v, k->size(0), 16, hkv, 128);
    r.at_least(table, B);
    r.at_least(lens, B);
    r.shape(out, B, hq, 128);
    r.shape(lse, B, hq);
    if (!r.done() || B > INT32_MAX || table->size(1) > INT32_MAX) return {};
    const int32_t batch = static_cast<int32_t>(B), stride = static_cast<int32_t>(table->size(1));
    const size_t need = workspace ? 0 : pa_decode_workspace_size(d, batch, max_len, split);
    Unlocked unlocked;
    Scratch scratch(workspace, need, st);
    pa_stream_t s = reinterpret_cast<pa_stream_t>(st);
    pa_status code;
    if (scored)
      code = attn_decode_paged_score(d, q->data_ptr(), k->data_ptr(), v->data_ptr(), k->size(0),
                                     ptr<const int32_t>(table), stride, ptr<const int32_t>(lens), batch, max_len,
                                     scale, split, out->data_ptr(), ptr<float>(lse), scratch.p, scratch.bytes,
                                     static_cast<int32_t*>(status), s, opts, &so);
    else
      code = attn_decode_paged_ex(d, q->data_ptr(), k->data_ptr(), v->data_ptr(), k->size(0),
                                  ptr<const int32_t>(table), stride, ptr<const int32_t>(lens), batch, max_len, scale,
                                  split, out->data_ptr(), ptr<float>(lse), scratch.p, scratch.bytes,
                                  static_cast<int32_t*>(status), s, opts);
    return {scored ? "attn_decode_paged_score" : "attn_decode_paged", code};
  });
}

// (q, cu_q_lens, k_pool, v_pool, block_table, seq_lens, max_q_len, max_seq_len, scale, out, lse,
//  workspace, status, stream, dims, max_ctas, options)
PyObject* prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> Made {
    Reader r(a, n);
    const at::Tensor* q = r.tensor(ScalarType::BFloat16, 3);
    const at::Tensor* cu = r.tensor(ScalarType::Int, 1);
    const at::Tensor* k = r.tensor(ScalarType::BFloat16, 4);
    const at::Tensor* v = r.tensor(ScalarType::BFloat16, 4);
    const at::Tensor* table = r.tensor(ScalarType::Int, 2);
    const at::Tensor* lens = r.tensor(ScalarType::Int, 1);
    const int32_t max_q = r.int32(), max_len = r.int32();
    const float scale = static_cast<float>(r.number());
    const at::Tensor* out = r.tensor(ScalarType::BFloat16, 3);
    const at::Tensor* lse = r.tensor_or_none(ScalarType::Float, 2);
    const at::Tensor* workspace = r.bytes_or_none();
    void* status = r.status();
    cudaStream_t st = r.stream();
    const pa_dims d = r.dims();
    pa_launch_opts lo{};
    const pa_launch_opts* opts = launch_options(r, lo);
    if (!r.good) return {};
    const int64_t B = lens->size(0), T = q->size(0), hq = d.num_q_heads, hkv = d.num_kv_heads;
    pa_score_opts so{};
    const bool scored = score_options(r, so, static_cast<int>(hq), B, T, max_len);
    r.shape(q, T, hq, 128);
    r.at_least(cu, B + 1);
    r.shape(k, k->size(0), 16, hkv, 128);
    r.shape(v, k->size(0), 16, hkv, 128);
    r.at_least(table, B);
    r.shape(out, T, hq, 128);
    r.shape(lse, T, hq);
    if (!r.done() || B > INT32_MAX || T > INT32_MAX || table->size(1) > INT32_MAX) return {};
    const int32_t batch = static_cast<int32_t>(B), rows = static_cast<int32_t>(T);
    const int32_t stride = static_cast<int32_t>(table->size(1));
    const size_t need = workspace ? 0
                        : scored  ? pa_prefill_score_workspace_size(d, batch, rows)
                                  : pa_prefill_workspace_size(d, batch, max_q, max_len);
    Unlocked unlocked;
    Scratch scratch(workspace, need, st);
    pa_stream_t s = reinterpret_cast<pa_stream_t>(st);
    pa_status code;
    if (scored)
      code = attn_prefill_chunk_score(d, q->data_ptr(), ptr<const int32_t>(cu), rows, k->data_ptr(), v->data_ptr(),
                                      k->size(0), ptr<const int32_t>(table), stride, ptr<const int32_t>(lens), batch,
                                      max_q, max_len, scale, out->data_ptr(), ptr<float>(lse), scratch.p,
                                      scratch.bytes, static_cast<int32_t*>(status), s, opts, &so);
    else
      code = attn_prefill_chunk_ex(d, q->data_ptr(), ptr<const int32_t>(cu), rows, k->data_ptr(), v->data_ptr(),
                                   k->size(0), ptr<const int32_t>(table), stride, ptr<const int32_t>(lens), batch,
                                   max_q, max_len, scale, out->data_ptr(), ptr<float>(lse), scratch.p, scratch.bytes,
                                   static_cast<int32_t*>(status), s, opts);
    return {scored ? "attn_prefill_chunk_score" : "attn_prefill_chunk", code};
  });
}

// A [T, heads, 128] bf16 tensor whose rows may lie apart: its stride between rows.
int64_t row_stride(Reader& r, const at::Tensor* t, int64_t T, int64_t heads) {
  r.require(t != nullptr && t->dim() == 3);
  r.shape(t, T, heads, 128);
  if (!r.good) return 0;
  r.require(t->stride(2) == 1 && (t->stride(1) == 128 || heads == 1));
  return T > 1 ? t->stride(0) : heads * 128;
}

// (q, k_new, v_new, positions, slot_map, k_pool, v_pool, inv_freq, interleaved, attn_factor, q_gamma,
//  k_gamma, eps, q_out, status, stream, dims)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> Made {
    Reader r(a, n);
    const at::Tensor* q = r.tensor_of(r.next(), ScalarType::BFloat16);
    const at::Tensor* k = r.tensor_of(r.next(), ScalarType::BFloat16);
    const at::Tensor* v = r.tensor_of(r.next(), ScalarType::BFloat16);
    const at::Tensor* pos = r.tensor(ScalarType::Int, 1);
    const at::Tensor* slots = r.tensor(ScalarType::Long, 1);
    const at::Tensor* kp = r.tensor(ScalarType::BFloat16, 4);
    const at::Tensor* vp = r.tensor(ScalarType::BFloat16, 4);
    const at::Tensor* freq = r.tensor(ScalarType::Double, 1);
    const int32_t interleaved = r.int32();
    const float factor = static_cast<float>(r.number());
    const at::Tensor* qg = r.tensor_or_none(ScalarType::Float, 1);
    const at::Tensor* kg = r.tensor_or_none(ScalarType::Float, 1);
    const float eps = static_cast<float>(r.number());
    const at::Tensor* out = r.tensor(ScalarType::BFloat16, 3);
    void* status = r.status();
    cudaStream_t st = r.stream();
    const pa_dims d = r.dims();
    if (!r.done() || q->dim() != 3) return {};
    const int64_t T = q->size(0), hq = d.num_q_heads, hkv = d.num_kv_heads;
    const int64_t qs = row_stride(r, q, T, hq), ks = row_stride(r, k, T, hkv), vs = row_stride(r, v, T, hkv);
    r.shape(pos, T);
    r.shape(slots, T);
    r.shape(kp, kp->size(0), 16, hkv, 128);
    r.shape(vp, kp->size(0), 16, hkv, 128);
    r.shape(qg, 128);
    r.shape(kg, 128);
    r.shape(out, T, hq, 128);
    if (!r.good || T > INT32_MAX || freq->size(0) > 128) return {};
    Unlocked unlocked;
    const pa_status code = rope_append_paged(d, 2 * static_cast<int32_t>(freq->size(0)), interleaved,
                                             ptr<const double>(freq), factor, q->data_ptr(), qs, k->data_ptr(), ks,
                                             v->data_ptr(), vs, static_cast<int32_t>(T), ptr<const int32_t>(pos),
                                             ptr<const int64_t>(slots), ptr<const float>(qg), ptr<const float>(kg),
                                             eps, out->data_ptr(), kp->data_ptr(), vp->data_ptr(), kp->size(0),
                                             static_cast<int32_t*>(status), reinterpret_cast<pa_stream_t>(st));
    return {"rope_append_paged", code};
  });
}

// (cached_lens, new_lens, block_table, free_pages, free_count, num_pages, total_rows, free_count_out,
//  cu_new_lens, seq_lens, positions, slot_map, status, stream)
PyObject* step_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> Made {
    Reader r(a, n);
    const at::Tensor* cached = r.tensor(ScalarType::Int, 1);
    const at::Tensor* fresh = r.tensor(ScalarType::Int, 1);
    const at::Tensor* table = r.tensor(ScalarType::Int, 2);
    const at::Tensor* free = r.tensor(ScalarType::Int, 1);
    const at::Tensor* count = r.tensor(ScalarType::Int, 1);
    const long long pages = r.integer();
    const int32_t rows = r.int32();
    const at::Tensor* count_out = r.tensor(ScalarType::Int, 1);
    const at::Tensor* cu = r.tensor(ScalarType::Int, 1);
    const at::Tensor* lens = r.tensor(ScalarType::Int, 1);
    const at::Tensor* pos = r.tensor(ScalarType::Int, 1);
    const at::Tensor* slots = r.tensor(ScalarType::Long, 1);
    void* status = r.status();
    cudaStream_t st = r.stream();
    if (!r.done()) return {};
    const int64_t B = cached->size(0);
    r.require(rows >= 0 && B <= INT32_MAX && table->size(1) <= INT32_MAX && free->size(0) <= INT32_MAX);
    r.shape(fresh, B);
    r.at_least(table, B);
    r.at_least(count, 1);
    r.shape(count_out, 1);
    r.shape(cu, B + 1);
    r.shape(lens, B);
    r.shape(pos, rows);
    r.shape(slots, rows);
    if (!r.good) return {};
    Unlocked unlocked;
    const pa_status code = paged_step_plan(ptr<const int32_t>(cached), ptr<const int32_t>(fresh),
                                           static_cast<int32_t>(B), ptr<int32_t>(table),
                                           static_cast<int32_t>(table->size(1)), ptr<const int32_t>(free),
                                           static_cast<int32_t>(free->size(0)), ptr<const int32_t>(count), pages,
                                           rows, ptr<int32_t>(count_out), ptr<int32_t>(cu), ptr<int32_t>(lens),
                                           ptr<int32_t>(pos), ptr<int64_t>(slots), static_cast<int32_t*>(status),
                                           reinterpret_cast<pa_stream_t>(st));
    return {"paged_step_plan", code};
  });
}

// (begin_pages, end_pages, block_table, free_pages, free_count, num_pages, free_count_out, status,
//  stream)
PyObject* release(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> Made {
    Reader r(a, n);
    const at::Tensor* begin = r.tensor(ScalarType::Int, 1);
    const at::Tensor* end = r.tensor(ScalarType::Int, 1);
    const at::Tensor* table = r.tensor(ScalarType::Int, 2);
    const at::Tensor* free = r.tensor(ScalarType::Int, 1);
    const at::Tensor* count = r.tensor(ScalarType::Int, 1);
    const long long pages = r.integer();
    const at::Tensor* count_out = r.tensor(ScalarType::Int, 1);
    void* status = r.status();
    cudaStream_t st = r.stream();
    if (!r.done()) return {};
    const int64_t B = begin->size(0);
    r.require(B <= INT32_MAX && table->size(1) <= INT32_MAX && free->size(0) <= INT32_MAX);
    r.shape(end, B);
    r.at_least(table, B);
    r.at_least(count, 1);
    r.shape(count_out, 1);
    if (!r.good) return {};
    Unlocked unlocked;
    const pa_status code = paged_release(ptr<const int32_t>(begin), ptr<const int32_t>(end), static_cast<int32_t>(B),
                                         ptr<int32_t>(table), static_cast<int32_t>(table->size(1)),
                                         ptr<int32_t>(free), static_cast<int32_t>(free->size(0)),
                                         ptr<const int32_t>(count), pages, ptr<int32_t>(count_out),
                                         static_cast<int32_t*>(status), reinterpret_cast<pa_stream_t>(st));
    return {"paged_release", code};
  });
}

PyObject* set_error(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 1 || !PyType_Check(a[0])) {
    PyErr_SetString(PyExc_TypeError, "set_error takes a class");
    return nullptr;
  }
  Py_INCREF(a[0]);
  Py_XDECREF(error_class);
  error_class = a[0];
  Py_RETURN_NONE;
}

#define PA_METHOD(name, doc) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, doc}
PyMethodDef methods[] = {
    PA_METHOD(decode, "attn_decode_paged"),      PA_METHOD(prefill, "attn_prefill_chunk"),
    PA_METHOD(rope, "rope_append_paged"),        PA_METHOD(step_plan, "paged_step_plan"),
    PA_METHOD(release, "paged_release"),         PA_METHOD(set_error, "class of the errors raised"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pa_call", "Fast path of the binding", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pa_call() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
