// Python binding of the paged-cache calls: argument checks, output allocation and marshalling
// for the C ABI (include/attn.h). A decode step makes these calls at intervals of tens of
// microseconds, and the same checks in Python cost more than the kernels' launches: a decode
// call over three short sequences took 19 us of host time through ctypes, 8 us here.
//
// Every function returns its outputs, or the call's attn_status as an int when it is not
// ATTN_OK (the callers raise AttnError); wrong tensors raise ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <initializer_list>

#include "attn.h"

namespace {

struct BadArgument {};  // a Python error is set

[[noreturn]] void fail(const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(PyExc_ValueError, format, args);
  va_end(args);
  throw BadArgument{};
}

const char* name_of(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kByte: return "torch.uint8";
    default: return c10::toString(t);
  }
}

bool none(PyObject* o) { return o == Py_None; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) fail("%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

void check_device(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) fail("%s must be a CUDA tensor", name);
  const int at = t.get_device(), current = c10::cuda::current_device();
  if (at != current) fail("%s is on cuda:%d, the current device is cuda:%d", name, at, current);
}

// A contiguous tensor of this type on the current device.
const at::Tensor& buffer(PyObject* o, at::ScalarType type, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type)
    fail("%s must be %s, got %s", name, name_of(type), name_of(t.scalar_type()));
  check_device(t, name);
  if (!t.is_contiguous()) fail("%s must be contiguous", name);
  return t;
}

void check_shape(const at::Tensor& t, std::initializer_list<int64_t> want, const char* name) {
  if (t.sizes() != c10::IntArrayRef(want)) fail("%s has the wrong shape", name);
}

int number(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw BadArgument{};
  if (v < INT_MIN || v > INT_MAX) fail("%s does not fit 32 bits", name);
  return (int)v;
}
// What int() makes of o: lengths and sizes may come as floats and as numpy or tensor scalars.
long long size_arg(PyObject* o) {
  if (PyLong_CheckExact(o)) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw BadArgument{};
    return v;
  }
  PyObject* i = PyNumber_Long(o);
  if (!i) throw BadArgument{};
  const long long v = PyLong_AsLongLong(i);
  Py_DECREF(i);
  if (v == -1 && PyErr_Occurred()) throw BadArgument{};
  return v;
}
int size_arg(PyObject* o, const char* name) {
  const long long v = size_arg(o);
  if (v < INT_MIN || v > INT_MAX) fail("%s does not fit 32 bits", name);
  return (int)v;
}
// total_kv_tokens, or without one (None or 0) every sequence at its bound.
long long total_tokens(PyObject* o, int B, int max_seq_len) {
  const long long v = none(o) ? 0 : size_arg(o);
  return v > 0 ? v : (long long)B * max_seq_len;
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw BadArgument{};
  return (float)v;
}
int size_of(int64_t n, const char* name) {
  if (n > INT_MAX) fail("%s is too large", name);
  return (int)n;
}

// The stream of a call: the current one, or a torch.cuda.Stream. Tensors for a call on another
// stream are made on that stream: memory freed on the current one may still be in use by work
// queued there, which the call does not wait for. Its outputs are recorded on the current
// stream too, where the caller goes on with them; the workspace goes back to its own.
struct Stream {
  c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream();
  cudaStream_t handle;
  bool foreign = false;
  explicit Stream(PyObject* o) {
    handle = current.stream();
    if (none(o)) return;
    PyObject* value = PyObject_GetAttrString(o, "cuda_stream");
    if (!value) throw BadArgument{};
    handle = static_cast<cudaStream_t>(PyLong_AsVoidPtr(value));
    Py_DECREF(value);
    if (!handle && PyErr_Occurred()) throw BadArgument{};
    foreign = handle != current.stream();
  }
  at::Tensor workspace(const at::Tensor& like, c10::IntArrayRef sizes, at::ScalarType type) const {
    const auto options = like.options().dtype(type).requires_grad(false);
    if (!foreign) return at::empty(sizes, options);
    const c10::cuda::CUDAStreamGuard on(
        c10::cuda::getStreamFromExternal(handle, c10::cuda::current_device()));
    return at::empty(sizes, options);
  }
  at::Tensor output(const at::Tensor& like, c10::IntArrayRef sizes, at::ScalarType type) const {
    at::Tensor t = workspace(like, sizes, type);
    if (foreign && t.numel() > 0) t.record_stream(current.unwrap());
    return t;
  }
};

int num_sms() {
  static int count[64];
  const int dev = c10::cuda::current_device();
  if (dev < 0 || dev >= 64) return 0;
  if (count[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) count[dev] = n;
  }
  return count[dev];
}

// The cache's tensors. kv_exp selects e4m3.
attn_paged_cache cache_of(PyObject* k, PyObject* v, PyObject* table, PyObject* kv_exp) {
  const bool e4m3 = !none(kv_exp);
  const at::ScalarType type = e4m3 ? at::kByte : at::kBFloat16;
  const at::Tensor& kt = buffer(k, type, "k_cache");
  const at::Tensor& vt = buffer(v, type, "v_cache");
  const at::Tensor& tt = buffer(table, at::kInt, "page_table");
  if (kt.dim() != 4 || vt.sizes() != kt.sizes())
    fail("k_cache and v_cache must be [pages, Hkv, page_size, d]");
  if (tt.dim() != 2) fail("page_table must be [B, max_pages]");
  attn_paged_cache c{};
  c.kind = e4m3 ? ATTN_CACHE_E4M3 : ATTN_CACHE_BF16;
  c.k = kt.data_ptr();
  c.v = vt.data_ptr();
  c.page_table = static_cast<const int32_t*>(tt.data_ptr());
  c.num_pages = size_of(kt.size(0), "the pool");
  c.Hkv = size_of(kt.size(1), "Hkv");
  c.page_size = size_of(kt.size(2), "page_size");
  c.d = size_of(kt.size(3), "d");
  c.max_pages_per_seq = size_of(tt.size(1), "page_table");
  if (e4m3) {
    const at::Tensor& et = buffer(kv_exp, at::kByte, "kv_exp");
    check_shape(et, {kt.size(0), kt.size(1), kt.size(2), 2}, "kv_exp");
    c.kv_exp = static_cast<uint8_t*>(et.data_ptr());
  }
  return c;
}

struct Batch {
  int B;
  const int32_t *offsets, *seq_lens;
};
Batch batch_of(PyObject* table, PyObject* offsets, PyObject* seq_lens) {
  const at::Tensor& o = buffer(offsets, at::kInt, "offsets");
  const at::Tensor& s = buffer(seq_lens, at::kInt, "seq_lens");
  if (s.dim() != 1 || o.dim() != 1 || o.size(0) != s.size(0) + 1)
    fail("offsets must be [B + 1] and seq_lens [B]");
  if (THPVariable_Unpack(table).size(0) != s.size(0)) fail("page_table must be [B, max_pages]");
  return Batch{size_of(s.size(0), "B"), static_cast<const int32_t*>(o.data_ptr()),
               static_cast<const int32_t*>(s.data_ptr())};
}

// Packed bf16 rows [T, H, d], d contiguous, any token and head stride.
struct Rows {
  void* p;
  int T, H;
  long long token, head;
};
Rows rows_of(PyObject* o, int H, int d, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kBFloat16)
    fail("%s must be torch.bfloat16, got %s", name, name_of(t.scalar_type()));
  check_device(t, name);
  if (t.dim() != 3 || t.size(2) != d) fail("%s must be [T, heads, %d]", name, d);
  if (H >= 0 && t.size(1) != H) fail("%s must have the cache's %d heads", name, H);
  if (t.stride(2) != 1) fail("%s must be contiguous along d", name);
  return Rows{t.data_ptr(), size_of(t.size(0), name), size_of(t.size(1), name),
              t.size(0) > 1 ? t.stride(0) : 0, t.size(1) > 1 ? t.stride(1) : 0};
}

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
  PyObject* x = THPVariable_Wrap(a);
  PyObject* y = THPVariable_Wrap(b);
  PyObject* r = PyTuple_Pack(2, x, y);
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

struct Scores {
  attn_mask_params mask{};
  attn_score_params score{};
  int mask_kind, score_kind;
  float scale;
  // mask_kind, window, score_kind, softcap
  Scores(PyObject* const* a, PyObject* scale_or_none, int d) {
    mask_kind = number(a[0], "mask_kind");
    mask.window = number(a[1], "window");
    score_kind = number(a[2], "score_kind");
    score.softcap = real(a[3]);
    scale = none(scale_or_none) ? (float)std::pow((double)d, -0.5) : real(scale_or_none);
  }
};

// A caller's workspace, or one made for this call.
struct Workspace {
  at::Tensor own;
  void* p = nullptr;
  size_t bytes = 0;
  Workspace(PyObject* o, bool allocate, const Stream& stream, const at::Tensor& like, size_t need) {
    if (!none(o)) {
      const at::Tensor& t = tensor(o, "workspace");
      check_device(t, "workspace");
      if (!t.is_contiguous()) fail("workspace must be contiguous");
      p = t.data_ptr();
      bytes = t.nbytes();
    } else if (allocate && need > 0) {
      own = stream.workspace(like, {(int64_t)need}, at::kByte);
      p = own.data_ptr();
      bytes = need;
    }
  }
};

#define BINDING(name, count)                                              \
  PyObject* name##_impl(PyObject* const* a);                              \
  PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t n) {           \
    HANDLE_TH_ERRORS                                                      \
    if (n != count) {                                                     \
      PyErr_SetString(PyExc_TypeError, #name " takes " #count " arguments"); \
      return nullptr;                                                     \
    }                                                                     \
    try {                                                                 \
      return name##_impl(a);                                              \
    } catch (const BadArgument&) {                                        \
      return nullptr;                                                     \
    }                                                                     \
    END_HANDLE_TH_ERRORS                                                  \
  }                                                                       \
  PyObject* name##_impl(PyObject* const* a)

PyObject* status(attn_status s) {
  if (s == ATTN_OK) Py_RETURN_NONE;
  return PyLong_FromLong(s);
}

// k, v, k_cache, v_cache, page_table, offsets, seq_lens, kv_exp, stream
BINDING(cache_write, 9) {
  const attn_paged_cache c = cache_of(a[2], a[3], a[4], a[7]);
  const Batch b = batch_of(a[4], a[5], a[6]);
  const Rows k = rows_of(a[0], c.Hkv, c.d, "k"), v = rows_of(a[1], c.Hkv, c.d, "v");
  if (k.T != v.T) fail("k and v disagree on the number of tokens");
  return status(attn_cache_write(&c, k.p, k.token, k.head, v.p, v.token, v.head, b.offsets,
                                 b.seq_lens, b.B, k.T, Stream(a[8]).handle));
}

// k_cache, v_cache, page_table, offsets, seq_lens, kv_exp, stream, k or None, v or None, n_tokens
BINDING(cache_read, 10) {
  const attn_paged_cache c = cache_of(a[0], a[1], a[2], a[5]);
  const Batch b = batch_of(a[2], a[3], a[4]);
  const Stream stream(a[6]);
  if (!none(a[7])) {
    const at::Tensor& k = buffer(a[7], at::kBFloat16, "k");
    const at::Tensor& v = buffer(a[8], at::kBFloat16, "v");
    if (k.dim() != 3 || k.size(1) != c.Hkv || k.size(2) != c.d || v.sizes() != k.sizes())
      fail("k and v must be [T, %d, %d]", c.Hkv, c.d);
    return status(attn_cache_read(&c, k.data_ptr(), v.data_ptr(), b.offsets, b.seq_lens, b.B,
                                  size_of(k.size(0), "k"), stream.handle));
  }
  const int T = size_arg(a[9], "n_tokens");
  if (T < 0) fail("n_tokens must not be negative");
  const at::Tensor& like = THPVariable_Unpack(a[0]);
  const at::Tensor k = stream.output(like, {T, c.Hkv, c.d}, at::kBFloat16);
  const at::Tensor v = stream.output(like, {T, c.Hkv, c.d}, at::kBFloat16);
  const attn_status s =
      attn_cache_read(&c, k.data_ptr(), v.data_ptr(), b.offsets, b.seq_lens, b.B, T, stream.handle);
  return s == ATTN_OK ? pair(k, v) : status(s);
}

// q, k_cache, v_cache, page_table, offsets, seq_lens, kv_exp, stream, o or None, lse or None,
// workspace or None, max_new, max_seq_len, split_keys, total_kv_tokens, scale (each None for
// the library's choice), mask_kind, window, score_kind, softcap
BINDING(prefill, 20) {
  const attn_paged_cache c = cache_of(a[1], a[2], a[3], a[6]);
  const Batch b = batch_of(a[3], a[4], a[5]);
  const Rows q = rows_of(a[0], -1, c.d, "q");
  const Scores sc(a + 16, a[15], c.d);
  const long long capacity = (long long)c.max_pages_per_seq * c.page_size;
  const int max_seq_len = none(a[12]) ? size_of(capacity, "the page table") : size_arg(a[12], "max_seq_len");
  const int max_new = none(a[11]) ? q.T : size_arg(a[11], "max_new");
  const long long total = total_tokens(a[14], b.B, max_seq_len);
  const int split = none(a[13]) ? attn_prefill_split_keys(c.kind, b.B, q.T, q.H, c.Hkv, max_new,
                                                          max_seq_len, total, num_sms())
                                : size_arg(a[13], "split_keys");
  const at::Tensor& like = THPVariable_Unpack(a[0]);
  const Stream stream(a[7]);
  const bool allocate = none(a[8]);
  at::Tensor o, lse;
  if (allocate) {
    o = stream.output(like, {q.T, q.H, c.d}, at::kBFloat16);
    lse = stream.output(like, {q.T, q.H}, at::kFloat);
  } else {
    o = buffer(a[8], at::kBFloat16, "o");
    lse = buffer(a[9], at::kFloat, "lse");
    check_shape(o, {q.T, q.H, c.d}, "o");
    check_shape(lse, {q.T, q.H}, "lse");
  }
  const Workspace ws(a[10], allocate, stream, like,
                     attn_prefill_workspace_size(q.T, q.H, c.d, max_seq_len, split));
  const attn_status s = attn_prefill_paged(
      &c, q.p, q.token, q.head, o.data_ptr(), static_cast<float*>(lse.data_ptr()), b.offsets, b.seq_lens,
      b.B, q.T, q.H, max_new, max_seq_len, split, sc.scale, sc.mask_kind, &sc.mask, sc.score_kind,
      &sc.score, ws.p, ws.bytes, stream.handle);
  if (s != ATTN_OK) return status(s);
  if (!allocate) Py_RETURN_NONE;
  return pair(o, lse);
}

// q, k_cache, v_cache, page_table, seq_lens, kv_exp, stream, o or None, lse or None, workspace
// or None, max_seq_len, split_keys, total_kv_tokens, scale (each None for the library's
// choice), mask_kind, window, score_kind, softcap
BINDING(decode, 18) {
  const attn_paged_cache c = cache_of(a[1], a[2], a[3], a[5]);
  const bool e4m3 = c.kind == ATTN_CACHE_E4M3;
  const at::Tensor& q = buffer(a[0], at::kBFloat16, "q");
  const at::Tensor& lens = buffer(a[4], at::kInt, "seq_lens");
  if (q.dim() != 4 || q.size(3) != c.d) fail("q must be [B, Hq, Nq, %d]", c.d);
  const int B = size_of(q.size(0), "B"), Hq = size_of(q.size(1), "Hq"), Nq = size_of(q.size(2), "Nq");
  check_shape(lens, {q.size(0)}, "seq_lens");
  if (THPVariable_Unpack(a[3]).size(0) != q.size(0)) fail("page_table must be [B, max_pages]");
  const Scores sc(a + 14, a[13], c.d);
  const long long capacity = (long long)c.max_pages_per_seq * c.page_size;
  const int max_seq_len = none(a[10]) ? size_of(capacity, "the page table") : size_arg(a[10], "max_seq_len");
  const long long total = total_tokens(a[12], B, max_seq_len);
  const int rows = size_of((int64_t)B * Nq, "B * Nq");
  const int split = !none(a[11]) ? size_arg(a[11], "split_keys")
                    : e4m3 ? attn_prefill_split_keys(c.kind, B, rows, Hq, c.Hkv, Nq, max_seq_len,
                                                     total, num_sms())
                           : attn_decode_split_keys(B, Hq, c.Hkv, Nq, total, num_sms());
  const Stream stream(a[6]);
  const bool allocate = none(a[7]);
  at::Tensor o, lse;
  if (allocate) {
    o = stream.output(q, q.sizes(), at::kBFloat16);
    lse = stream.output(q, {B, Hq, Nq}, at::kFloat);
  } else {
    o = buffer(a[7], at::kBFloat16, "o");
    lse = buffer(a[8], at::kFloat, "lse");
    check_shape(o, {B, Hq, Nq, c.d}, "o");
    check_shape(lse, {B, Hq, Nq}, "lse");
  }
  const Workspace ws(a[9], allocate, stream, q,
                     e4m3 ? attn_prefill_workspace_size(rows, Hq, c.d, max_seq_len, split)
                          : attn_decode_workspace_size(B, Hq, c.Hkv, Nq, c.d, max_seq_len, split));
  const int32_t* seq_lens = static_cast<const int32_t*>(lens.data_ptr());
  float* l = static_cast<float*>(lse.data_ptr());
  const attn_status s =
      e4m3 ? attn_decode_paged_e4m3(&c, q.data_ptr(), seq_lens, o.data_ptr(), l, B, Hq, Nq, max_seq_len,
                                    split, sc.scale, sc.mask_kind, &sc.mask, sc.score_kind, &sc.score,
                                    ws.p, ws.bytes, stream.handle)
           : attn_decode_paged(q.data_ptr(), c.k, c.v, c.page_table, seq_lens, o.data_ptr(), l, B, Hq,
                               c.Hkv, Nq, c.d, c.num_pages, c.page_size, c.max_pages_per_seq,
                               max_seq_len, split, sc.scale, sc.mask_kind, &sc.mask, sc.score_kind,
                               &sc.score, ws.p, ws.bytes, stream.handle);
  if (s != ATTN_OK) return status(s);
  if (!allocate) Py_RETURN_NONE;
  return pair(o, lse);
}

PyMethodDef kMethods[] = {
    {"cache_write", (PyCFunction)(void (*)())cache_write, METH_FASTCALL, nullptr},
    {"cache_read", (PyCFunction)(void (*)())cache_read, METH_FASTCALL, nullptr},
    {"prefill", (PyCFunction)(void (*)())prefill, METH_FASTCALL, nullptr},
    {"decode", (PyCFunction)(void (*)())decode, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", "Binding of the paged-cache calls.", -1,
                       kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
