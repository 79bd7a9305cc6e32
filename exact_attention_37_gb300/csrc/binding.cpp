// Native marshalling of the calls that matter at a few microseconds: it checks torch
// tensors, allocates the outputs and the workspace, and passes pointers, sizes and the
// current stream to the C ABI.  No step of the computation is here.  The C functions are
// those of the library that the ctypes binding has loaded; their addresses come from it
// (bind), so there is one library and one set of device records in a process.
//
// A function returns its outputs, or an int: the fa_status that the C call gave, which the
// caller turns into an exception.  Wrong arguments raise ValueError or TypeError.
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "../../include/fa_attention.h"

namespace {

decltype(&fa_fwd_rule_workspace_size) p_fwd_ws;
decltype(&fa_bwd_rule_workspace_size) p_bwd_ws;
decltype(&fa_fwd_rule) p_fwd;
decltype(&fa_bwd_rule) p_bwd;
decltype(&fa_kv4_append) p_append;
decltype(&fa_kv4_read) p_read;
decltype(&fa_kv4_attend_workspace_size) p_attend_ws;
decltype(&fa_kv4_attend) p_attend;
decltype(&fa_kv4_attend_tree_workspace_size) p_tree_ws;
decltype(&fa_kv4_attend_tree) p_tree;
decltype(&fa_kv4_keep) p_keep;
decltype(&fa_kv4_plan) p_plan;
decltype(&fa_rotary) p_rotary;

struct BadArgument {
  PyObject* type;
  const char* text;
};
[[noreturn]] void bad(const char* text) { throw BadArgument{PyExc_ValueError, text}; }

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) throw BadArgument{PyExc_TypeError, what};
  return THPVariable_Unpack(o);
}
// A contiguous CUDA tensor of a type on device `dev`; `what` names the rule that it broke.
void check(const at::Tensor& t, at::ScalarType type, int64_t dev, const char* what) {
  if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || !t.is_contiguous()) bad(what);
}
void check_sizes(const at::Tensor& t, at::IntArrayRef sizes, const char* what) {
  if (t.sizes() != sizes) bad(what);
}
fa_dtype dtype_of(const at::Tensor& t) {
  if (t.scalar_type() == at::kHalf) return FA_FP16;
  if (t.scalar_type() == at::kBFloat16) return FA_BF16;
  throw BadArgument{PyExc_TypeError, "unsupported dtype: fp16 or bf16 only"};
}
int to_int(int64_t x) {
  if (x < 0 || x > INT32_MAX) bad("a size is outside 32 bits");
  return (int)x;
}
double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw BadArgument{nullptr, nullptr};
  return x;
}
bool truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw BadArgument{nullptr, nullptr};
  return x != 0;
}
const int32_t* ints(PyObject* o, at::IntArrayRef sizes, int64_t dev, const char* what) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, what);
  check(t, at::kInt, dev, what);
  check_sizes(t, sizes, what);
  return t.const_data_ptr<int32_t>();
}
const float* slopes_of(PyObject* o, int64_t H, int64_t dev) {
  if (o == Py_None) return nullptr;
  const char* what = "slopes must be a contiguous float32 tensor [H] on the inputs' device";
  const at::Tensor& t = tensor(o, what);
  check(t, at::kFloat, dev, what);
  check_sizes(t, {H}, what);
  return t.const_data_ptr<float>();
}
fa_stream_t stream_of(int64_t dev) {
  return reinterpret_cast<fa_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
}
at::Tensor bytes(size_t n, const at::Tensor& like) { return at::empty({(int64_t)n}, like.options().dtype(at::kByte)); }

PyObject* status(fa_status s) { return PyLong_FromLong((long)s); }
PyObject* pack(std::initializer_list<at::Tensor> ts) {
  PyObject* out = PyTuple_New((Py_ssize_t)ts.size());
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = THPVariable_Wrap(t);
    if (!o) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}

// Runs f with torch's and this file's exceptions turned into Python's, and no device or
// allocation left behind by one.
template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const BadArgument& e) {
    if (e.type) PyErr_SetString(e.type, e.text);
    return nullptr;
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

struct Problem {
  int B, H, Hkv, Nq, Nk, d;
  int64_t dev;
  fa_dtype dtype;
  Problem(const at::Tensor& q, const at::Tensor& k, const at::Tensor& v) {
    if (q.dim() != 4 || k.dim() != 4) bad("expected [B, H, N, d] tensors");
    dtype = dtype_of(q);
    if (!q.is_cuda()) bad("tensors must be on a CUDA device");
    dev = q.get_device();
    const char* what = "q, k and v must be contiguous, of one type and on one device";
    check(q, q.scalar_type(), dev, what);
    check(k, q.scalar_type(), dev, what);
    check(v, q.scalar_type(), dev, what);
    if (v.sizes() != k.sizes() || k.size(0) != q.size(0) || k.size(3) != q.size(3))
      bad("k and v must be [B, H_kv, N_k, d] with q's B and d");
    if (k.size(1) < 1 || q.size(1) % k.size(1)) bad("the key/value head count must divide the query head count");
    B = to_int(q.size(0)), H = to_int(q.size(1)), Hkv = to_int(k.size(1));
    Nq = to_int(q.size(2)), Nk = to_int(k.size(2)), d = to_int(q.size(3));
  }
};

// A rule from (causal, cap, slopes, q_doc, k_doc, prefix).
fa_score_rule rule_of(PyObject* const* a, const Problem& p) {
  fa_score_rule r{};
  r.causal = truth(a[0]);
  r.cap = (float)number(a[1]);
  r.slopes = slopes_of(a[2], p.H, p.dev);
  if ((a[3] == Py_None) != (a[4] == Py_None)) bad("q_doc and k_doc go together");
  r.q_doc = ints(a[3], {p.B, p.Nq}, p.dev, "q_doc must be a contiguous int32 tensor [B, N_q] on the inputs' device");
  r.k_doc = ints(a[4], {p.B, p.Nk}, p.dev, "k_doc must be a contiguous int32 tensor [B, N_k] on the inputs' device");
  r.prefix = ints(a[5], {p.B}, p.dev, "prefix must be a contiguous int32 tensor [B] on the inputs' device");
  return r;
}
float scale_of(PyObject* o, int d) { return (float)(o == Py_None ? 1.0 / std::sqrt((double)d) : number(o)); }

// (q, k, v, causal, cap, slopes, q_doc, k_doc, prefix, scale) -> (o, lse)
PyObject* forward_rule(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q must be a tensor"), &k = tensor(a[1], "k must be a tensor"),
                     &v = tensor(a[2], "v must be a tensor");
    const Problem p(q, k, v);
    const fa_score_rule r = rule_of(a + 3, p);
    const float scale = scale_of(a[9], p.d);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.dev);
    const at::Tensor o = at::empty_like(q);
    const at::Tensor lse = at::empty({p.B, p.H, p.Nq}, q.options().dtype(at::kFloat));
    at::Tensor ws;
    size_t size = 0;
    if (r.q_doc) {
      size = p_fwd_ws(p.B, p.H, p.Nq, p.Nk, p.d, 1);
      ws = bytes(size, q);
    }
    const fa_status s = p_fwd(q.const_data_ptr(), k.const_data_ptr(), v.const_data_ptr(), o.mutable_data_ptr(),
                              static_cast<float*>(lse.mutable_data_ptr()), &r, size ? ws.mutable_data_ptr() : nullptr, size,
                              p.B, p.H, p.Hkv, p.Nq, p.Nk, p.d, scale, p.dtype, stream_of(p.dev));
    return s == FA_OK ? pack({o, lse}) : status(s);
  });
}

// (q, k, v, o, lse, dout, causal, cap, slopes, q_doc, k_doc, prefix, scale, workspace) -> (dq, dk, dv)
PyObject* backward_rule(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q must be a tensor"), &k = tensor(a[1], "k must be a tensor"),
                     &v = tensor(a[2], "v must be a tensor"), &o = tensor(a[3], "o must be a tensor"),
                     &lse = tensor(a[4], "lse must be a tensor"), &dout = tensor(a[5], "dout must be a tensor");
    const Problem p(q, k, v);
    const char* what = "o and dout must be like q, lse a contiguous float32 tensor [B, H, N_q], on q's device";
    check(o, q.scalar_type(), p.dev, what);
    check(dout, q.scalar_type(), p.dev, what);
    check(lse, at::kFloat, p.dev, what);
    check_sizes(o, q.sizes(), what);
    check_sizes(dout, q.sizes(), what);
    check_sizes(lse, {p.B, p.H, p.Nq}, what);
    const fa_score_rule r = rule_of(a + 6, p);
    const float scale = scale_of(a[12], p.d);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.dev);
    const at::Tensor dq = at::empty_like(q), dk = at::empty_like(k), dv = at::empty_like(v);
    at::Tensor ws;
    if (a[13] == Py_None) {
      ws = bytes(p_bwd_ws(p.B, p.H, p.Nq, p.Nk, p.d, r.q_doc != nullptr), q);
    } else {
      ws = tensor(a[13], "workspace must be a tensor");
      if (!ws.is_cuda() || ws.get_device() != p.dev || !ws.is_contiguous())
        bad("the workspace must be a contiguous tensor on q's device");
    }
    const fa_status s =
        p_bwd(q.const_data_ptr(), k.const_data_ptr(), v.const_data_ptr(), o.const_data_ptr(), dout.const_data_ptr(),
              static_cast<const float*>(lse.const_data_ptr()), dq.mutable_data_ptr(), dk.mutable_data_ptr(),
              dv.mutable_data_ptr(), &r, ws.mutable_data_ptr(), ws.nbytes(), p.B, p.H, p.Hkv, p.Nq, p.Nk, p.d, scale,
              p.dtype, stream_of(p.dev));
    return s == FA_OK ? pack({dq, dk, dv}) : status(s);
  });
}

// The pools of a cache, checked: (k_codes, k_params, v_codes, v_params).
struct Cache {
  fa_kv4_cache c{};
  at::Tensor codes, params;
  int64_t dev;
  explicit Cache(PyObject* const* a) {
    const char* what =
        "codes must be contiguous uint8 tensors [pages, H_kv, page_size, d / 2] and params contiguous fp16 or bf16 tensors "
        "[pages, H_kv, page_size, d / 32, 2] on one CUDA device";
    codes = tensor(a[0], what), params = tensor(a[1], what);
    const at::Tensor &vc = tensor(a[2], what), &vp = tensor(a[3], what);
    c.dtype = dtype_of(params);
    if (!codes.is_cuda() || codes.dim() != 4) bad(what);
    dev = codes.get_device();
    check(codes, at::kByte, dev, what);
    check(vc, at::kByte, dev, what);
    check(params, params.scalar_type(), dev, what);
    check(vp, params.scalar_type(), dev, what);
    check_sizes(vc, codes.sizes(), what);
    const int64_t shape[5] = {codes.size(0), codes.size(1), codes.size(2), codes.size(3) / 16, 2};
    check_sizes(params, shape, what);
    check_sizes(vp, shape, what);
    c.k_codes = codes.mutable_data_ptr(), c.k_params = params.mutable_data_ptr();
    c.v_codes = vc.mutable_data_ptr(), c.v_params = vp.mutable_data_ptr();
    c.num_pages = to_int(codes.size(0)), c.H_kv = to_int(codes.size(1));
    c.page_size = to_int(codes.size(2)), c.d = to_int(2 * codes.size(3));
  }
};
struct Table {
  const int32_t* data;
  int B, max_pages;
  Table(PyObject* o, int64_t dev) {
    const char* what = "page_table must be a contiguous int32 tensor [B, max_pages] on the cache's device";
    const at::Tensor& t = tensor(o, what);
    check(t, at::kInt, dev, what);
    if (t.dim() != 2) bad(what);
    B = to_int(t.size(0)), max_pages = to_int(t.size(1));
    data = t.const_data_ptr<int32_t>();
  }
};
constexpr const char* kInts = "start, count and lengths must be contiguous int32 tensors [B] on the cache's device";
constexpr const char* kParents = "parents must be a contiguous int32 tensor [B, N] on the same device";
constexpr const char* kPlanInts = "start and count must be contiguous int32 tensors [B] on the pages' device";
int whole(PyObject* o) {
  const int64_t x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw BadArgument{nullptr, nullptr};
  return to_int(x);
}

// (4 pools) -> (pages, H_kv, page_size, d, dtype code, device): the checks of a cache
PyObject* kv4_check(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* {
    const Cache c(a);
    return Py_BuildValue("iiiiiL", c.c.num_pages, c.c.H_kv, c.c.page_size, c.c.d, (int)c.c.dtype, (long long)c.dev);
  });
}

// (4 pools, k, v, page_table, start, count) -> None
PyObject* kv4_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const Cache c(a);
    const char* what = "k and v must be contiguous tensors [B, H_kv, N, d] of the cache's type, on its device";
    const at::Tensor &k = tensor(a[4], what), &v = tensor(a[5], what);
    const Table t(a[6], c.dev);
    check(k, c.params.scalar_type(), c.dev, what);
    check(v, c.params.scalar_type(), c.dev, what);
    if (k.dim() != 4) bad(what);
    check_sizes(k, {t.B, c.c.H_kv, k.size(2), c.c.d}, what);
    check_sizes(v, k.sizes(), what);
    if (a[7] == Py_None) bad(kInts);
    const int32_t *start = ints(a[7], {t.B}, c.dev, kInts), *count = ints(a[8], {t.B}, c.dev, kInts);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.dev);
    const fa_status s = p_append(&c.c, k.const_data_ptr(), v.const_data_ptr(), t.data, t.max_pages, start, count, t.B,
                                 to_int(k.size(2)), stream_of(c.dev));
    if (s != FA_OK) return status(s);
    Py_RETURN_NONE;
  });
}

// (4 pools, page_table, start, N, lengths) -> (k, v)
PyObject* kv4_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const Cache c(a);
    const Table t(a[4], c.dev);
    if (a[5] == Py_None || a[7] == Py_None) bad(kInts);
    const int32_t *start = ints(a[5], {t.B}, c.dev, kInts), *lengths = ints(a[7], {t.B}, c.dev, kInts);
    const int64_t N = PyLong_AsLongLong(a[6]);
    if (N == -1 && PyErr_Occurred()) throw BadArgument{nullptr, nullptr};
    const int rows = to_int(N);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.dev);
    const at::Tensor k = at::empty({t.B, c.c.H_kv, N, c.c.d}, c.params.options());
    const at::Tensor v = at::empty({t.B, c.c.H_kv, N, c.c.d}, c.params.options());
    const fa_status s = p_read(&c.c, t.data, t.max_pages, start, lengths, k.mutable_data_ptr(), v.mutable_data_ptr(), t.B,
                               rows, stream_of(c.dev));
    return s == FA_OK ? pack({k, v}) : status(s);
  });
}

// (q, 4 pools, page_table, lengths, scale, causal, cap, slopes, workspace) -> (o, lse)
PyObject* kv4_attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const Cache c(a + 1);
    const char* what = "q must be a contiguous tensor [B, H, N_q, d] of the cache's type, on its device, H_kv dividing H";
    const at::Tensor& q = tensor(a[0], what);
    check(q, c.params.scalar_type(), c.dev, what);
    const Table t(a[5], c.dev);
    if (q.dim() != 4 || q.size(0) != t.B || q.size(3) != c.c.d || c.c.H_kv < 1 || q.size(1) % c.c.H_kv) bad(what);
    if (a[6] == Py_None) bad(kInts);
    const int32_t* lengths = ints(a[6], {t.B}, c.dev, kInts);
    const float scale = scale_of(a[7], c.c.d);
    const bool causal = truth(a[8]);
    const float cap = (float)number(a[9]);
    const int H = to_int(q.size(1)), Nq = to_int(q.size(2));
    const float* slopes = slopes_of(a[10], H, c.dev);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.dev);
    const at::Tensor o = at::empty_like(q);
    const at::Tensor lse = at::empty({t.B, H, Nq}, q.options().dtype(at::kFloat));
    at::Tensor ws;
    if (a[11] == Py_None) {
      ws = bytes(p_attend_ws(t.B, H, c.c.H_kv, Nq, c.c.d), q);
    } else {
      ws = tensor(a[11], "workspace must be a tensor");
      if (!ws.is_cuda() || ws.get_device() != c.dev || !ws.is_contiguous())
        bad("the workspace must be a contiguous tensor on the cache's device");
    }
    const fa_status s = p_attend(q.const_data_ptr(), &c.c, t.data, t.max_pages, lengths, o.mutable_data_ptr(),
                                 static_cast<float*>(lse.mutable_data_ptr()), causal, cap, slopes, ws.mutable_data_ptr(),
                                 ws.nbytes(), t.B, H, Nq, scale, stream_of(c.dev));
    return s == FA_OK ? pack({o, lse}) : status(s);
  });
}

// (q, 4 pools, page_table, lengths, parents, count, scale, cap, slopes, workspace) -> (o, lse)
PyObject* kv4_attend_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const Cache c(a + 1);
    const char* what = "q must be a contiguous tensor [B, H, N_q, d] of the cache's type, on its device, H_kv dividing H";
    const at::Tensor& q = tensor(a[0], what);
    check(q, c.params.scalar_type(), c.dev, what);
    const Table t(a[5], c.dev);
    if (q.dim() != 4 || q.size(0) != t.B || q.size(3) != c.c.d || c.c.H_kv < 1 || q.size(1) % c.c.H_kv) bad(what);
    if (a[6] == Py_None) bad(kInts);
    const int32_t *lengths = ints(a[6], {t.B}, c.dev, kInts), *count = ints(a[8], {t.B}, c.dev, kInts);
    const int H = to_int(q.size(1)), Nq = to_int(q.size(2));
    if (a[7] == Py_None) bad(kParents);
    const int32_t* parents = ints(a[7], {t.B, Nq}, c.dev, kParents);
    const float scale = scale_of(a[9], c.c.d);
    const float cap = (float)number(a[10]);
    const float* slopes = slopes_of(a[11], H, c.dev);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.dev);
    const at::Tensor o = at::empty_like(q);
    const at::Tensor lse = at::empty({t.B, H, Nq}, q.options().dtype(at::kFloat));
    at::Tensor ws;
    if (a[12] == Py_None) {
      ws = bytes(p_tree_ws(t.B, H, c.c.H_kv, Nq, c.c.d), q);
    } else {
      ws = tensor(a[12], "workspace must be a tensor");
      if (!ws.is_cuda() || ws.get_device() != c.dev || !ws.is_contiguous())
        bad("the workspace must be a contiguous tensor on the cache's device");
    }
    const fa_status s = p_tree(q.const_data_ptr(), &c.c, t.data, t.max_pages, lengths, parents, count, o.mutable_data_ptr(),
                               static_cast<float*>(lse.mutable_data_ptr()), cap, slopes, ws.mutable_data_ptr(), ws.nbytes(),
                               t.B, H, Nq, scale, stream_of(c.dev));
    return s == FA_OK ? pack({o, lse}) : status(s);
  });
}

// (4 pools, page_table, start, path, kept) -> None
PyObject* kv4_keep(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const Cache c(a);
    const Table t(a[4], c.dev);
    const char* what = "path must be a contiguous int32 tensor [B, N] on the cache's device";
    const at::Tensor& path = tensor(a[6], what);
    check(path, at::kInt, c.dev, what);
    if (path.dim() != 2 || path.size(0) != t.B) bad(what);
    if (a[5] == Py_None || a[7] == Py_None) bad(kInts);
    const int32_t *start = ints(a[5], {t.B}, c.dev, kInts), *kept = ints(a[7], {t.B}, c.dev, kInts);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)c.dev);
    const fa_status s = p_keep(&c.c, t.data, t.max_pages, start, path.const_data_ptr<int32_t>(), kept, t.B,
                               to_int(path.size(1)), stream_of(c.dev));
    if (s != FA_OK) return status(s);
    Py_RETURN_NONE;
  });
}

// (table, held, free, free_count) -> device: the checks of a server's pages
constexpr const char* kPages =
    "pages must be contiguous int32 tensors table [B, max_pages], held [B], free [pages] and free_count [1] on one CUDA device";
struct Pages {
  int32_t *table, *held, *free, *free_count;
  int B, max_pages, num_free;
  int64_t dev;
  at::TensorOptions options;
  explicit Pages(PyObject* const* a) {
    const at::Tensor &t = tensor(a[0], kPages), &h = tensor(a[1], kPages), &f = tensor(a[2], kPages), &c = tensor(a[3], kPages);
    if (!t.is_cuda() || t.dim() != 2 || f.dim() != 1) bad(kPages);
    dev = t.get_device();
    for (const at::Tensor* x : {&t, &h, &f, &c}) check(*x, at::kInt, dev, kPages);
    check_sizes(h, {t.size(0)}, kPages);
    check_sizes(c, {1}, kPages);
    B = to_int(t.size(0)), max_pages = to_int(t.size(1)), num_free = to_int(f.size(0));
    table = t.mutable_data_ptr<int32_t>(), held = h.mutable_data_ptr<int32_t>();
    free = f.mutable_data_ptr<int32_t>(), free_count = c.mutable_data_ptr<int32_t>();
    options = t.options();
  }
};
PyObject* kv4_pages_check(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* { return PyLong_FromLongLong(Pages(a).dev); });
}

// (table, held, free, free_count, page_size, start, count, N, parents) -> (count, lengths, slots, positions)
PyObject* kv4_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const Pages p(a);
    if (a[5] == Py_None || a[6] == Py_None) bad(kPlanInts);
    const int32_t *start = ints(a[5], {p.B}, p.dev, kPlanInts), *count = ints(a[6], {p.B}, p.dev, kPlanInts);
    const int page_size = whole(a[4]), N = whole(a[7]);
    const int32_t* parents = ints(a[8], {p.B, N}, p.dev, kParents);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)p.dev);
    const at::Tensor out_count = at::empty({p.B}, p.options), lengths = at::empty({p.B}, p.options);
    const at::Tensor slots = at::empty({p.B, N}, p.options.dtype(at::kLong)), positions = at::empty({p.B, N}, p.options);
    const fa_status s = p_plan(p.table, p.held, p.max_pages, p.free, p.num_free, p.free_count, page_size, start, count, parents,
                               out_count.mutable_data_ptr<int32_t>(), lengths.mutable_data_ptr<int32_t>(),
                               slots.mutable_data_ptr<int64_t>(), positions.mutable_data_ptr<int32_t>(), p.B, N, stream_of(p.dev));
    return s == FA_OK ? pack({out_count, lengths, slots, positions}) : status(s);
  });
}

// Rows [B, heads, N, d] with any strides but of neighbouring channels.
fa_rotary_rows rows_of(const at::Tensor& in, const at::Tensor& out) {
  fa_rotary_rows r{};
  r.in = in.const_data_ptr();
  r.out = out.mutable_data_ptr();
  for (int i = 0; i < 3; ++i) r.in_stride[i] = in.stride(i), r.out_stride[i] = out.stride(i);
  return r;
}
// (q, k, positions, freqs, interleaved, backward, amplitude, out q, out k) -> (q, k)
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const char* what = "q and k must be [B, H, N, d] and [B, H_kv, N, d] of one type on one CUDA device, their channels neighbours";
    const at::Tensor& q = tensor(a[0], what);
    const bool has_k = a[1] != Py_None;
    const at::Tensor k = has_k ? tensor(a[1], what) : at::Tensor();
    if (!q.is_cuda() || q.dim() != 4) bad(what);
    const int64_t dev = q.get_device();
    const fa_dtype dtype = dtype_of(q);
    auto rows = [&](const at::Tensor& t, const at::Tensor& like, const char* text) {
      if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != q.scalar_type() || t.sizes() != like.sizes() ||
          (t.size(3) > 1 && t.stride(3) != 1))
        bad(text);
    };
    rows(q, q, what);
    if (has_k) {
      if (k.dim() != 4 || k.size(0) != q.size(0) || k.size(2) != q.size(2) || k.size(3) != q.size(3)) bad(what);
      rows(k, k, what);
    }
    const int B = to_int(q.size(0)), N = to_int(q.size(2));
    const int32_t* pos = ints(a[2], {B, N}, dev, "positions must be a contiguous int32 tensor [B, N] on q's device");
    const char* freq_what = "freqs must be a contiguous float64 tensor [dims / 2] on q's device";
    const at::Tensor& freqs = tensor(a[3], freq_what);
    check(freqs, at::kDouble, dev, freq_what);
    if (freqs.dim() != 1) bad(freq_what);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    const char* out_what = "out must be tensors like q and k, their channels neighbours";
    auto out_of = [&](PyObject* o, const at::Tensor& in) {
      if (o == Py_None) return at::empty(in.sizes(), in.options());
      const at::Tensor t = tensor(o, out_what);
      rows(t, in, out_what);
      return t;
    };
    if (!has_k && a[8] != Py_None) bad(out_what);
    const at::Tensor oq = out_of(a[7], q), ok = has_k ? out_of(a[8], k) : at::Tensor();
    const fa_rotary_rows rq = rows_of(q, oq), rk = has_k ? rows_of(k, ok) : fa_rotary_rows{};
    const fa_status s = p_rotary(&rq, has_k ? &rk : nullptr, pos, freqs.const_data_ptr<double>(), to_int(2 * freqs.size(0)),
                                 truth(a[4]), truth(a[5]), (float)number(a[6]), B, to_int(q.size(1)),
                                 has_k ? to_int(k.size(1)) : 0, N, to_int(q.size(3)), dtype, stream_of(dev));
    if (s != FA_OK) return status(s);
    if (has_k) return pack({oq, ok});
    return Py_BuildValue("NO", THPVariable_Wrap(oq), Py_None);
  });
}

// bind(addresses of the C functions, in the order below)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int kCalls = 13;
  return guarded(n, kCalls, [&]() -> PyObject* {
    void* p[kCalls];
    for (int i = 0; i < kCalls; ++i) {
      p[i] = PyLong_AsVoidPtr(a[i]);
      if (!p[i]) {
        if (PyErr_Occurred()) throw BadArgument{nullptr, nullptr};
        bad("a null function");
      }
    }
    p_fwd_ws = reinterpret_cast<decltype(p_fwd_ws)>(p[0]);
    p_bwd_ws = reinterpret_cast<decltype(p_bwd_ws)>(p[1]);
    p_fwd = reinterpret_cast<decltype(p_fwd)>(p[2]);
    p_bwd = reinterpret_cast<decltype(p_bwd)>(p[3]);
    p_append = reinterpret_cast<decltype(p_append)>(p[4]);
    p_read = reinterpret_cast<decltype(p_read)>(p[5]);
    p_attend_ws = reinterpret_cast<decltype(p_attend_ws)>(p[6]);
    p_attend = reinterpret_cast<decltype(p_attend)>(p[7]);
    p_tree_ws = reinterpret_cast<decltype(p_tree_ws)>(p[8]);
    p_tree = reinterpret_cast<decltype(p_tree)>(p[9]);
    p_keep = reinterpret_cast<decltype(p_keep)>(p[10]);
    p_plan = reinterpret_cast<decltype(p_plan)>(p[11]);
    p_rotary = reinterpret_cast<decltype(p_rotary)>(p[12]);
    Py_RETURN_NONE;
  });
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),     FAST(forward_rule), FAST(backward_rule), FAST(kv4_check), FAST(kv4_append),
                         FAST(kv4_read), FAST(kv4_attend),   FAST(kv4_attend_tree), FAST(kv4_keep),
                         FAST(kv4_pages_check), FAST(kv4_plan), FAST(rotary), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
