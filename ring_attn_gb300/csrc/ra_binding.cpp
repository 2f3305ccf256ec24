// Marshals torch tensors into the C ABI's cache calls, the rotation and the attention with changed scores.  They
// serve single tokens and short sequences,
// whose kernels take a few microseconds; describing a call's tensors through
// Python and ctypes takes 15 to 27 us on the host, here 5 to 9.
//
// Each function checks devices, types and dimensions (ValueError, as the rest of
// the binding), makes the cache's (the queries') device current, allocates outputs that were not
// given, calls the library on the device's current stream and returns
// (status, outputs).  Everything else is checked by the library.
#include <Python.h>

#include <algorithm>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/ringattn.h"

namespace {

decltype(&ring_attn_cache_append) g_append;
decltype(&ring_attn_cache_read) g_read;
decltype(&ring_attn_cache_fwd) g_fwd;
decltype(&ring_attn_cache_workspace_size) g_ws_size;
decltype(&ring_attn_scored_cache_fwd) g_scored_fwd;
decltype(&ring_attn_rope) g_rope;
decltype(&ring_attn_scored_fwd) g_sfwd;
decltype(&ring_attn_scored_bwd) g_sbwd;
decltype(&ring_attn_scored_varlen_fwd) g_svfwd;
decltype(&ring_attn_scored_varlen_bwd) g_svbwd;
decltype(&ring_attn_workspace_size) g_bwd_ws;
decltype(&ring_attn_varlen_workspace_size) g_varlen_ws;

#define RA_REFUSE(cond, ...) TORCH_CHECK_VALUE(!(cond), __VA_ARGS__)

// KVCache._call, and the arrays of a CuSeqlens as it holds them now.
struct CacheArg {
  const ra_kv_cache* cache;
  int index;
  int64_t hk, d;
};
struct CuArg {
  const int32_t *dev, *host;
  int n;
  int64_t total;
  int64_t max_new() const {
    int64_t m = 0;
    for (int i = 0; i < n; ++i) m = std::max<int64_t>(m, (int64_t)host[i + 1] - host[i]);
    return m;
  }
};
int64_t item(PyObject* t, Py_ssize_t i) {
  const long long v = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
CacheArg cache_arg(PyObject* t) {
  return {reinterpret_cast<const ra_kv_cache*>(item(t, 0)), (int)item(t, 1), item(t, 2), item(t, 3)};
}
CuArg cu_arg(PyObject* dev, PyObject* host, const CacheArg& c) {
  RA_REFUSE(!THPVariable_Check(dev) || !THPVariable_Check(host), "cu_seqlens must hold tensors");
  const at::Tensor &d = THPVariable_Unpack(dev), &h = THPVariable_Unpack(host);
  RA_REFUSE(!d.is_cuda() || d.get_device() != c.index, "CuSeqlens was prepared for ", d.device(), ", not cuda:", c.index);
  RA_REFUSE(!h.is_cpu() || h.dim() != 1 || h.numel() < 2 || h.numel() > INT32_MAX || h.scalar_type() != at::kInt ||
                !h.is_contiguous(),
            "cu_seqlens must be a 1-D array of n_seqs + 1 prefix sums");
  RA_REFUSE(d.scalar_type() != at::kInt || d.dim() != 1 || d.numel() != h.numel() || !d.is_contiguous(),
            "cu_seqlens's device array must be its host array's copy");
  CuArg u{d.const_data_ptr<int32_t>(), h.const_data_ptr<int32_t>(), (int)h.numel() - 1, 0};
  u.total = u.host[u.n];
  return u;
}

const at::Tensor& tensor(PyObject* o, int index) {
  RA_REFUSE(!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda(), "ring_attn_gb300 takes CUDA tensors only");
  const at::Tensor& t = THPVariable_Unpack(o);
  RA_REFUSE(t.get_device() != index, "tensor on ", t.device(), ", cache on cuda:", index);
  return t;
}

ra_tensor describe(const at::Tensor& t, int64_t dims) {
  ra_tensor r{};
  RA_REFUSE(t.dim() != dims, "expected a ", dims, "-D tensor, got ", t.sizes());
  RA_REFUSE(dims < 1 || dims > (int64_t)(sizeof(r.shape) / sizeof(r.shape[0])), "tensors must have 1 to 4 dimensions");
  r.data = t.data_ptr();
  RA_REFUSE(t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat, "unsupported dtype ", t.scalar_type());
  r.dtype = t.scalar_type() == at::kFloat ? RA_FP32 : RA_BF16;
  r.ndim = (int32_t)dims;
  for (int64_t i = 0; i < dims; ++i) {
    r.shape[i] = t.size(i);
    r.stride[i] = t.stride(i);
  }
  return r;
}

const int32_t* ints(PyObject* o, int64_t dims, int index, const char* what) {
  RA_REFUSE(!THPVariable_Check(o), what, " must be a ", dims, "-D int32 tensor on cuda:", index);
  const at::Tensor& t = THPVariable_Unpack(o);
  RA_REFUSE(t.scalar_type() != at::kInt || t.dim() != dims || !t.is_cuda() || t.get_device() != index, what,
            " must be a ", dims, "-D int32 tensor on cuda:", index);
  RA_REFUSE(t.size(-1) > 1 && t.stride(-1) != 1, what, " must be contiguous along its last dimension");
  return t.data_ptr<int32_t>();
}

ra_kv_seqs sequences(PyObject* page_table, PyObject* kv_lens, const CuArg& cu, int index) {
  ra_kv_seqs s{};
  s.page_table = ints(page_table, 2, index, "page_table");
  s.kv_lens = ints(kv_lens, 1, index, "kv_lens");
  const at::Tensor& table = THPVariable_Unpack(page_table);
  RA_REFUSE(table.size(0) != cu.n || THPVariable_Unpack(kv_lens).size(0) != cu.n,
            "page_table and kv_lens must have one row for each of the ", cu.n, " sequences");
  RA_REFUSE(table.size(1) > INT32_MAX, "page_table is too wide");
  s.page_table_stride = cu.n > 1 ? table.stride(0) : table.size(1);
  s.cu_seqlens_dev = cu.dev;
  s.cu_seqlens_host = cu.host;
  s.max_pages = (int32_t)table.size(1);
  s.n_seqs = cu.n;
  return s;
}

void* current_stream(int index) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream(); }
at::TensorOptions on(int index, at::ScalarType type) {
  return at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, (c10::DeviceIndex)index));
}
bool given(PyObject* o) { return o != Py_None; }
int truth(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw python_error();
  return r;
}

// (cache, cu's device array, its host array, k, v, page_table, kv_lens, q, cos, sin, positions, interleaved, q_out) -> (status, q_out)
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_VALUE(n == 13, "13 arguments");
  const CacheArg c = cache_arg(a[0]);
  const CuArg cu = cu_arg(a[1], a[2], c);
  const c10::cuda::OptionalCUDAGuard guard(at::Device(at::kCUDA, (c10::DeviceIndex)c.index));
  const ra_kv_seqs seqs = sequences(a[5], a[6], cu, c.index);
  const ra_tensor k = describe(tensor(a[3], c.index), 3), v = describe(tensor(a[4], c.index), 3);
  RA_REFUSE(given(a[12]) && !given(a[7]), "q_out without q");
  ra_tensor q{}, out{}, cos{}, sin{};
  at::Tensor q_out;
  if (given(a[7])) {
    const at::Tensor& tq = tensor(a[7], c.index);
    q = describe(tq, 3);
    q_out = given(a[12]) ? tensor(a[12], c.index) : at::empty(tq.sizes(), tq.options());
    out = describe(q_out, 3);
  }
  if (given(a[8])) {
    cos = describe(tensor(a[8], c.index), 2);
    sin = describe(tensor(a[9], c.index), 2);
  }
  const int32_t* pos = nullptr;
  if (given(a[10])) {
    pos = ints(a[10], 1, c.index, "positions");
    RA_REFUSE(THPVariable_Unpack(a[10]).size(0) < cu.total, "positions must have an entry for every new token");
  }
  const int inter = truth(a[11]);
  const int status = g_append(given(a[7]) ? &q : nullptr, &k, &v, given(a[8]) ? &cos : nullptr, given(a[8]) ? &sin : nullptr,
                              inter, pos, c.cache, &seqs, given(a[7]) ? &out : nullptr, current_stream(c.index));
  PyObject* r = given(a[12]) ? Py_NewRef(a[12]) : q_out.defined() ? THPVariable_Wrap(q_out) : Py_NewRef(Py_None);
  return Py_BuildValue("(iN)", status, r);
  END_HANDLE_TH_ERRORS
}

// (cache, cu's device array, its host array, page_table, kv_lens, k_out, v_out) -> (status, k_out, v_out)
PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_VALUE(n == 7, "7 arguments");
  const CacheArg c = cache_arg(a[0]);
  const CuArg cu = cu_arg(a[1], a[2], c);
  const c10::cuda::OptionalCUDAGuard guard(at::Device(at::kCUDA, (c10::DeviceIndex)c.index));
  const ra_kv_seqs seqs = sequences(a[3], a[4], cu, c.index);
  at::Tensor t[2];
  ra_tensor r[2];
  for (int i = 0; i < 2; ++i) {
    t[i] = given(a[5 + i]) ? tensor(a[5 + i], c.index) : at::empty({cu.total, c.hk, c.d}, on(c.index, at::kBFloat16));
    r[i] = describe(t[i], 3);
  }
  const int status = g_read(c.cache, &seqs, &r[0], &r[1], current_stream(c.index));
  return Py_BuildValue("(iNN)", status, given(a[5]) ? Py_NewRef(a[5]) : THPVariable_Wrap(t[0]),
                       given(a[6]) ? Py_NewRef(a[6]) : THPVariable_Wrap(t[1]));
  END_HANDLE_TH_ERRORS
}

// Scores._parts (softcap, slopes, prefix) for a call of h query heads and n sequences on device `index`, with the
// tensors as they are now; `given` is false for None.
struct ScoresArg {
  bool given;
  ra_scores c;
  const ra_scores* get() const { return given ? &c : nullptr; }
};
const void* per_entry(PyObject* o, at::ScalarType type, int index, int64_t n, const char* what, const char* of) {
  if (!given(o)) return nullptr;
  RA_REFUSE(!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda(), "ring_attn_gb300 takes CUDA tensors only");
  const at::Tensor& t = THPVariable_Unpack(o);
  RA_REFUSE(t.scalar_type() != type || t.dim() != 1 || !t.is_contiguous(), what, " must be a contiguous 1-D ", type, " tensor");
  RA_REFUSE(t.get_device() != index, "scores on cuda:", t.get_device(), ", call on cuda:", index);
  RA_REFUSE(t.numel() != n, what, " must have one entry for each of the ", n, " ", of);
  return t.data_ptr();
}
ScoresArg scores_arg(PyObject* t, int index, int64_t h, int64_t n) {
  ScoresArg r{};
  if (!given(t)) return r;
  RA_REFUSE(!PyTuple_Check(t) || PyTuple_GET_SIZE(t) != 3, "scores must be a Scores");
  r.given = true;
  r.c.softcap = (float)PyFloat_AsDouble(PyTuple_GET_ITEM(t, 0));
  if (PyErr_Occurred()) throw python_error();
  r.c.slopes = static_cast<const float*>(per_entry(PyTuple_GET_ITEM(t, 1), at::kFloat, index, h, "slopes", "query heads"));
  r.c.prefix = static_cast<const int32_t*>(per_entry(PyTuple_GET_ITEM(t, 2), at::kInt, index, n, "prefix", "sequences"));
  return r;
}

// (cache, cu's device array, its host array, q, page_table, kv_lens, causal, scale, max_kv_len, out, lse, out_fp32, workspace, scores) -> (status, out, lse)
PyObject* cache_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_VALUE(n == 14, "14 arguments");
  const CacheArg c = cache_arg(a[0]);
  const CuArg cu = cu_arg(a[1], a[2], c);
  const c10::cuda::OptionalCUDAGuard guard(at::Device(at::kCUDA, (c10::DeviceIndex)c.index));
  const ra_kv_seqs seqs = sequences(a[4], a[5], cu, c.index);
  const at::Tensor& tq = tensor(a[3], c.index);
  const ra_tensor q = describe(tq, 3);
  const ScoresArg scores = scores_arg(a[13], c.index, tq.size(1), cu.n);
  const int causal = truth(a[6]), fp32 = truth(a[11]);
  const double scale = PyFloat_AsDouble(a[7]);
  const long max_kv = PyLong_AsLong(a[8]);
  if (PyErr_Occurred()) throw python_error();
  RA_REFUSE(max_kv < 0 || max_kv > INT32_MAX, "max_kv_len must be 0 or a length");
  const at::Tensor out = given(a[9]) ? tensor(a[9], c.index)
                                     : at::empty(tq.sizes(), on(c.index, fp32 ? at::kFloat : at::kBFloat16));
  const at::Tensor lse = given(a[10]) ? tensor(a[10], c.index) : at::empty({tq.size(1), tq.size(0)}, on(c.index, at::kFloat));
  ra_tensor o = describe(out, 3), l = describe(lse, 2);
  at::Tensor ws;
  if (given(a[12])) {
    ws = tensor(a[12], c.index);
    RA_REFUSE(!ws.is_contiguous(), "workspace must be contiguous");
  } else if (cu.total > 0) {
    ws = at::empty({(int64_t)g_ws_size(cu.total, cu.max_new(), tq.size(1), c.hk, c.d, cu.n)}, on(c.index, at::kByte));
  }
  void *wp = ws.defined() ? ws.data_ptr() : nullptr, *stream = current_stream(c.index);
  const size_t wn = ws.defined() ? ws.nbytes() : 0;
  const int status = scores.given ? g_scored_fwd(&q, c.cache, &seqs, causal, (float)scale, scores.get(), (int32_t)max_kv, &o, &l, wp, wn, stream)
                            : g_fwd(&q, c.cache, &seqs, causal, (float)scale, (int32_t)max_kv, &o, &l, wp, wn, stream);
  return Py_BuildValue("(iNN)", status, given(a[9]) ? Py_NewRef(a[9]) : THPVariable_Wrap(out),
                       given(a[10]) ? Py_NewRef(a[10]) : THPVariable_Wrap(lse));
  END_HANDLE_TH_ERRORS
}

// A (b, h, s, d) tensor, or (rows, h, d) as b = 1.
ra_tensor describe_rows(const at::Tensor& t) {
  if (t.dim() != 3) return describe(t, 4);
  const ra_tensor x = describe(t, 3);
  ra_tensor r = x;
  r.ndim = 4;
  const int from[4] = {-1, 1, 0, 2};
  for (int i = 0; i < 4; ++i) {
    r.shape[i] = from[i] < 0 ? 1 : x.shape[from[i]];
    r.stride[i] = from[i] < 0 ? 8 : x.stride[from[i]];
  }
  return r;
}

// (q, k, cos, sin, positions, axes, interleaved, inverse, layout, n_shards, q_out, k_out) -> (status, q_out, k_out)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_VALUE(n == 12, "12 arguments");
  RA_REFUSE(!THPVariable_Check(a[0]) || !THPVariable_Unpack(a[0]).is_cuda(), "ring_attn_gb300 takes CUDA tensors only");
  const at::Tensor& tq = THPVariable_Unpack(a[0]);
  const int index = tq.get_device();
  auto here = [index](PyObject* o) -> const at::Tensor& {
    RA_REFUSE(!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda(), "ring_attn_gb300 takes CUDA tensors only");
    const at::Tensor& t = THPVariable_Unpack(o);
    RA_REFUSE(t.get_device() != index, "tensor on ", t.device(), ", q on cuda:", index);
    return t;
  };
  const c10::cuda::OptionalCUDAGuard guard(at::Device(at::kCUDA, (c10::DeviceIndex)index));
  const bool has_k = given(a[1]);
  RA_REFUSE(given(a[11]) && !has_k, "k_out without k");
  ra_tensor in[2], out[2];
  at::Tensor made[2];
  for (int i = 0; i < (has_k ? 2 : 1); ++i) {
    const at::Tensor& t = here(a[i]);
    RA_REFUSE(t.dim() != tq.dim(), "q and k must both be (b, h, s, d) or (rows, h, d)");
    in[i] = describe_rows(t);
    made[i] = given(a[10 + i]) ? here(a[10 + i]) : at::empty(t.sizes(), t.options());
    RA_REFUSE(made[i].dim() != tq.dim(), "outputs must have their inputs' shapes");
    out[i] = describe_rows(made[i]);
  }
  const ra_tensor cos = describe(here(a[2]), 2), sin = describe(here(a[3]), 2);
  ra_rope_positions p{};
  if (given(a[4])) {
    const at::Tensor& t = here(a[4]);
    const int64_t rows = tq.dim() == 3 ? 1 : 2;  // dimensions of one axis
    RA_REFUSE(t.scalar_type() != at::kInt || (t.dim() != rows && t.dim() != rows + 1),
              "positions must be int32, ", rows == 1 ? "(rows) or (axes, rows)" : "(b, s) or (axes, b, s)");
    const bool axes = t.dim() == rows + 1;
    p.n_axes = axes ? (int32_t)std::min<int64_t>(t.size(0), 256) : 1;
    p.stride_axis = axes ? t.stride(0) : 0;
    p.stride_s = t.stride(-1);
    p.stride_b = rows == 2 ? t.stride(-2) : 0;
    RA_REFUSE(t.size(-1) != in[0].shape[2] || (rows == 2 && t.size(-2) != in[0].shape[0]),
              "positions must have an entry for every row");
    p.positions = t.const_data_ptr<int32_t>();
  }
  if (given(a[5])) {
    RA_REFUSE(!PyBytes_Check(a[5]) || PyBytes_GET_SIZE(a[5]) != cos.shape[1], "axes must name an axis for each of the ", cos.shape[1],
              " pairs");
    RA_REFUSE(!given(a[4]), "axes without positions");
    p.pair_axis = reinterpret_cast<const uint8_t*>(PyBytes_AS_STRING(a[5]));
  }
  const int inter = truth(a[6]), inverse = truth(a[7]);
  const long layout = PyLong_AsLong(a[8]), shards = PyLong_AsLong(a[9]);
  if (PyErr_Occurred()) throw python_error();
  const int status = g_rope(&in[0], has_k ? &in[1] : nullptr, &cos, &sin, inter, given(a[4]) ? &p : nullptr, (int32_t)layout,
                            (int32_t)shards, inverse, &out[0], has_k ? &out[1] : nullptr, current_stream(index));
  return Py_BuildValue("(iNN)", status, given(a[10]) ? Py_NewRef(a[10]) : THPVariable_Wrap(made[0]),
                       !has_k ? Py_NewRef(Py_None) : given(a[11]) ? Py_NewRef(a[11]) : THPVariable_Wrap(made[1]));
  END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- attention with changed scores
// Tensors of one call, on q's device: the inputs a[0 .. n) and the results r[0 .. m), where given, are checked first.
struct OnDevice {
  int index;
  OnDevice(PyObject* q, PyObject* const* a, int n, PyObject* const* r, int m) : index(-1) {
    RA_REFUSE(!THPVariable_Check(q) || !THPVariable_Unpack(q).is_cuda(), "ring_attn_gb300 takes CUDA tensors only");
    index = THPVariable_Unpack(q).get_device();
    auto check = [this](PyObject* o) {
      const at::Tensor& t = (*this)(o);
      RA_REFUSE(t.dim() < 1 || t.dim() > 4, "tensors must have 1 to 4 dimensions, got ", t.sizes());
    };
    for (int i = 0; i < n; ++i) check(a[i]);
    for (int i = 0; i < m; ++i)
      if (given(r[i])) check(r[i]);
  }
  const at::Tensor& operator()(PyObject* o) const {
    RA_REFUSE(!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda(), "ring_attn_gb300 takes CUDA tensors only");
    const at::Tensor& t = THPVariable_Unpack(o);
    RA_REFUSE(t.get_device() != index, "tensor on ", t.device(), ", q on cuda:", index);
    return t;
  }
};
// A result that the caller gave, or a new one.
struct Result {
  PyObject* mine;
  at::Tensor t;
  ra_tensor d;
  template <class F>
  Result(PyObject* o, const OnDevice& on, F&& make) : mine(given(o) ? o : nullptr), t(mine ? on(o) : make()), d(describe(t, t.dim())) {}
  PyObject* out() const { return mine ? Py_NewRef(mine) : THPVariable_Wrap(t); }
};
struct Space {
  at::Tensor t;
  Space(PyObject* o, const OnDevice& dev, size_t need) {
    if (given(o)) {
      t = dev(o);
      RA_REFUSE(!t.is_contiguous(), "workspace must be contiguous");
    } else if (need) {
      t = at::empty({(int64_t)need}, on(dev.index, at::kByte));
    }
  }
  void* data() const { return t.defined() ? t.data_ptr() : nullptr; }
  size_t bytes() const { return t.defined() ? t.nbytes() : 0; }
};
struct How {
  int layout, shards, causal;
  float scale;
};
// layout, n_shards, causal, scale
How how(PyObject* const* a) {
  How h{(int)PyLong_AsLong(a[0]), (int)PyLong_AsLong(a[1]), truth(a[2]), (float)PyFloat_AsDouble(a[3])};
  if (PyErr_Occurred()) throw python_error();
  return h;
}
ScoresArg scores_of(PyObject* t, int index, int64_t h, int64_t n) {
  RA_REFUSE(!given(t), "scores must be a Scores");
  return scores_arg(t, index, h, n);
}
at::Tensor four(const at::Tensor& q) {
  RA_REFUSE(q.dim() != 4, "expected a 4-D tensor, got ", q.sizes());
  return q;
}

// (q, k, v, layout, n_shards, causal, scale, scores, out, lse) -> (status, out, lse)
PyObject* scored_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_VALUE(n == 10, "10 arguments");
  const OnDevice dev(a[0], a, 3, a + 8, 2);
  const at::Tensor q = four(dev(a[0]));
  const How x = how(a + 3);
  const ScoresArg z = scores_of(a[7], dev.index, q.size(1), q.size(0));
  const c10::cuda::OptionalCUDAGuard guard(at::Device(at::kCUDA, (c10::DeviceIndex)dev.index));
  const ra_tensor tq = describe(q, 4), tk = describe(dev(a[1]), 4), tv = describe(dev(a[2]), 4);
  Result out(a[8], dev, [&] { return at::empty_like(q); });
  Result lse(a[9], dev, [&] { return at::empty({q.size(0), q.size(1), q.size(2)}, on(dev.index, at::kFloat)); });
  const int status = g_sfwd(&tq, &tk, &tv, x.layout, x.shards, x.causal, x.scale, z.get(), &out.d, &lse.d, current_stream(dev.index));
  return Py_BuildValue("(iNN)", status, out.out(), lse.out());
  END_HANDLE_TH_ERRORS
}

// (dout, q, k, v, out, lse, layout, n_shards, causal, scale, scores, dq, dk, dv, workspace) -> (status, dq, dk, dv)
PyObject* scored_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_VALUE(n == 15, "15 arguments");
  const OnDevice dev(a[1], a, 6, a + 11, 3);
  const at::Tensor q = four(dev(a[1]));
  const How x = how(a + 6);
  const ScoresArg z = scores_of(a[10], dev.index, q.size(1), q.size(0));
  const c10::cuda::OptionalCUDAGuard guard(at::Device(at::kCUDA, (c10::DeviceIndex)dev.index));
  ra_tensor t[6];
  for (int i = 0; i < 6; ++i) t[i] = describe(dev(a[i]), dev(a[i]).dim());
  Result dq(a[11], dev, [&] { return at::empty_like(q); });
  Result dk(a[12], dev, [&] { return at::empty_like(dev(a[2])); });
  Result dv(a[13], dev, [&] { return at::empty_like(dev(a[3])); });
  const Space ws(a[14], dev, g_bwd_ws(RA_OP_BWD, q.size(0), q.size(1), q.size(2), q.size(3), x.shards));
  const int status = g_sbwd(&t[0], &t[1], &t[2], &t[3], &t[4], &t[5], x.layout, x.shards, x.causal, x.scale, z.get(), &dq.d, &dk.d,
                            &dv.d, ws.data(), ws.bytes(), current_stream(dev.index));
  return Py_BuildValue("(iNNN)", status, dq.out(), dk.out(), dv.out());
  END_HANDLE_TH_ERRORS
}

// The prefix sums of a varlen call, its longest sequence (max_seqlen, if given) and q's heads and head dim.
struct Packed {
  CuArg cu;
  int32_t longest;
  int64_t h, d;
  Packed(PyObject* dev, PyObject* host, PyObject* max_seqlen, const at::Tensor& q, int index)
      : cu(cu_arg(dev, host, CacheArg{nullptr, index, 0, 0})), longest(0), h(0), d(0) {
    RA_REFUSE(q.dim() != 3, "expected a 3-D tensor, got ", q.sizes());
    const long m = given(max_seqlen) ? PyLong_AsLong(max_seqlen) : (long)cu.max_new();
    if (PyErr_Occurred()) throw python_error();
    longest = (int32_t)std::min<long>(std::max<long>(m, -1), INT32_MAX);
    h = q.size(0) == cu.total ? q.size(1) : q.size(0);
    d = q.size(2);
  }
};

// (q, k, v, cu's device array, its host array, max_seqlen, layout, n_shards, causal, scale, scores, out, lse, workspace) -> (status, out, lse)
PyObject* scored_varlen_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_VALUE(n == 14, "14 arguments");
  const OnDevice dev(a[0], a, 3, a + 11, 2);
  const c10::cuda::OptionalCUDAGuard guard(at::Device(at::kCUDA, (c10::DeviceIndex)dev.index));
  const at::Tensor& q = dev(a[0]);
  const Packed p(a[3], a[4], a[5], q, dev.index);
  const ra_tensor tq = describe(q, 3), tk = describe(dev(a[1]), 3), tv = describe(dev(a[2]), 3);
  const How x = how(a + 6);
  const ScoresArg z = scores_of(a[10], dev.index, p.h, p.cu.n);
  Result out(a[11], dev, [&] { return at::empty_like(q); });
  Result lse(a[12], dev, [&] { return at::empty({p.h, p.cu.total}, on(dev.index, at::kFloat)); });
  const Space ws(a[13], dev, g_varlen_ws(RA_OP_FWD, p.cu.total, p.h, p.d, x.layout, x.shards));
  const int status = g_svfwd(&tq, &tk, &tv, p.cu.dev, p.cu.host, p.cu.n, p.longest, x.layout, x.shards, x.causal, x.scale, z.get(),
                             &out.d, &lse.d, ws.data(), ws.bytes(), current_stream(dev.index));
  return Py_BuildValue("(iNN)", status, out.out(), lse.out());
  END_HANDLE_TH_ERRORS
}

// (dout, q, k, v, out, lse, cu's device array, its host array, max_seqlen, layout, n_shards, causal, scale, scores, dq, dk, dv, workspace)
// -> (status, dq, dk, dv)
PyObject* scored_varlen_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_VALUE(n == 18, "18 arguments");
  const OnDevice dev(a[1], a, 6, a + 14, 3);
  const c10::cuda::OptionalCUDAGuard guard(at::Device(at::kCUDA, (c10::DeviceIndex)dev.index));
  const at::Tensor& q = dev(a[1]);
  const Packed p(a[6], a[7], a[8], q, dev.index);
  ra_tensor t[6];
  for (int i = 0; i < 6; ++i) t[i] = describe(dev(a[i]), dev(a[i]).dim());
  const How x = how(a + 9);
  const ScoresArg z = scores_of(a[13], dev.index, p.h, p.cu.n);
  Result dq(a[14], dev, [&] { return at::empty_like(q); });
  Result dk(a[15], dev, [&] { return at::empty_like(dev(a[2])); });
  Result dv(a[16], dev, [&] { return at::empty_like(dev(a[3])); });
  const Space ws(a[17], dev, g_varlen_ws(RA_OP_BWD, p.cu.total, p.h, p.d, x.layout, x.shards));
  const int status = g_svbwd(&t[0], &t[1], &t[2], &t[3], &t[4], &t[5], p.cu.dev, p.cu.host, p.cu.n, p.longest, x.layout, x.shards,
                             x.causal, x.scale, z.get(), &dq.d, &dk.d, &dv.d, ws.data(), ws.bytes(), current_stream(dev.index));
  return Py_BuildValue("(iNNN)", status, dq.out(), dk.out(), dv.out());
  END_HANDLE_TH_ERRORS
}

// The library's functions, by address.
PyObject* use(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_VALUE(n == 12, "12 arguments");
  void* p[12];
  for (int i = 0; i < 12; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null function");
      throw python_error();
    }
  }
  g_append = reinterpret_cast<decltype(g_append)>(p[0]);
  g_read = reinterpret_cast<decltype(g_read)>(p[1]);
  g_fwd = reinterpret_cast<decltype(g_fwd)>(p[2]);
  g_ws_size = reinterpret_cast<decltype(g_ws_size)>(p[3]);
  g_scored_fwd = reinterpret_cast<decltype(g_scored_fwd)>(p[4]);
  g_rope = reinterpret_cast<decltype(g_rope)>(p[5]);
  g_sfwd = reinterpret_cast<decltype(g_sfwd)>(p[6]);
  g_sbwd = reinterpret_cast<decltype(g_sbwd)>(p[7]);
  g_svfwd = reinterpret_cast<decltype(g_svfwd)>(p[8]);
  g_svbwd = reinterpret_cast<decltype(g_svbwd)>(p[9]);
  g_bwd_ws = reinterpret_cast<decltype(g_bwd_ws)>(p[10]);
  g_varlen_ws = reinterpret_cast<decltype(g_varlen_ws)>(p[11]);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}
PyMethodDef g_methods[] = {{"use", fast(use), METH_FASTCALL, nullptr},
                           {"cache_append", fast(cache_append), METH_FASTCALL, nullptr},
                           {"cache_read", fast(cache_read), METH_FASTCALL, nullptr},
                           {"cache_fwd", fast(cache_fwd), METH_FASTCALL, nullptr},
                           {"rope", fast(rope), METH_FASTCALL, nullptr},
                           {"scored_fwd", fast(scored_fwd), METH_FASTCALL, nullptr},
                           {"scored_bwd", fast(scored_bwd), METH_FASTCALL, nullptr},
                           {"scored_varlen_fwd", fast(scored_varlen_fwd), METH_FASTCALL, nullptr},
                           {"scored_varlen_bwd", fast(scored_varlen_bwd), METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ra_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ra_binding(void) { return PyModule_Create(&g_module); }
