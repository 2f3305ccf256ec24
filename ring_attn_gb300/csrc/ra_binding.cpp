// Marshals torch tensors into the C ABI's cache calls.  They serve single tokens,
// whose kernels take a few microseconds; describing a call's tensors through
// Python and ctypes takes 15 to 27 us on the host, here 5 to 9.
//
// Each function checks devices, types and dimensions (ValueError, as the rest of
// the binding), makes the cache's device current, allocates outputs that were not
// given, calls the library on the device's current stream and returns
// (status, outputs).  Everything else is checked by the library.
#include <Python.h>

#include <algorithm>

#include <ATen/ops/empty.h>
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
  r.data = t.data_ptr();
  RA_REFUSE(t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat, "unsupported dtype ", t.scalar_type());
  r.dtype = t.scalar_type() == at::kFloat ? RA_FP32 : RA_BF16;
  RA_REFUSE(t.dim() != dims, "expected a ", dims, "-D tensor, got ", t.sizes());
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

// (cache, cu's device array, its host array, q, page_table, kv_lens, causal, scale, max_kv_len, out, lse, out_fp32, workspace) -> (status, out, lse)
PyObject* cache_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_VALUE(n == 13, "13 arguments");
  const CacheArg c = cache_arg(a[0]);
  const CuArg cu = cu_arg(a[1], a[2], c);
  const c10::cuda::OptionalCUDAGuard guard(at::Device(at::kCUDA, (c10::DeviceIndex)c.index));
  const ra_kv_seqs seqs = sequences(a[4], a[5], cu, c.index);
  const at::Tensor& tq = tensor(a[3], c.index);
  const ra_tensor q = describe(tq, 3);
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
  const int status = g_fwd(&q, c.cache, &seqs, causal, (float)scale, (int32_t)max_kv, &o, &l, ws.defined() ? ws.data_ptr() : nullptr,
                           ws.defined() ? ws.nbytes() : 0, current_stream(c.index));
  return Py_BuildValue("(iNN)", status, given(a[9]) ? Py_NewRef(a[9]) : THPVariable_Wrap(out),
                       given(a[10]) ? Py_NewRef(a[10]) : THPVariable_Wrap(lse));
  END_HANDLE_TH_ERRORS
}

// The library's functions, by address.
PyObject* use(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_VALUE(n == 4, "4 arguments");
  void* p[4];
  for (int i = 0; i < 4; ++i) {
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
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ra_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ra_binding(void) { return PyModule_Create(&g_module); }
