// swa_bind.cpp — the rotary and paged-cache calls as a CPython extension: checks
// torch tensors against a call's parameters, takes their pointers and strides,
// and calls the C entry point whose address it is given.  It does what ctypes
// would, in a microsecond instead of ten: these calls run once per layer and
// token, where a kernel takes a few microseconds.
//
// A tensor that does not fit raises ValueError before anything is enqueued; the
// entry point's status is returned.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <optional>
#include <sstream>
#include <stdexcept>
#include <vector>

#include "swa.h"

namespace {

using Shape = c10::IntArrayRef;

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

const at::Tensor* tensor_or_none(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + ": expected a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o, const char* name) {
  const at::Tensor* t = tensor_or_none(o, name);
  if (!t) throw Refused(std::string(name) + " is required");
  return *t;
}

[[noreturn]] void refuse(const at::Tensor& t, const char* name, Shape shape, at::ScalarType type, int device,
                         const char* what) {
  std::ostringstream s;
  s << name << ": expected " << shape << " " << type << " on CUDA device " << device << what << ", got " << t.sizes()
    << " " << t.scalar_type() << " on " << t.device() << " with strides " << t.strides();
  throw Refused(s.str());
}
void expect(const at::Tensor& t, const char* name, Shape shape, at::ScalarType type, int device) {
  if (t.scalar_type() != type || t.sizes() != shape || !t.is_cuda() || t.get_device() != device)
    refuse(t, name, shape, type, device, "");
}
void expect_dense(const at::Tensor& t, const char* name, Shape shape, at::ScalarType type, int device) {
  expect(t, name, shape, type, device);
  if (!t.is_contiguous()) refuse(t, name, shape, type, device, " (contiguous)");
}
void expect_rows(const at::Tensor& t, const char* name, Shape shape, at::ScalarType type, int device) {
  if (t.stride(-1) != 1 && shape.back() != 1) refuse(t, name, shape, type, device, " (the last dimension contiguous)");
}

at::ScalarType scalar_type(int32_t dtype) {
  return dtype == SWA_DTYPE_FP16 ? at::kHalf : (dtype == SWA_DTYPE_FP32 ? at::kFloat : at::kBFloat16);
}

// Pointer and strides (none when dense) of a [B,N,S,D] / [T,N,D] tensor.
struct Arg {
  void* ptr = nullptr;
  swa_strides_t s{};
  bool strided = false;
  const swa_strides_t* strides() const { return strided ? &s : nullptr; }
};
Arg arg(const at::Tensor& t, const char* name, Shape shape, at::ScalarType type, int device) {
  expect(t, name, shape, type, device);
  Arg a;
  a.ptr = t.data_ptr();
  if (!t.is_contiguous()) {
    expect_rows(t, name, shape, type, device);
    a.strided = true;
    if (shape.size() == 4) a.s = swa_strides_t{t.stride(0), t.stride(2), t.stride(1)};
    else a.s = swa_strides_t{0, t.stride(0), t.stride(1)};
  }
  return a;
}

struct Pages {
  void* ptr = nullptr;
  swa_page_strides_t s{};
  bool strided = false;
  const swa_page_strides_t* strides() const { return strided ? &s : nullptr; }
};
Pages pages(const at::Tensor& t, const char* name, const swa_paged_params_t& p, at::ScalarType type, int device) {
  const int64_t n_kv = p.N_kv ? p.N_kv : p.N;
  const bool bnsd = p.cache_layout == SWA_LAYOUT_BNSD;
  const int64_t shape[4] = {p.num_pages, bnsd ? n_kv : p.page_size, bnsd ? p.page_size : n_kv, p.D};
  expect(t, name, shape, type, device);
  Pages a;
  a.ptr = t.data_ptr();
  if (!t.is_contiguous()) {
    expect_rows(t, name, shape, type, device);
    a.strided = true;
    a.s = bnsd ? swa_page_strides_t{t.stride(0), t.stride(1), t.stride(2)}
               : swa_page_strides_t{t.stride(0), t.stride(2), t.stride(1)};
  }
  return a;
}

const int32_t* block_table(const at::Tensor& t, const swa_paged_params_t& p, int device, int64_t* row) {
  const int64_t shape[2] = {p.B, p.max_pages};
  expect(t, "block_table", shape, at::kInt, device);
  *row = 0;
  if (!t.is_contiguous()) {
    if ((t.stride(1) != 1 && p.max_pages > 1) || (t.stride(0) < p.max_pages && p.B > 1))
      refuse(t, "block_table", shape, at::kInt, device, " (rows contiguous and apart)");
    if (p.B > 1) *row = t.stride(0);
  }
  return static_cast<const int32_t*>(t.data_ptr());
}

at::ScalarType page_type(const swa_paged_params_t& p) {
  return p.cache_dtype == SWA_CACHE_E4M3 ? at::kFloat8_e4m3fn : scalar_type(p.dtype);
}
// The exponents of an 8-bit cache, NULL for None (the library says which it wants).
int8_t* exponents(PyObject* o, const char* name, const swa_paged_params_t& p, int device) {
  const at::Tensor* t = tensor_or_none(o, name);
  if (!t) return nullptr;
  const int64_t shape[3] = {p.num_pages, p.N_kv ? p.N_kv : p.N, p.page_size};
  expect_dense(*t, name, shape, at::kChar, device);
  return static_cast<int8_t*>(t->data_ptr());
}
// The bits of a tree, [T_q, words], and the words between rows.
const uint32_t* tree_rows(const at::Tensor& t, const swa_paged_params_t& p, int device, int64_t* row) {
  int64_t longest = 0, last = 0;
  for (int64_t b = 0; b < p.B; ++b) {
    longest = std::max(longest, p.cu_seqlens_q[b] - last);
    last = p.cu_seqlens_q[b];
  }
  const int64_t words = std::max<int64_t>((longest + 31) / 32, 1);
  const int64_t shape[2] = {p.T_q, words};
  if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != p.T_q || t.size(1) < words || !t.is_cuda() ||
      t.get_device() != device || (t.stride(1) != 1 && t.size(1) > 1) || (t.stride(0) < t.size(1) && p.T_q > 1))
    refuse(t, "tree", shape, at::kInt, device, " (rows contiguous and apart; more words may follow)");
  *row = p.T_q > 1 ? t.stride(0) : t.size(1);
  return static_cast<const uint32_t*>(t.data_ptr());
}

// [n_axes, rows], the rows in any shape; one axis may leave its dimension out.
const int32_t* positions(const at::Tensor& t, int64_t n_axes, int64_t rows, int device) {
  if (t.scalar_type() != at::kInt || !t.is_cuda() || t.get_device() != device || t.numel() != n_axes * rows ||
      (n_axes > 1 && (t.dim() < 2 || t.size(0) != n_axes)) || !t.is_contiguous())
    refuse(t, "positions", {n_axes, rows}, at::kInt, device, " (contiguous)");
  return static_cast<const int32_t*>(t.data_ptr());
}

const at::Tensor& workspace(PyObject* o, int device) {
  const at::Tensor& t = tensor(o, "workspace");
  if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous())
    throw Refused("workspace must be contiguous and on the device of the tensors");
  return t;
}

int device_of(const at::Tensor& t) {
  if (!t.is_cuda()) throw Refused("the tensors must be on a CUDA device");
  return static_cast<int>(t.get_device());
}

// An integer as a pointer.  Anything else is refused: the NULL that the
// conversion gives in its place would be taken for an answer.
template <typename T>
T address(PyObject* o, const char* name) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused(std::string(name) + ": expected an address as an integer");
  }
  return reinterpret_cast<T>(p);
}

// Makes `device` current if it is not, and picks the stream.
struct On {
  std::optional<c10::cuda::CUDAGuard> guard;
  swa_stream_t stream;
  On(int device, PyObject* s) {
    if (c10::cuda::current_device() != device) guard.emplace(static_cast<c10::DeviceIndex>(device));
    if (s == Py_None)
      stream = reinterpret_cast<swa_stream_t>(
          c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream());
    else
      stream = address<swa_stream_t>(s, "stream");  // (0 is the default stream)
  }
};

// The library's part of a call, without the interpreter's lock: a launch waits
// while the stream's queue is full, and other threads run meanwhile.  Whatever
// comes from a Python object is taken before.
template <typename F, typename... A>
swa_status_t unlocked(F* fn, A... a) {
  PyThreadState* const state = PyEval_SaveThread();
  const swa_status_t st = fn(a...);
  PyEval_RestoreThread(state);
  return st;
}

template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F&& body) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    return nullptr;
  }
  try {
    return PyLong_FromLong(body());
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// rope(fn, params, q, k, positions, q_out, k_out, stream)
PyObject* bind_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> swa_status_t {
    const auto fn = address<decltype(&swa_rope_forward)>(a[0], "entry point");
    const swa_rope_params_t& p = *address<const swa_rope_params_t*>(a[1], "parameters");
    const at::Tensor *q = tensor_or_none(a[2], "q"), *k = tensor_or_none(a[3], "k");
    const at::Tensor *qo = tensor_or_none(a[5], "q_out"), *ko = tensor_or_none(a[6], "k_out");
    if (!q && !k) throw Refused("q or k is required");
    if ((q != nullptr) != (qo != nullptr) || (k != nullptr) != (ko != nullptr))
      throw Refused("q and q_out, k and k_out come together");
    const int dev = device_of(q ? *q : *k);
    const at::ScalarType type = scalar_type(p.dtype);
    Arg x[4];
    const at::Tensor* t[4] = {q, k, qo, ko};
    const char* names[4] = {"q", "k", "q_out", "k_out"};
    for (int i = 0; i < 4; ++i) {
      if (!t[i]) continue;
      const int64_t heads = i % 2 == 0 || p.N_kv == 0 ? p.N : p.N_kv;
      if (p.layout == SWA_LAYOUT_BNSD) {
        const int64_t shape[4] = {p.B, heads, p.S, p.D};
        x[i] = arg(*t[i], names[i], shape, type, dev);
      } else {
        const int64_t shape[3] = {p.B * p.S, heads, p.D};
        x[i] = arg(*t[i], names[i], shape, type, dev);
      }
    }
    const int32_t* pos = positions(tensor(a[4], "positions"), p.n_axes, p.B * p.S, dev);
    const On on(dev, a[7]);
    return unlocked(fn, &p, x[0].ptr, x[0].strides(), x[1].ptr, x[1].strides(), pos, x[2].ptr, x[2].strides(),
                    x[3].ptr, x[3].strides(), on.stream);
  });
}

// paged_append(fn, params, k, v, k_pages, v_pages, block_table, kv_lens, rope params or 0, positions, q, q_out,
//              workspace, stream, k_exponents, v_exponents)
PyObject* bind_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> swa_status_t {
    const auto fn = address<decltype(&swa_paged_append_ext)>(a[0], "entry point");
    const swa_paged_params_t& p = *address<const swa_paged_params_t*>(a[1], "parameters");
    const auto* rope = address<const swa_rope_params_t*>(a[8], "rope");
    const at::Tensor& k = tensor(a[2], "k");
    const int dev = device_of(k);
    const at::ScalarType type = scalar_type(p.dtype);
    const int64_t kv[3] = {p.T_q, p.N_kv ? p.N_kv : p.N, p.D}, qs[3] = {p.T_q, p.N, p.D}, lens[1] = {p.B};
    const Arg xk = arg(k, "k", kv, type, dev), xv = arg(tensor(a[3], "v"), "v", kv, type, dev);
    const Pages kp = pages(tensor(a[4], "k_pages"), "k_pages", p, page_type(p), dev);
    const Pages vp = pages(tensor(a[5], "v_pages"), "v_pages", p, page_type(p), dev);
    int8_t* const ke = exponents(a[14], "k_exponents", p, dev);
    int8_t* const ve = exponents(a[15], "v_exponents", p, dev);
    int64_t row;
    const int32_t* table = block_table(tensor(a[6], "block_table"), p, dev, &row);
    const at::Tensor& l = tensor(a[7], "kv_lens");
    expect_dense(l, "kv_lens", lens, at::kInt, dev);
    const at::Tensor *pos = tensor_or_none(a[9], "positions"), *q = tensor_or_none(a[10], "q");
    const at::Tensor* qo = tensor_or_none(a[11], "q_out");
    if (pos && !rope) throw Refused("positions are taken with rope only");
    const int32_t* pp = pos ? positions(*pos, rope->n_axes, rope->B * rope->S, dev) : nullptr;
    Arg xq, xo;
    if (q) xq = arg(*q, "q", qs, type, dev);
    if (qo) xo = arg(*qo, "q_out", qs, type, dev);
    const at::Tensor& ws = workspace(a[12], dev);
    const On on(dev, a[13]);
    return unlocked(fn, &p, xk.ptr, xk.strides(), xv.ptr, xv.strides(), kp.ptr, kp.strides(), vp.ptr, vp.strides(), ke, ve,
                    table, row, static_cast<const int32_t*>(l.data_ptr()), rope, pp, xq.ptr, xq.strides(), xo.ptr, xo.strides(),
                    ws.data_ptr(), ws.nbytes(), on.stream);
  });
}

// paged_forward(fn, params, q, k_pages, v_pages, block_table, kv_lens, out, softmax_max, softmax_sum, workspace, stream,
//               k_exponents, v_exponents, tree, depth)
PyObject* bind_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> swa_status_t {
    const auto fn = address<decltype(&swa_paged_forward_ext)>(a[0], "entry point");
    const swa_paged_params_t& p = *address<const swa_paged_params_t*>(a[1], "parameters");
    const at::Tensor& q = tensor(a[2], "q");
    const int dev = device_of(q);
    const at::ScalarType type = scalar_type(p.dtype);
    const int64_t qs[3] = {p.T_q, p.N, p.D}, stats[2] = {p.T_q, p.N}, lens[1] = {p.B};
    const Arg xq = arg(q, "q", qs, type, dev);
    const Pages kp = pages(tensor(a[3], "k_pages"), "k_pages", p, page_type(p), dev);
    const Pages vp = pages(tensor(a[4], "v_pages"), "v_pages", p, page_type(p), dev);
    swa_paged_extra_t extra{};
    extra.k_exponents = exponents(a[12], "k_exponents", p, dev);
    extra.v_exponents = exponents(a[13], "v_exponents", p, dev);
    if (const at::Tensor* t = tensor_or_none(a[14], "tree")) extra.tree = tree_rows(*t, p, dev, &extra.tree_stride);
    if (const at::Tensor* t = tensor_or_none(a[15], "depth")) {
      const int64_t tokens[1] = {p.T_q};
      expect_dense(*t, "depth", tokens, at::kInt, dev);
      extra.depth = static_cast<const int32_t*>(t->data_ptr());
    }
    int64_t row;
    const int32_t* table = block_table(tensor(a[5], "block_table"), p, dev, &row);
    const at::Tensor& l = tensor(a[6], "kv_lens");
    expect_dense(l, "kv_lens", lens, at::kInt, dev);
    const at::Tensor &out = tensor(a[7], "out"), &sm = tensor(a[8], "softmax_max"), &ss = tensor(a[9], "softmax_sum");
    expect_dense(out, "out", qs, type, dev);
    expect_dense(sm, "softmax_max", stats, at::kFloat, dev);
    expect_dense(ss, "softmax_sum", stats, at::kFloat, dev);
    const at::Tensor& ws = workspace(a[10], dev);
    const On on(dev, a[11]);
    return unlocked(fn, &p, xq.ptr, xq.strides(), kp.ptr, kp.strides(), vp.ptr, vp.strides(),
                    static_cast<const swa_paged_extra_t*>(&extra), table, row,
                    static_cast<const int32_t*>(l.data_ptr()), out.data_ptr(), static_cast<float*>(sm.data_ptr()),
                    static_cast<float*>(ss.data_ptr()), ws.data_ptr(), ws.nbytes(), on.stream);
  });
}

// paged_gather(fn, params, k_pages, v_pages, block_table, kv_lens, k, v, workspace, stream, k_exponents, v_exponents)
PyObject* bind_gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> swa_status_t {
    const auto fn = address<decltype(&swa_paged_gather)>(a[0], "entry point");
    const swa_paged_params_t& p = *address<const swa_paged_params_t*>(a[1], "parameters");
    const at::Tensor& k = tensor(a[6], "k");
    const int dev = device_of(k);
    const at::ScalarType type = scalar_type(p.dtype);
    const int64_t kv[3] = {p.T_q, p.N_kv ? p.N_kv : p.N, p.D}, lens[1] = {p.B};
    const Arg xk = arg(k, "k", kv, type, dev), xv = arg(tensor(a[7], "v"), "v", kv, type, dev);
    const Pages kp = pages(tensor(a[2], "k_pages"), "k_pages", p, page_type(p), dev);
    const Pages vp = pages(tensor(a[3], "v_pages"), "v_pages", p, page_type(p), dev);
    int8_t* const ke = exponents(a[10], "k_exponents", p, dev);
    int8_t* const ve = exponents(a[11], "v_exponents", p, dev);
    int64_t row;
    const int32_t* table = block_table(tensor(a[4], "block_table"), p, dev, &row);
    const at::Tensor& l = tensor(a[5], "kv_lens");
    expect_dense(l, "kv_lens", lens, at::kInt, dev);
    const at::Tensor& ws = workspace(a[8], dev);
    const On on(dev, a[9]);
    return unlocked(fn, &p, kp.ptr, kp.strides(), vp.ptr, vp.strides(), ke, ve, table, row,
                    static_cast<const int32_t*>(l.data_ptr()), xk.ptr, xk.strides(), xv.ptr, xv.strides(), ws.data_ptr(),
                    ws.nbytes(), on.stream);
  });
}

PyMethodDef methods[] = {
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_rope)), METH_FASTCALL, nullptr},
    {"paged_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_append)), METH_FASTCALL, nullptr},
    {"paged_forward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_forward)), METH_FASTCALL,
     nullptr},
    {"paged_gather", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind_gather)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_swa_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__swa_bind() { return PyModule_Create(&module); }
