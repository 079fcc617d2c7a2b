// The layer operators' Python calls: arguments are checked and handed to the C interface.
//
// A decode step makes these calls for 4 to 9 us of GPU work each. Marshalled in Python, the
// dozen tensors of a call (each looked at for shape, type, device and strides) and its thirty
// C arguments took 8 to 14 us of the host's time, more than the kernels.
//
// Tensors stay the caller's; nothing is kept from one call for the next but what bind() gives.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/StreamGuard.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/Stream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <climits>
#include <cmath>
#include <cstring>
#include <utility>

#include "fp8gemm.h"
#include "fp8layer.h"

namespace {

using at::Device;
using at::ScalarType;
using at::Tensor;

struct Library {
  decltype(&fp8_rmsnorm_quantize_1x128) norm;
  decltype(&fp8_rmsnorm_backward) norm_grad;
  decltype(&fp8_rmsnorm_backward_workspace_size) norm_grad_workspace;
  decltype(&fp8_rope_append_paged_kv) append;
  decltype(&fp8_paged_attention) attend;
  decltype(&fp8_gemm_scale_ld) scale_ld;
  PyObject* check;            // check(status, name) raises
  PyObject* current_stream;   // current_stream(device index): its raw handle
  PyObject* external_stream;  // external_stream(raw handle, device index): a torch stream
} library;

// ----------------------------------------------------------------------------- arguments

bool given(PyObject* o) { return o != Py_None; }

const Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}
const Tensor& gpu_tensor(PyObject* o, const char* name, int64_t dims) {
  const Tensor& t = tensor(o, name);
  TORCH_CHECK_VALUE(t.is_cuda() && t.dim() == dims, name, " must be a ", dims, "-D GPU tensor");
  return t;
}

int to_int(int64_t n, const char* name) {
  TORCH_CHECK_VALUE(n >= INT_MIN && n <= INT_MAX, name, " does not fit 32 bits");
  return (int)n;
}
int to_int(PyObject* o, const char* name) {
  const long long n = PyLong_AsLongLong(o);
  if (n == -1 && PyErr_Occurred()) throw python_error();
  return to_int(n, name);
}
float to_float(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)x;
}

bool rows_type(const Tensor& t) { return t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kFloat; }
int type_code(const Tensor& t) { return t.scalar_type() == at::kBFloat16 ? FP8GEMM_QUANT_BF16 : FP8GEMM_QUANT_FP32; }
bool codes_type(const Tensor& t) { return t.scalar_type() == at::kByte || t.scalar_type() == at::kFloat8_e4m3fn; }

// Row stride of a matrix; a single row may carry any.
int64_t row_stride(const Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

// Row stride of a tensor that must be `type` [M, K] with a unit inner stride.
int64_t matrix(const Tensor& t, const char* name, int64_t M, int64_t K, ScalarType type, Device dev) {
  TORCH_CHECK_VALUE(t.dim() == 2 && t.size(0) == M && t.size(1) == K && t.scalar_type() == type && t.device() == dev && t.stride(1) == 1,
                    name, " must be ", type, " [", M, ", ", K, "] on ", dev, " with a unit inner stride");
  return row_stride(t);
}
// Row stride of a tensor that must be BF16 [T, H, D] with contiguous rows.
int64_t heads(const Tensor& t, const char* name, int64_t T, int64_t H, int64_t D, Device dev) {
  TORCH_CHECK_VALUE(t.dim() == 3 && t.size(0) == T && t.size(1) == H && t.size(2) == D && t.scalar_type() == at::kBFloat16 &&
                        t.device() == dev && t.stride(2) == 1 && (H <= 1 || t.stride(1) == D),
                    name, " must be bfloat16 [", T, ", ", H, ", ", D, "] on ", dev, " with contiguous rows");
  return T > 1 ? t.stride(0) : H * D;
}
// Address of a tensor that must be contiguous `type` [n].
void* vector(const Tensor& t, const char* name, int64_t n, ScalarType type, Device dev) {
  TORCH_CHECK_VALUE(t.dim() == 1 && t.size(0) == n && t.scalar_type() == type && t.device() == dev && (n <= 1 || t.stride(0) == 1), name,
                    " must be contiguous ", type, " [", n, "] on ", dev);
  return t.data_ptr();
}
void* weight(const Tensor& t, int64_t K, Device dev) {
  return vector(t, "weight", K, t.scalar_type() == at::kBFloat16 ? at::kBFloat16 : at::kFloat, dev);
}

// The stream that a call runs on. While this lives it is the current one, so that what the call
// allocates is not memory on which earlier work of the caller's stream is still queued.
class Launch {
 public:
  Launch(PyObject* stream, Device dev) : dev_(dev) {
    THPObjectPtr index(PyLong_FromLong(dev.index()));
    if (!index) throw python_error();
    THPObjectPtr raw(given(stream) ? PyObject_GetAttrString(stream, "cuda_stream")
                                   : PyObject_CallFunctionObjArgs(library.current_stream, index.get(), nullptr));
    if (!raw) throw python_error();
    void* const p = PyLong_AsVoidPtr(raw);
    if (!p && PyErr_Occurred()) throw python_error();
    handle_ = static_cast<hipStream_t>(p);
    if (!given(stream)) return;
    THPObjectPtr made;  // of an object that has only the handle
    if (!THPStream_Check(stream)) {
      made = PyObject_CallFunctionObjArgs(library.external_stream, raw.get(), index.get(), nullptr);
      if (!made) throw python_error();
      stream = made;
    }
    const auto* const s = reinterpret_cast<const THPStream*>(stream);
    const auto to =
        c10::Stream::unpack3(s->stream_id, (c10::DeviceIndex)s->device_index, static_cast<c10::DeviceType>(s->device_type));
    TORCH_CHECK_VALUE(to.device() == dev, "stream must be one of ", dev);
    if (to != c10::impl::VirtualGuardImpl(dev.type()).getStream(dev)) guard_.reset_stream(to);
  }

  hipStream_t handle() const { return handle_; }

  Tensor scratch(at::IntArrayRef shape, ScalarType type) const {
    return at::empty(shape, at::TensorOptions().dtype(type).device(dev_));
  }
  // The tensor that was given, or a new one. The caller will use it on its own stream.
  Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, ScalarType type) const {
    if (given(o)) return tensor(o, name);
    Tensor t = scratch(shape, type);
    if (const auto caller = guard_.original_stream()) t.record_stream(*caller);
    return t;
  }

 private:
  Device dev_;
  hipStream_t handle_;
  c10::OptionalStreamGuard guard_;
};

// Calls the library without Python's lock (a full queue makes a launch wait).
template <typename F>
void call(const char* name, F f) {
  int status;
  Py_BEGIN_ALLOW_THREADS status = f();
  Py_END_ALLOW_THREADS
  if (status != FP8GEMM_OK) {
    PyObject* r = PyObject_CallFunction(library.check, "is", status, name);
    Py_XDECREF(r);
    throw python_error();
  }
}

void arguments(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n); }

// Of a paged cache.
struct Cache {
  Tensor k, k_scale, v, v_scale;
  int num_pages, heads, page, dim;
};
Cache cache_of(PyObject* o, Device dev) {
  TORCH_CHECK_TYPE(PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 4, "cache must be a PagedKVCache");
  Cache c;
  c.k = tensor(PyTuple_GET_ITEM(o, 0), "cache.k"), c.k_scale = tensor(PyTuple_GET_ITEM(o, 1), "cache.k_scale");
  c.v = tensor(PyTuple_GET_ITEM(o, 2), "cache.v"), c.v_scale = tensor(PyTuple_GET_ITEM(o, 3), "cache.v_scale");
  for (const Tensor* t : {&c.k, &c.v})
    TORCH_CHECK_VALUE(t->dim() == 4 && t->sizes() == c.k.sizes() && codes_type(*t) && t->is_contiguous() && t->device() == dev,
                      "cache codes must be contiguous uint8 or float8_e4m3fn [num_pages, Hkv, page_size, D] on ", dev,
                      ", keys and values alike");
  for (const Tensor* t : {&c.k_scale, &c.v_scale})
    TORCH_CHECK_VALUE(t->dim() == 2 && t->size(0) == c.k.size(0) && t->size(1) == c.k.size(1) && t->scalar_type() == at::kFloat &&
                          t->is_contiguous() && t->device() == dev,
                      "cache scales must be contiguous float32 [num_pages, Hkv] on ", dev);
  c.num_pages = to_int(c.k.size(0), "num_pages"), c.heads = to_int(c.k.size(1), "Hkv");
  c.page = to_int(c.k.size(2), "page_size"), c.dim = to_int(c.k.size(3), "D");
  return c;
}

// Of the sequences of a call.
struct Sequences {
  const int32_t *table, *lens, *cu;
  int64_t stride;
  int count, pages;
};
Sequences sequences(PyObject* block_table, PyObject* seq_lens, PyObject* cu_q, Device dev) {
  const Tensor &table = tensor(block_table, "block_table"), &lens = tensor(seq_lens, "seq_lens"), &cu = tensor(cu_q, "cu_q");
  TORCH_CHECK_VALUE(lens.dim() == 1, "seq_lens must be int32 [B]");
  const int64_t B = lens.size(0);
  TORCH_CHECK_VALUE(table.dim() == 2 && table.size(0) == B && table.scalar_type() == at::kInt && table.device() == dev &&
                        (table.size(1) <= 1 || table.stride(1) == 1),
                    "block_table must be int32 [", B, ", max_pages] on ", dev, " with a unit inner stride");
  return {static_cast<const int32_t*>(table.data_ptr()),
          static_cast<const int32_t*>(vector(lens, "seq_lens", B, at::kInt, dev)),
          static_cast<const int32_t*>(vector(cu, "cu_q", B + 1, at::kInt, dev)),
          row_stride(table),
          to_int(B, "B"),
          to_int(table.size(1), "max_pages")};
}

// M x K rows that a norm call is about.
void norm_rows(const Tensor& t, const char* name) {
  TORCH_CHECK_VALUE(t.stride(1) == 1 && rows_type(t) && t.size(1) % 128 == 0, name,
                    " must be a 2-D bfloat16 or float32 GPU tensor with a unit inner stride and a multiple of 128 columns");
}

// ----------------------------------------------------------------------------- operators

// X, weight, residual, eps, Q, sa, H, rstd, Y, stream -> (Q, sa, H, rstd)
PyObject* rmsnorm_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 10);
  const Tensor& X = gpu_tensor(a[0], "X", 2);
  norm_rows(X, "X");
  const Device dev = X.device();
  const c10::DeviceGuard guard(dev);
  const Launch launch(a[9], dev);
  const int64_t M = X.size(0), K = X.size(1);
  const Tensor& w = tensor(a[1], "weight");
  void* const wp = weight(w, K, dev);
  const void* r = nullptr;
  void *h = nullptr, *y = nullptr;
  int64_t ldr = 0, ldh = 0, ldy = 0;
  Tensor H = X;
  if (given(a[2])) {
    const Tensor& R = tensor(a[2], "residual");
    ldr = matrix(R, "residual", M, K, X.scalar_type(), dev), r = R.data_ptr();
    H = launch.output(a[6], "H", {M, K}, X.scalar_type());
    ldh = matrix(H, "H", M, K, X.scalar_type(), dev), h = H.data_ptr();
  } else {
    TORCH_CHECK_VALUE(!given(a[6]) || a[6] == a[0], "H is written only with a residual");
  }
  const Tensor Q = launch.output(a[4], "Q", {M, K}, at::kByte);
  const Tensor sa = launch.output(a[5], "sa", {K / 128, given(a[5]) ? 0 : library.scale_ld(to_int(M, "M"))}, at::kFloat);
  const Tensor rstd = launch.output(a[7], "rstd", {M}, at::kFloat);
  const int64_t ldq = matrix(Q, "Q", M, K, codes_type(Q) ? Q.scalar_type() : at::kByte, dev);
  TORCH_CHECK_VALUE(sa.scalar_type() == at::kFloat && sa.dim() == 2 && sa.size(0) == K / 128 && sa.size(1) >= M && sa.stride(1) == 1 &&
                        sa.device() == dev,
                    "sa must be float32 [", K / 128, ", >= ", M, "] on ", dev, " with a unit inner stride");
  if (given(a[8])) {
    const Tensor& Y = tensor(a[8], "Y");
    ldy = matrix(Y, "Y", M, K, at::kBFloat16, dev), y = Y.data_ptr();
  }
  const float eps = to_float(a[3]);
  const int rows = to_int(M, "M"), cols = to_int(K, "K");
  auto* const rstd_p = static_cast<float*>(vector(rstd, "rstd", M, at::kFloat, dev));
  call("fp8_rmsnorm_quantize_1x128", [&] {
    return library.norm(X.data_ptr(), row_stride(X), r, ldr, type_code(X), wp, type_code(w), eps, h, ldh, y, ldy, rstd_p, Q.data_ptr(), ldq,
                        static_cast<float*>(sa.data_ptr()), sa.size(0) > 1 ? sa.stride(0) : library.scale_ld(sa.size(1)), rows, cols,
                        launch.handle());
  });
  return Py_BuildValue("NNNN", THPVariable_Wrap(Q), THPVariable_Wrap(sa), THPVariable_Wrap(H), THPVariable_Wrap(rstd));
  END_HANDLE_TH_ERRORS
}

// dY, H, rstd, weight, dH, dX, dW, workspace, stream -> (dX, dW)
PyObject* rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 9);
  const Tensor& dY = gpu_tensor(a[0], "dY", 2);
  norm_rows(dY, "dY");
  const Device dev = dY.device();
  const c10::DeviceGuard guard(dev);
  const Launch launch(a[8], dev);
  const int64_t M = dY.size(0), K = dY.size(1);
  const ScalarType type = dY.scalar_type();
  const Tensor &H = tensor(a[1], "H"), &rstd = tensor(a[2], "rstd"), &w = tensor(a[3], "weight");
  const int64_t ldh = matrix(H, "H", M, K, type, dev);
  void* const wp = weight(w, K, dev);
  auto* const rstd_p = static_cast<const float*>(vector(rstd, "rstd", M, at::kFloat, dev));
  const void* dh = nullptr;
  int64_t lddh = 0;
  if (given(a[4])) {
    const Tensor& dH = tensor(a[4], "dH");
    lddh = matrix(dH, "dH", M, K, type, dev), dh = dH.data_ptr();
  }
  const Tensor dX = launch.output(a[5], "dX", {M, K}, type);
  const int64_t lddx = matrix(dX, "dX", M, K, type, dev);
  const Tensor dW = launch.output(a[6], "dW", {K}, at::kFloat);
  auto* const dw = static_cast<float*>(vector(dW, "dW", K, at::kFloat, dev));
  const int rows = to_int(M, "M"), cols = to_int(K, "K");
  const Tensor ws =
      given(a[7]) ? tensor(a[7], "workspace") : launch.scratch({(int64_t)library.norm_grad_workspace(rows, cols)}, at::kByte);
  TORCH_CHECK_VALUE(ws.device() == dev && ws.is_contiguous(), "workspace must be contiguous on dY's device");
  call("fp8_rmsnorm_backward", [&] {
    return library.norm_grad(dY.data_ptr(), row_stride(dY), H.data_ptr(), ldh, dh, lddh, type_code(dY), rstd_p, wp, type_code(w),
                             dX.data_ptr(), lddx, dw, rows, cols, ws.data_ptr(), ws.nbytes(), launch.handle());
  });
  return Py_BuildValue("NN", THPVariable_Wrap(dX), THPVariable_Wrap(dW));
  END_HANDLE_TH_ERRORS
}

// q, k, v, cos_sin, cache, block_table, seq_lens, cu_q, positions, interleaved, q_out, stream -> q_out
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 12);
  const Tensor& k = gpu_tensor(a[1], "k", 3);
  const Device dev = k.device();
  const c10::DeviceGuard guard(dev);
  const Launch launch(a[11], dev);
  const int64_t T = k.size(0), Hkv = k.size(1), D = k.size(2);
  const Cache c = cache_of(a[4], dev);
  TORCH_CHECK_VALUE(c.heads == Hkv && c.dim == D, "the cache has other heads than k");
  const Tensor& v = tensor(a[2], "v");
  const int64_t ldk = heads(k, "k", T, Hkv, D, dev), ldv = heads(v, "v", T, Hkv, D, dev);
  int64_t Hq = Hkv, ldq = 0, ldqo = 0;
  const void* q = nullptr;
  void* qo = nullptr;
  Tensor q_out;
  if (given(a[0])) {
    const Tensor& Q = gpu_tensor(a[0], "q", 3);
    Hq = Q.size(1);
    ldq = heads(Q, "q", T, Hq, D, dev), q = Q.data_ptr();
    q_out = launch.output(a[10], "q_out", {T, Hq, D}, at::kBFloat16);
    ldqo = heads(q_out, "q_out", T, Hq, D, dev), qo = q_out.data_ptr();
  } else {
    TORCH_CHECK_VALUE(!given(a[10]), "q_out without q");
  }
  const float* table = nullptr;
  int max_pos = 0, rot_dim = 0;
  int64_t ld_cs = 0;
  if (given(a[3])) {
    const Tensor& t = tensor(a[3], "cos_sin");
    TORCH_CHECK_VALUE(t.scalar_type() == at::kFloat && t.dim() == 2 && t.device() == dev && t.stride(1) == 1,
                      "cos_sin must be float32 [max_pos, rot_dim] on ", dev, " with a unit inner stride");
    table = static_cast<const float*>(t.data_ptr());
    max_pos = to_int(t.size(0), "max_pos"), rot_dim = to_int(t.size(1), "rot_dim"), ld_cs = row_stride(t);
  }
  const Sequences s = sequences(a[5], a[6], a[7], dev);
  const int32_t* positions = nullptr;
  if (given(a[8])) positions = static_cast<const int32_t*>(vector(tensor(a[8], "positions"), "positions", T, at::kInt, dev));
  const int interleaved = PyObject_IsTrue(a[9]);
  if (interleaved < 0) throw python_error();
  const int tokens = to_int(T, "T"), q_heads = to_int(Hq, "Hq");
  call("fp8_rope_append_paged_kv", [&] {
    return library.append(q, ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, table, ld_cs, max_pos, rot_dim, interleaved, positions, s.table,
                          s.stride, s.pages, s.lens, s.cu, qo, ldqo, c.k.data_ptr(), static_cast<float*>(c.k_scale.data_ptr()),
                          c.v.data_ptr(), static_cast<float*>(c.v_scale.data_ptr()), c.num_pages, c.page, s.count, tokens, q_heads,
                          c.heads, c.dim, launch.handle());
  });
  if (!q_out.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(q_out);
  END_HANDLE_TH_ERRORS
}

// q, cache, block_table, seq_lens, cu_q, out, lse, softmax_scale (None: D^-1/2), window, workspace, stream -> out
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 11);
  const Tensor& q = gpu_tensor(a[0], "q", 3);
  const Device dev = q.device();
  const c10::DeviceGuard guard(dev);
  const Launch launch(a[10], dev);
  const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
  const Cache c = cache_of(a[1], dev);
  TORCH_CHECK_VALUE(c.dim == D && c.heads != 0 && Hq % c.heads == 0, "q's heads do not match the cache's");
  const int64_t ldq = heads(q, "q", T, Hq, D, dev);
  const Tensor out = launch.output(a[5], "out", {T, Hq, D}, at::kBFloat16);
  const int64_t ldo = heads(out, "out", T, Hq, D, dev);
  float* lse = nullptr;
  if (given(a[6])) {
    const Tensor& t = tensor(a[6], "lse");
    TORCH_CHECK_VALUE(t.scalar_type() == at::kFloat && t.dim() == 2 && t.size(0) == T && t.size(1) == Hq && t.is_contiguous() &&
                          t.device() == dev,
                      "lse must be contiguous float32 [", T, ", ", Hq, "] on ", dev);
    lse = static_cast<float*>(t.data_ptr());
  }
  const Sequences s = sequences(a[2], a[3], a[4], dev);
  void* ws = nullptr;
  size_t ws_bytes = 0;
  if (given(a[9])) {
    const Tensor& t = tensor(a[9], "workspace");
    TORCH_CHECK_VALUE(t.device() == dev && t.is_contiguous(), "workspace must be contiguous on q's device");
    ws = t.data_ptr(), ws_bytes = t.nbytes();
  }
  const float scale = given(a[7]) ? to_float(a[7]) : (float)(1.0 / std::sqrt((double)D));
  const int window = to_int(a[8], "window"), tokens = to_int(T, "T"), q_heads = to_int(Hq, "Hq");
  call("fp8_paged_attention", [&] {
    return library.attend(q.data_ptr(), ldq, c.k.data_ptr(), static_cast<const float*>(c.k_scale.data_ptr()), c.v.data_ptr(),
                          static_cast<const float*>(c.v_scale.data_ptr()), c.num_pages, c.page, s.table, s.stride, s.pages, s.lens, s.cu,
                          out.data_ptr(), ldo, lse, scale, window, s.count, tokens, q_heads, c.heads, c.dim, ws, ws_bytes,
                          launch.handle());
  });
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// Sets f to the address that a dict has under `name`.
template <typename F>
void set_address(PyObject* dict, F& f, const char* name) {
  TORCH_CHECK_TYPE(PyDict_Check(dict), "expected a dict of addresses");
  PyObject* at = PyDict_GetItemString(dict, name);
  TORCH_CHECK_VALUE(at != nullptr, "no address of ", name);
  f = reinterpret_cast<F>(PyLong_AsVoidPtr(at));
  if (!f) throw python_error();
}

}  // namespace

#include "../csrc_moe/binding_moe.hpp"

namespace {

// The library's functions as a dict of addresses by name, check, current_stream, external_stream
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 4);
  set_address(a[0], library.norm, "fp8_rmsnorm_quantize_1x128");
  set_address(a[0], library.norm_grad, "fp8_rmsnorm_backward");
  set_address(a[0], library.norm_grad_workspace, "fp8_rmsnorm_backward_workspace_size");
  set_address(a[0], library.append, "fp8_rope_append_paged_kv");
  set_address(a[0], library.attend, "fp8_paged_attention");
  set_address(a[0], library.scale_ld, "fp8_gemm_scale_ld");
  Py_INCREF(a[1]), Py_INCREF(a[2]), Py_INCREF(a[3]);
  library.check = a[1], library.current_stream = a[2], library.external_stream = a[3];
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {
    {"bind", fast(bind), METH_FASTCALL, nullptr},
    {"rmsnorm_quantize", fast(rmsnorm_quantize), METH_FASTCALL, nullptr},
    {"rmsnorm_backward", fast(rmsnorm_backward), METH_FASTCALL, nullptr},
    {"rope_append", fast(rope_append), METH_FASTCALL, nullptr},
    {"attend", fast(attend), METH_FASTCALL, nullptr},
    {"bind_moe", fast(bind_moe), METH_FASTCALL, nullptr},
    {"moe_route", fast(moe_route), METH_FASTCALL, nullptr},
    {"moe_route_backward", fast(moe_route_backward), METH_FASTCALL, nullptr},
    {"moe_dispatch", fast(moe_dispatch), METH_FASTCALL, nullptr},
    {"moe_gather", fast(moe_gather), METH_FASTCALL, nullptr},
    {"moe_combine", fast(moe_combine), METH_FASTCALL, nullptr},
    {"moe_combine_backward", fast(moe_combine_backward), METH_FASTCALL, nullptr},
    {"qk_norm_rope", fast(qk_norm_rope), METH_FASTCALL, nullptr},
    {"qk_norm_rope_backward", fast(qk_norm_rope_backward), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer_call() { return PyModule_Create(&module); }
