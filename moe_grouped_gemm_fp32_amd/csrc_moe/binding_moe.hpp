// The expert and head operators' Python calls: part of binding.cpp, whose helpers they use.
#pragma once

#include "fp8moe.h"

namespace {

struct MoeLibrary {
  decltype(&fp8_moe_route) route;
  decltype(&fp8_moe_route_backward) route_grad;
  decltype(&fp8_moe_rows) rows;
  decltype(&fp8_moe_dispatch) dispatch;
  decltype(&fp8_moe_dispatch_workspace_size) dispatch_workspace;
  decltype(&fp8_moe_gather) gather;
  decltype(&fp8_moe_combine) combine;
  decltype(&fp8_moe_combine_backward) combine_grad;
  decltype(&fp8_qk_norm_rope) heads;
  decltype(&fp8_qk_norm_rope_backward) heads_grad;
  decltype(&fp8_qk_norm_rope_backward_workspace_size) heads_workspace;
} moe;

bool to_bool(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}
// Address of a tensor that must be contiguous `type` [M, K].
void* table(const Tensor& t, const char* name, int64_t M, int64_t K, ScalarType type, Device dev) {
  TORCH_CHECK_VALUE(t.dim() == 2 && t.size(0) == M && t.size(1) == K && t.scalar_type() == type && t.device() == dev && t.is_contiguous(),
                    name, " must be contiguous ", type, " [", M, ", ", K, "] on ", dev);
  return t.data_ptr();
}
// A matrix of rows in BF16 or FP32 with a unit inner stride.
const Tensor& rows_of(PyObject* o, const char* name) {
  const Tensor& t = gpu_tensor(o, name, 2);
  TORCH_CHECK_VALUE(rows_type(t) && (t.size(1) <= 1 || t.stride(1) == 1), name,
                    " must be a 2-D bfloat16 or float32 GPU tensor with a unit inner stride");
  return t;
}
int scoring_of(PyObject* o) {
  const char* s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
  if (!s && PyErr_Occurred()) throw python_error();
  const bool sigmoid = s && std::strcmp(s, "sigmoid") == 0;
  TORCH_CHECK_VALUE(sigmoid || (s && std::strcmp(s, "softmax") == 0), "scoring must be 'softmax' or 'sigmoid'");
  return sigmoid ? FP8MOE_SIGMOID : FP8MOE_SOFTMAX;
}

// logits, top_k, bias, scoring, groups, top_groups, group_best, renormalize, scale, ids, weights, scores, stream -> (ids, weights)
PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 13);
  const Tensor& x = rows_of(a[0], "logits");
  const Device dev = x.device();
  const c10::DeviceGuard guard(dev);
  const Launch launch(a[12], dev);
  const int64_t T = x.size(0), E = x.size(1);
  const int k = to_int(a[1], "top_k"), tokens = to_int(T, "T"), experts = to_int(E, "E");
  TORCH_CHECK_VALUE(k >= 1 && k <= E, "top_k must be 1 to ", E);
  const float* bias = given(a[2]) ? static_cast<const float*>(vector(tensor(a[2], "bias"), "bias", E, at::kFloat, dev)) : nullptr;
  const int scoring = scoring_of(a[3]), groups = to_int(a[4], "groups"), top_groups = to_int(a[5], "top_groups");
  const int best = to_int(a[6], "group_best");
  const bool renormalize = to_bool(a[7]);
  const float scale = to_float(a[8]);
  const Tensor ids = launch.output(a[9], "ids", {T, k}, at::kInt), w = launch.output(a[10], "weights", {T, k}, at::kFloat);
  auto* const ids_p = static_cast<int32_t*>(table(ids, "ids", T, k, at::kInt, dev));
  auto* const w_p = static_cast<float*>(table(w, "weights", T, k, at::kFloat, dev));
  float* scores = nullptr;
  int64_t lds = 0;
  if (given(a[11])) {
    const Tensor& s = tensor(a[11], "scores");
    lds = matrix(s, "scores", T, E, at::kFloat, dev), scores = static_cast<float*>(s.data_ptr());
  }
  call("fp8_moe_route", [&] {
    return moe.route(x.data_ptr(), row_stride(x), type_code(x), bias, scoring, groups, top_groups, best, renormalize, scale, ids_p, w_p,
                     scores, lds, tokens, experts, k, launch.handle());
  });
  return Py_BuildValue("NN", THPVariable_Wrap(ids), THPVariable_Wrap(w));
  END_HANDLE_TH_ERRORS
}

// dweights, logits, ids, scoring, renormalize, scale, dscores, dlogits, stream -> dlogits
PyObject* moe_route_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 9);
  const Tensor& x = rows_of(a[1], "logits");
  const Device dev = x.device();
  const c10::DeviceGuard guard(dev);
  const Launch launch(a[8], dev);
  const int64_t T = x.size(0), E = x.size(1);
  const Tensor& ids = gpu_tensor(a[2], "ids", 2);
  const int k = to_int(ids.size(1), "top_k"), tokens = to_int(T, "T"), experts = to_int(E, "E");
  auto* const ids_p = static_cast<const int32_t*>(table(ids, "ids", T, k, at::kInt, dev));
  auto* const dw = static_cast<const float*>(table(tensor(a[0], "dweights"), "dweights", T, k, at::kFloat, dev));
  const int scoring = scoring_of(a[3]);
  const bool renormalize = to_bool(a[4]);
  const float scale = to_float(a[5]);
  const float* ds = nullptr;
  int64_t ldds = 0;
  if (given(a[6])) {
    const Tensor& s = tensor(a[6], "dscores");
    ldds = matrix(s, "dscores", T, E, at::kFloat, dev), ds = static_cast<const float*>(s.data_ptr());
  }
  const Tensor dx = launch.output(a[7], "dlogits", {T, E}, x.scalar_type());
  const int64_t lddx = matrix(dx, "dlogits", T, E, x.scalar_type(), dev);
  call("fp8_moe_route_backward", [&] {
    return moe.route_grad(dw, x.data_ptr(), row_stride(x), type_code(x), ids_p, scoring, renormalize, scale, ds, ldds, dx.data_ptr(), lddx,
                          tokens, experts, k, launch.handle());
  });
  return THPVariable_Wrap(dx);
  END_HANDLE_TH_ERRORS
}

// The tensors of a MoeLayout; m_indices is undefined in the masked layout.
struct MoeRows {
  Tensor positions, sources, m_indices, counts;
};
MoeRows layout_of(PyObject* o) {
  TORCH_CHECK_TYPE(PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 4, "layout must be a MoeLayout");
  MoeRows r;
  r.positions = tensor(PyTuple_GET_ITEM(o, 0), "layout.positions"), r.sources = tensor(PyTuple_GET_ITEM(o, 1), "layout.sources");
  if (given(PyTuple_GET_ITEM(o, 2))) r.m_indices = tensor(PyTuple_GET_ITEM(o, 2), "layout.m_indices");
  r.counts = tensor(PyTuple_GET_ITEM(o, 3), "layout.counts");
  return r;
}

// Stride of the rows of a 3-D tensor, which has to be one for all; `alone` for a single row.
int64_t one_stride(const Tensor& t, const char* name, int64_t alone) {
  if (t.size(1) <= 1) return t.size(0) > 1 ? t.stride(0) : alone;
  TORCH_CHECK_VALUE(t.size(0) <= 1 || t.stride(0) == t.size(1) * t.stride(1), name, "'s rows must lie at one stride");
  return t.stride(1);
}

// What a dispatch and a gather have in common: the tokens' rows, and the expanded ones.
struct MoeCopy {
  Tensor Qx, sax;
  const void* q;
  const float *sa, *weights;
  int64_t ldq, ld_sa, ldqx, ld_sax;
  int cols;
};
MoeCopy copy_of(const Launch& launch, const Tensor& Q, PyObject* sa_o, PyObject* weights, PyObject* Qx_o, PyObject* sax_o, int64_t T, int64_t k,
                int64_t E, int64_t rows, int64_t max_m, Device dev) {
  const int64_t K = Q.size(1), blocks = K / 128;
  TORCH_CHECK_VALUE(codes_type(Q) && K >= 128 && K % 128 == 0 && Q.stride(1) == 1,
                    "Q must be uint8 or float8_e4m3fn [T, K] with a unit inner stride, K a multiple of 128");
  MoeCopy c;
  const Tensor& sa = tensor(sa_o, "sa");
  TORCH_CHECK_VALUE(sa.dim() == 2 && sa.size(0) == blocks && sa.size(1) >= T && sa.scalar_type() == at::kFloat && sa.device() == dev &&
                        (sa.size(1) <= 1 || sa.stride(1) == 1),
                    "sa must be float32 [", blocks, ", >= ", T, "] on ", dev, " with a unit inner stride");
  c.q = Q.data_ptr(), c.ldq = row_stride(Q), c.sa = static_cast<const float*>(sa.data_ptr());
  c.ld_sa = blocks > 1 ? sa.stride(0) : library.scale_ld(sa.size(1));
  c.weights = given(weights) ? static_cast<const float*>(table(tensor(weights, "weights"), "weights", T, k, at::kFloat, dev)) : nullptr;
  c.cols = to_int(K, "K");
  if (max_m) {
    c.Qx = launch.output(Qx_o, "Qx", {E, max_m, K}, at::kByte);
    c.sax = launch.output(sax_o, "sax", {E, blocks, library.scale_ld(max_m)}, at::kFloat);
    TORCH_CHECK_VALUE(c.Qx.dim() == 3 && c.Qx.size(0) == E && c.Qx.size(1) == max_m && c.Qx.size(2) == K && codes_type(c.Qx) &&
                          c.Qx.device() == dev && c.Qx.stride(2) == 1,
                      "Qx must be uint8 or float8_e4m3fn [", E, ", ", max_m, ", ", K, "] on ", dev, " with a unit inner stride");
    c.ldqx = one_stride(c.Qx, "Qx", K);
    TORCH_CHECK_VALUE(c.sax.dim() == 3 && c.sax.size(0) == E && c.sax.size(1) == blocks && c.sax.size(2) >= max_m &&
                          c.sax.scalar_type() == at::kFloat && c.sax.device() == dev && (c.sax.size(2) <= 1 || c.sax.stride(2) == 1),
                      "sax must be float32 [", E, ", ", blocks, ", >= ", max_m, "] on ", dev, " with a unit inner stride");
    c.ld_sax = one_stride(c.sax, "sax", library.scale_ld(c.sax.size(2)));
  } else {
    c.Qx = launch.output(Qx_o, "Qx", {rows, K}, at::kByte);
    c.sax = launch.output(sax_o, "sax", {blocks, library.scale_ld(rows)}, at::kFloat);
    c.ldqx = matrix(c.Qx, "Qx", rows, K, codes_type(c.Qx) ? c.Qx.scalar_type() : at::kByte, dev);
    TORCH_CHECK_VALUE(c.sax.dim() == 2 && c.sax.size(0) == blocks && c.sax.size(1) >= rows && c.sax.scalar_type() == at::kFloat &&
                          c.sax.device() == dev && (c.sax.size(1) <= 1 || c.sax.stride(1) == 1),
                      "sax must be float32 [", blocks, ", >= ", rows, "] on ", dev, " with a unit inner stride");
    c.ld_sax = blocks > 1 ? c.sax.stride(0) : library.scale_ld(c.sax.size(1));
  }
  return c;
}

// Q, sa, ids, num_experts, max_m, weights, Qx, sax, layout, workspace, stream -> (Qx, sax, layout's four tensors)
PyObject* moe_dispatch(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 11);
  const Tensor& Q = gpu_tensor(a[0], "Q", 2);
  const Device dev = Q.device();
  const c10::DeviceGuard guard(dev);
  const Launch launch(a[10], dev);
  const Tensor& ids = tensor(a[2], "ids");
  const int64_t T = Q.size(0);
  TORCH_CHECK_VALUE(ids.dim() == 2, "ids must be int32 [T, top_k]");
  const int64_t k = ids.size(1);
  auto* const ids_p = static_cast<const int32_t*>(table(ids, "ids", T, k, at::kInt, dev));
  const int tokens = to_int(T, "T"), top_k = to_int(k, "top_k"), E = to_int(a[3], "num_experts");
  const int max_m = given(a[4]) ? to_int(a[4], "max_m") : 0;
  TORCH_CHECK_VALUE(E >= 1 && top_k >= 1, "num_experts and top_k must be at least 1");
  TORCH_CHECK_VALUE(!given(a[4]) || max_m >= 1, "max_m must be at least 1");
  MoeRows r;
  int64_t rows;
  if (given(a[8])) {
    r = layout_of(a[8]);
    rows = max_m ? (int64_t)E * max_m : r.sources.numel();
  } else {
    rows = max_m ? (int64_t)E * max_m : moe.rows(tokens, top_k, E);
    r.positions = launch.output(Py_None, "positions", {T, k}, at::kInt);
    r.sources = launch.output(Py_None, "sources", {rows}, at::kInt);
    if (!max_m) r.m_indices = launch.output(Py_None, "m_indices", {rows}, at::kInt);
    r.counts = launch.output(Py_None, "counts", {E}, at::kInt);
  }
  auto* const positions = static_cast<int32_t*>(table(r.positions, "layout.positions", T, k, at::kInt, dev));
  auto* const sources = static_cast<int32_t*>(vector(r.sources, "layout.sources", rows, at::kInt, dev));
  TORCH_CHECK_VALUE(r.m_indices.defined() == (max_m == 0), "layout.m_indices belongs to the contiguous layout, max_m to the masked one");
  auto* const m_indices = max_m ? nullptr : static_cast<int32_t*>(vector(r.m_indices, "layout.m_indices", rows, at::kInt, dev));
  auto* const counts = static_cast<int32_t*>(vector(r.counts, "layout.counts", E, at::kInt, dev));
  const MoeCopy c = copy_of(launch, Q, a[1], a[5], a[6], a[7], T, k, E, rows, max_m, dev);
  const size_t need = moe.dispatch_workspace(tokens, top_k, E);
  void* ws = nullptr;
  size_t ws_bytes = 0;
  Tensor scratch;
  if (given(a[9])) {
    const Tensor& t = tensor(a[9], "workspace");
    TORCH_CHECK_VALUE(t.device() == dev && t.is_contiguous(), "workspace must be contiguous on Q's device");
    ws = t.data_ptr(), ws_bytes = t.nbytes();
  } else if (need) {
    scratch = launch.scratch({(int64_t)need}, at::kByte);
    ws = scratch.data_ptr(), ws_bytes = need;
  }
  call("fp8_moe_dispatch", [&] {
    return moe.dispatch(c.q, c.ldq, c.sa, c.ld_sa, ids_p, c.weights, c.Qx.data_ptr(), c.ldqx, static_cast<float*>(c.sax.data_ptr()),
                        c.ld_sax, positions, sources, m_indices, counts, rows, max_m, tokens, top_k, E, c.cols, ws, ws_bytes,
                        launch.handle());
  });
  PyObject* m = r.m_indices.defined() ? THPVariable_Wrap(r.m_indices) : Py_NewRef(Py_None);
  return Py_BuildValue("NN(NNNN)", THPVariable_Wrap(c.Qx), THPVariable_Wrap(c.sax), THPVariable_Wrap(r.positions),
                       THPVariable_Wrap(r.sources), m, THPVariable_Wrap(r.counts));
  END_HANDLE_TH_ERRORS
}

// Q, sa, layout, weights, Qx, sax, stream -> (Qx, sax)
PyObject* moe_gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 7);
  const Tensor& Q = gpu_tensor(a[0], "Q", 2);
  const Device dev = Q.device();
  const c10::DeviceGuard guard(dev);
  const Launch launch(a[6], dev);
  const MoeRows r = layout_of(a[2]);
  const int64_t T = Q.size(0), rows = r.sources.numel(), E = r.counts.numel();
  TORCH_CHECK_VALUE(r.positions.dim() == 2, "layout.positions must be int32 [T, top_k]");
  const int64_t k = r.positions.size(1);
  auto* const positions = static_cast<const int32_t*>(table(r.positions, "layout.positions", T, k, at::kInt, dev));
  auto* const sources = static_cast<const int32_t*>(vector(r.sources, "layout.sources", rows, at::kInt, dev));
  const bool masked = !r.m_indices.defined();
  TORCH_CHECK_VALUE(!masked || (E >= 1 && rows % E == 0 && rows > 0), "a masked layout has max_m sources for each expert");
  const int tokens = to_int(T, "T"), top_k = to_int(k, "top_k"), max_m = masked ? to_int(rows / E, "max_m") : 0, experts = to_int(E, "E");
  const MoeCopy c = copy_of(launch, Q, a[1], a[3], a[4], a[5], T, k, E, rows, max_m, dev);
  call("fp8_moe_gather", [&] {
    return moe.gather(c.q, c.ldq, c.sa, c.ld_sa, c.weights, c.Qx.data_ptr(), c.ldqx, static_cast<float*>(c.sax.data_ptr()), c.ld_sax,
                      positions, sources, rows, max_m, tokens, top_k, experts, c.cols, launch.handle());
  });
  return Py_BuildValue("NN", THPVariable_Wrap(c.Qx), THPVariable_Wrap(c.sax));
  END_HANDLE_TH_ERRORS
}

// Experts' rows: [rows, N], or [E, max_m, N] with one row stride. -> (rows, row stride)
std::pair<int64_t, int64_t> expert_rows(const Tensor& t, const char* name, int64_t N, ScalarType type, Device dev) {
  TORCH_CHECK_VALUE((t.dim() == 2 || t.dim() == 3) && t.size(-1) == N && t.scalar_type() == type && t.device() == dev && t.stride(-1) == 1,
                    name, " must be ", type, " [rows, ", N, "] or [E, max_m, ", N, "] on ", dev, " with a unit inner stride");
  if (t.dim() == 2) return {t.size(0), row_stride(t)};
  return {t.size(0) * t.size(1), one_stride(t, name, N)};
}
const Tensor& experts_tensor(PyObject* o, const char* name) {
  const Tensor& t = tensor(o, name);
  TORCH_CHECK_VALUE(t.is_cuda() && rows_type(t) && (t.dim() == 2 || t.dim() == 3), name,
                    " must be a bfloat16 or float32 GPU tensor [rows, N] or [E, max_m, N]");
  return t;
}

// Y, positions, weights, C, out, stream -> out
PyObject* moe_combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 6);
  const Tensor& Y = experts_tensor(a[0], "Y");
  const Device dev = Y.device();
  const c10::DeviceGuard guard(dev);
  const Launch launch(a[5], dev);
  const int64_t N = Y.size(-1);
  const auto [rows, ldy] = expert_rows(Y, "Y", N, Y.scalar_type(), dev);
  const Tensor& at_ = gpu_tensor(a[1], "positions", 2);
  const int64_t T = at_.size(0), k = at_.size(1), count = rows, stride = ldy;
  auto* const positions = static_cast<const int32_t*>(table(at_, "positions", T, k, at::kInt, dev));
  const float* w = given(a[2]) ? static_cast<const float*>(table(tensor(a[2], "weights"), "weights", T, k, at::kFloat, dev)) : nullptr;
  const void* c = nullptr;
  int64_t ldc = 0;
  if (given(a[3])) {
    const Tensor& C = tensor(a[3], "C");
    ldc = matrix(C, "C", T, N, Y.scalar_type(), dev), c = C.data_ptr();
  }
  const Tensor out = launch.output(a[4], "out", {T, N}, Y.scalar_type());
  const int64_t ldo = matrix(out, "out", T, N, Y.scalar_type(), dev);
  const int tokens = to_int(T, "T"), top_k = to_int(k, "top_k"), cols = to_int(N, "N");
  call("fp8_moe_combine", [&] {
    return moe.combine(Y.data_ptr(), stride, type_code(Y), positions, w, c, ldc, out.data_ptr(), ldo, count, tokens, top_k, cols,
                       launch.handle());
  });
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// dO, Y, positions, weights, dY, dweights, rows, stream -> (dY, dweights)
PyObject* moe_combine_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 8);
  const Tensor &dO = rows_of(a[0], "dO"), &Y = experts_tensor(a[1], "Y");
  const Device dev = dO.device();
  const c10::DeviceGuard guard(dev);
  const Launch launch(a[7], dev);
  const int64_t T = dO.size(0), N = dO.size(1);
  const auto [rows, ldy] = expert_rows(Y, "Y", N, dO.scalar_type(), dev);
  const Tensor& at_ = gpu_tensor(a[2], "positions", 2);
  const int64_t k = at_.size(1), count = rows, stride = ldy;
  auto* const positions = static_cast<const int32_t*>(table(at_, "positions", T, k, at::kInt, dev));
  auto* const w = static_cast<const float*>(table(tensor(a[3], "weights"), "weights", T, k, at::kFloat, dev));
  Tensor dY;
  int64_t lddy = 0;
  if (to_bool(a[6])) {
    dY = launch.output(a[4], "dY", Y.sizes(), Y.scalar_type());
    TORCH_CHECK_VALUE(dY.sizes() == Y.sizes(), "dY must have Y's shape");
    lddy = expert_rows(dY, "dY", N, Y.scalar_type(), dev).second;
  } else {
    TORCH_CHECK_VALUE(!given(a[4]), "dY is written only with rows");
  }
  const Tensor dw = launch.output(a[5], "dweights", {T, k}, at::kFloat);
  auto* const dw_p = static_cast<float*>(table(dw, "dweights", T, k, at::kFloat, dev));
  const int tokens = to_int(T, "T"), top_k = to_int(k, "top_k"), cols = to_int(N, "N");
  call("fp8_moe_combine_backward", [&] {
    return moe.combine_grad(dO.data_ptr(), row_stride(dO), Y.data_ptr(), stride, type_code(dO), positions, w,
                            dY.defined() ? dY.data_ptr() : nullptr, lddy, dw_p, count, tokens, top_k, cols, launch.handle());
  });
  PyObject* d = dY.defined() ? THPVariable_Wrap(dY) : Py_NewRef(Py_None);
  return Py_BuildValue("NN", d, THPVariable_Wrap(dw));
  END_HANDLE_TH_ERRORS
}

// Row stride of a tensor that must be `type` [T, H, D] with contiguous rows.
int64_t typed_heads(const Tensor& t, const char* name, int64_t T, int64_t H, int64_t D, ScalarType type, Device dev) {
  TORCH_CHECK_VALUE(t.dim() == 3 && t.size(0) == T && t.size(1) == H && t.size(2) == D && t.scalar_type() == type && t.device() == dev &&
                        t.stride(2) == 1 && (H <= 1 || t.stride(1) == D),
                    name, " must be ", type, " [", T, ", ", H, ", ", D, "] on ", dev, " with contiguous rows");
  return T > 1 ? t.stride(0) : H * D;
}

// Table and positions of a rotation.
struct Rotation {
  const float* table = nullptr;
  const int32_t* positions = nullptr;
  int64_t ld = 0;
  int max_pos = 0, dim = 0;
};
Rotation rotation_of(PyObject* cos_sin, PyObject* positions, int64_t T, Device dev) {
  Rotation r;
  if (given(cos_sin)) {
    const Tensor& t = tensor(cos_sin, "cos_sin");
    TORCH_CHECK_VALUE(t.scalar_type() == at::kFloat && t.dim() == 2 && t.device() == dev && (t.size(1) <= 1 || t.stride(1) == 1),
                      "cos_sin must be float32 [max_pos, rot_dim] on ", dev, " with a unit inner stride");
    r.table = static_cast<const float*>(t.data_ptr());
    r.max_pos = to_int(t.size(0), "max_pos"), r.dim = to_int(t.size(1), "rot_dim"), r.ld = row_stride(t);
  }
  if (given(positions)) r.positions = static_cast<const int32_t*>(vector(tensor(positions, "positions"), "positions", T, at::kInt, dev));
  return r;
}
void* head_weight(PyObject* o, const char* name, int64_t D, const Tensor& like, Device dev) {
  const Tensor& t = tensor(o, name);
  TORCH_CHECK_VALUE(rows_type(t) && t.scalar_type() == like.scalar_type(), name, " must be bfloat16 or float32, both weights alike");
  return vector(t, name, D, t.scalar_type(), dev);
}

// q, k, q_weight, k_weight, cos_sin, positions, eps, interleaved, q_out, k_out, stream -> (q_out, k_out)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 11);
  TORCH_CHECK_VALUE(given(a[0]) || given(a[1]), "q and k are both missing");
  const Tensor& first = gpu_tensor(given(a[0]) ? a[0] : a[1], given(a[0]) ? "q" : "k", 3);
  TORCH_CHECK_VALUE(rows_type(first), "q and k must be bfloat16 or float32");
  const Device dev = first.device();
  const c10::DeviceGuard guard(dev);
  const Launch launch(a[10], dev);
  const int64_t T = first.size(0), D = first.size(2);
  const ScalarType type = first.scalar_type();
  const Tensor& weight = tensor(given(a[0]) ? a[2] : a[3], "weight");
  struct Part {
    const void *x = nullptr, *w = nullptr;
    void* y = nullptr;
    int64_t ldx = 0, ldy = 0, heads = 0;
    Tensor out;
  } part[2];
  const char *names[] = {"q", "k"}, *weights[] = {"q_weight", "k_weight"}, *outs[] = {"q_out", "k_out"};
  for (int i = 0; i < 2; ++i) {
    Part& p = part[i];
    if (!given(a[i])) {
      TORCH_CHECK_VALUE(!given(a[8 + i]), outs[i], " without ", names[i]);
      continue;
    }
    const Tensor& x = gpu_tensor(a[i], names[i], 3);
    p.heads = x.size(1);
    p.ldx = typed_heads(x, names[i], T, p.heads, D, type, dev), p.x = x.data_ptr();
    p.w = head_weight(a[2 + i], weights[i], D, weight, dev);
    p.out = launch.output(a[8 + i], outs[i], {T, p.heads, D}, type);
    p.ldy = typed_heads(p.out, outs[i], T, p.heads, D, type, dev), p.y = p.out.data_ptr();
  }
  const Rotation r = rotation_of(a[4], a[5], T, dev);
  const float eps = to_float(a[6]);
  const bool interleaved = to_bool(a[7]);
  const int tokens = to_int(T, "T"), Hq = to_int(part[0].heads, "Hq"), Hk = to_int(part[1].heads, "Hk"), dim = to_int(D, "D");
  call("fp8_qk_norm_rope", [&] {
    return moe.heads(part[0].x, part[0].ldx, part[1].x, part[1].ldx, type_code(first), part[0].w, part[1].w, type_code(weight), r.table,
                     r.ld, r.max_pos, r.dim, interleaved, r.positions, eps, part[0].y, part[0].ldy, part[1].y, part[1].ldy, tokens, Hq, Hk,
                     dim, launch.handle());
  });
  PyObject* made[2];
  for (int i = 0; i < 2; ++i) made[i] = part[i].out.defined() ? THPVariable_Wrap(part[i].out) : Py_NewRef(Py_None);
  return Py_BuildValue("NN", made[0], made[1]);
  END_HANDLE_TH_ERRORS
}

// dq, dk, q, k, q_weight, k_weight, cos_sin, positions, eps, interleaved, dq_out, dk_out, workspace, stream
// -> (dq_out, dk_out, dq_weight, dk_weight)
PyObject* qk_norm_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 14);
  TORCH_CHECK_VALUE(given(a[0]) || given(a[1]), "dq and dk are both missing");
  const Tensor& first = gpu_tensor(given(a[0]) ? a[0] : a[1], given(a[0]) ? "dq" : "dk", 3);
  TORCH_CHECK_VALUE(rows_type(first), "dq and dk must be bfloat16 or float32");
  const Device dev = first.device();
  const c10::DeviceGuard guard(dev);
  const Launch launch(a[13], dev);
  const int64_t T = first.size(0), D = first.size(2);
  const ScalarType type = first.scalar_type();
  const Tensor& weight = tensor(given(a[0]) ? a[4] : a[5], "weight");
  struct Part {
    const void *dy = nullptr, *x = nullptr, *w = nullptr;
    void *dx = nullptr, *dw = nullptr;
    int64_t lddy = 0, ldx = 0, lddx = 0, heads = 0;
    Tensor out, dweight;
  } part[2];
  const char *grads[] = {"dq", "dk"}, *names[] = {"q", "k"}, *weights[] = {"q_weight", "k_weight"}, *outs[] = {"dq_out", "dk_out"};
  for (int i = 0; i < 2; ++i) {
    Part& p = part[i];
    if (!given(a[i])) {
      TORCH_CHECK_VALUE(!given(a[10 + i]), outs[i], " without ", grads[i]);
      continue;
    }
    const Tensor &dy = gpu_tensor(a[i], grads[i], 3), &x = tensor(a[2 + i], names[i]);
    p.heads = dy.size(1);
    p.lddy = typed_heads(dy, grads[i], T, p.heads, D, type, dev), p.dy = dy.data_ptr();
    p.ldx = typed_heads(x, names[i], T, p.heads, D, type, dev), p.x = x.data_ptr();
    p.w = head_weight(a[4 + i], weights[i], D, weight, dev);
    p.out = launch.output(a[10 + i], outs[i], {T, p.heads, D}, type);
    p.lddx = typed_heads(p.out, outs[i], T, p.heads, D, type, dev), p.dx = p.out.data_ptr();
    p.dweight = launch.output(Py_None, "dweight", {D}, at::kFloat), p.dw = p.dweight.data_ptr();
  }
  const Rotation r = rotation_of(a[6], a[7], T, dev);
  const float eps = to_float(a[8]);
  const bool interleaved = to_bool(a[9]);
  const int tokens = to_int(T, "T"), Hq = to_int(part[0].heads, "Hq"), Hk = to_int(part[1].heads, "Hk"), dim = to_int(D, "D");
  const Tensor ws = given(a[12]) ? tensor(a[12], "workspace") : launch.scratch({(int64_t)moe.heads_workspace(dim)}, at::kByte);
  TORCH_CHECK_VALUE(ws.device() == dev && ws.is_contiguous(), "workspace must be contiguous on the gradients' device");
  call("fp8_qk_norm_rope_backward", [&] {
    return moe.heads_grad(part[0].dy, part[0].lddy, part[1].dy, part[1].lddy, part[0].x, part[0].ldx, part[1].x, part[1].ldx,
                          type_code(first), part[0].w, part[1].w, type_code(weight), r.table, r.ld, r.max_pos, r.dim, interleaved,
                          r.positions, eps, part[0].dx, part[0].lddx, part[1].dx, part[1].lddx, static_cast<float*>(part[0].dw),
                          static_cast<float*>(part[1].dw), tokens, Hq, Hk, dim, ws.data_ptr(), ws.nbytes(), launch.handle());
  });
  PyObject* made[4];
  for (int i = 0; i < 2; ++i) {
    made[i] = part[i].out.defined() ? THPVariable_Wrap(part[i].out) : Py_NewRef(Py_None);
    made[2 + i] = part[i].dweight.defined() ? THPVariable_Wrap(part[i].dweight) : Py_NewRef(Py_None);
  }
  return Py_BuildValue("NNNN", made[0], made[1], made[2], made[3]);
  END_HANDLE_TH_ERRORS
}

// The functions of fp8moe.h as a dict of addresses by name
PyObject* bind_moe(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 1);
  set_address(a[0], moe.route, "fp8_moe_route");
  set_address(a[0], moe.route_grad, "fp8_moe_route_backward");
  set_address(a[0], moe.rows, "fp8_moe_rows");
  set_address(a[0], moe.dispatch, "fp8_moe_dispatch");
  set_address(a[0], moe.dispatch_workspace, "fp8_moe_dispatch_workspace_size");
  set_address(a[0], moe.gather, "fp8_moe_gather");
  set_address(a[0], moe.combine, "fp8_moe_combine");
  set_address(a[0], moe.combine_grad, "fp8_moe_combine_backward");
  set_address(a[0], moe.heads, "fp8_qk_norm_rope");
  set_address(a[0], moe.heads_grad, "fp8_qk_norm_rope_backward");
  set_address(a[0], moe.heads_workspace, "fp8_qk_norm_rope_backward_workspace_size");
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

}  // namespace
