/*
 * fp8moe.h -- C ABI of the operators that a mixture-of-experts decoder layer needs around
 * the grouped GEMMs of fp8gemm.h and the layer operators of fp8layer.h, in libfp8gemm.so.
 *
 *   fp8_moe_route                scores of experts, the choice among them, weights
 *   fp8_moe_route_backward       the gradient of the logits
 *   fp8_moe_dispatch             lays tokens' 8-bit rows out by expert
 *   fp8_moe_gather               the same rows again, for a layout that is there
 *   fp8_moe_combine              weighted sum of the experts' rows of each token
 *   fp8_moe_combine_backward     its gradients
 *   fp8_qk_norm_rope             norm of queries and keys for each head, and rotation
 *   fp8_qk_norm_rope_backward    its gradients
 *
 * The conventions of fp8gemm.h and fp8layer.h hold: device pointers owned by the caller,
 * asynchronous work on `stream`, nothing allocated, freed or synchronised, device memory
 * never read by the host, strides in ELEMENTS, FP8GEMM_* status codes, nothing launched on
 * an argument error, no exception across the ABI. Calls may be captured into graphs. Types
 * of rows are FP8GEMM_QUANT_BF16 and FP8GEMM_QUANT_FP32. Sums are FP32 in an order that the
 * inputs, the shapes and the compute units in use (fp8_gemm_set_num_cus) fix, so equal calls
 * give equal bits. Among calls of other numbers of tokens or units a row's scores and weights, and
 * the heads' weight gradients, may differ in their last bits; chosen experts, layouts and what
 * is not summed over tokens do not. Expert and row numbers on the device are not trusted with
 * addresses: one outside its range counts as none. A call without tokens (T == 0) looks at no
 * pointer to tokens' data. Arrays do not overlap, except where said; calls that may run at the
 * same time do not share a workspace.
 */
#ifndef FP8MOE_H_
#define FP8MOE_H_

#include "fp8gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { FP8MOE_SOFTMAX = 0, FP8MOE_SIGMOID = 1 };

/*
 * For each token t of logits x [T, E]:
 *     s = softmax(x) over all E, or sigmoid(x)
 *     key = s + bias (s without one)
 *     with groups > 1: the experts are `groups` runs of E / groups; a group's score is the
 *     sum of its group_best (1 or 2) largest keys, as many as it has, and the experts of
 *     the top_groups best groups are left
 *     ids = the top_k largest keys that are left, in falling order
 *     w = scale * s[ids] / (sum of s[ids] + 1e-20), or scale * s[ids] without renormalize
 * Ties go to the lower index, of groups and experts alike. The order is that of the exact
 * keys: where FP32 cannot tell two of them apart they are computed in FP64 (without a bias
 * the logits' own order decides between experts). An expert whose logit or key is -inf is
 * never chosen; where fewer than top_k are left, the last ids are -1 with weight 0. NaN
 * keys are chosen last, after every number; the weights are what the formula gives.
 *   logits  BF16 or FP32 (dtype), row stride ldl. bias fp32 [E] or NULL.
 *   ids     int32 [T, top_k], weights fp32 [T, top_k], contiguous.
 *   scores  optional fp32 [T, E], row stride lds: s.
 * 1 <= E <= 1024, 1 <= top_k <= min(E, 64), groups divides E and is at most 64,
 * 1 <= top_groups <= groups, scale between -2^60 and 2^60.
 */
int fp8_moe_route(const void* logits, int64_t ldl, int dtype, const float* bias, int scoring, int groups,
                  int top_groups, int group_best, int renormalize, float scale, int32_t* ids, float* weights,
                  float* scores, int64_t lds, int T, int E, int top_k, hipStream_t stream);

/*
 * Gradient of the logits, for dweights [T, top_k] (FP32, contiguous) that arrives at w, and
 * optionally dscores [T, E] (FP32, row stride ldds) at s, the choice taken as given: with
 * S = sum of s[ids] + 1e-20 and g = scale * dweights,
 *     ds[ids_i] = (g_i - sum_j g_j s[ids_j] / S) / S, or g_i without renormalize; plus dscores
 *     dx = s (ds - sum_e ds_e s_e) for the softmax, ds s (1 - s) for the sigmoid
 * s is computed from the logits again. An id outside [0, E) has no part in it. dlogits [T, E]
 * of the logits' type, row stride lddl; may be the logits themselves. Limits as above.
 */
int fp8_moe_route_backward(const float* dweights, const void* logits, int64_t ldl, int dtype, const int32_t* ids,
                           int scoring, int renormalize, float scale, const float* dscores, int64_t ldds,
                           void* dlogits, int64_t lddl, int T, int E, int top_k, hipStream_t stream);

/* Rows that the contiguous layout of T tokens with top_k choices each among E experts can
 * need: segments rounded up to 128 rows, at worst. 0 for arguments out of range. */
int64_t fp8_moe_rows(int T, int top_k, int E);

/*
 * Lays tokens out by expert, in the layouts of the grouped GEMMs:
 *   contiguous (max_m == 0): expert e's segment begins at a multiple of 128 rows, after
 *       those of the experts before it; `rows` rows in all, a multiple of 128.
 *       Qx e4m3 [rows, K], sax fp32 [K/128][ld_sax], m_indices int32 [rows].
 *   masked (max_m > 0): expert e has rows e max_m .. e max_m + max_m - 1; rows == E max_m.
 *       Qx e4m3 [E, max_m, K], sax fp32 [E][K/128][ld_sax], masked_m = counts.
 * Within an expert the choices come in the order of tokens (and of a token's choices).
 *   Q       e4m3 [T, K], row stride ldq; sa fp32 [K/128][ld_sa].
 *   ids     int32 [T, top_k], contiguous. An id outside [0, E) is no choice.
 *   weights optional fp32 [T, top_k], contiguous: the row's scales are multiplied by it
 *           (one rounding), so that the row stands for weight * token.
 *   positions  int32 [T, top_k]: the row of each choice, -1 where it has none: no choice, or
 *              past max_m rows of its expert, or past `rows`.
 *   sources    int32 [rows]: the choice t top_k + j in each row, -1 in the others.
 *   m_indices  int32 [rows] (contiguous only): the expert of each row, -1 in rows without a
 *              choice.
 *   counts     int32 [E]: each expert's rows that hold a choice.
 * Rows of Qx and columns of sax without a choice keep what they held.
 * With Q NULL the layout alone is made (sa, Qx and sax are not looked at).
 *   workspace  fp8_moe_dispatch_workspace_size(T, top_k, E) bytes, 16-byte aligned (may be
 *              NULL where that is 0); needs no initial value.
 * K a multiple of 128 up to 65536; Q, Qx 16-byte aligned with strides multiples of 16; ld_sa
 * >= T, ld_sax >= rows (masked: max_m), multiples of 4. 1 <= E <= 1024, 1 <= top_k <= 64;
 * T * top_k and rows below 2^31 - 2^18 (the segments of 1024 experts end within 32 bits).
 */
int fp8_moe_dispatch(const void* Q, int64_t ldq, const float* sa, int64_t ld_sa, const int32_t* ids,
                     const float* weights, void* Qx, int64_t ldqx, float* sax, int64_t ld_sax, int32_t* positions,
                     int32_t* sources, int32_t* m_indices, int32_t* counts, int64_t rows, int max_m, int T, int top_k,
                     int E, int K, void* workspace, size_t workspace_bytes, hipStream_t stream);
size_t fp8_moe_dispatch_workspace_size(int T, int top_k, int E);

/* The rows of a layout that is there: Qx and sax as fp8_moe_dispatch writes them for Q, sa
 * and weights (a gradient's rows, for instance). positions and sources as written by it; E is
 * needed with max_m > 0 only. */
int fp8_moe_gather(const void* Q, int64_t ldq, const float* sa, int64_t ld_sa, const float* weights, void* Qx,
                   int64_t ldqx, float* sax, int64_t ld_sax, const int32_t* positions, const int32_t* sources,
                   int64_t rows, int max_m, int T, int top_k, int E, int K, hipStream_t stream);

/*
 * out[t] = C[t] + sum_j weights[t, j] * Y[positions[t, j]], in FP32 in the order of j,
 * rounded once. positions outside [0, rows) add nothing. Without weights (NULL) each is 1:
 * that is the gradient of a dispatch.
 *   Y    [rows, N] BF16 or FP32 (dtype), row stride ldy. The masked layout's rows are
 *        e max_m + r.
 *   C    optional [T, N] of that type, row stride ldc; may be out itself.
 *   out  [T, N] of that type, row stride ldo.
 *   weights fp32, positions int32 [T, top_k], contiguous.
 * N a multiple of 8; Y, C, out 16-byte aligned, strides multiples of 16 bytes; 1 <= top_k <=
 * 64, rows below 2^31.
 */
int fp8_moe_combine(const void* Y, int64_t ldy, int dtype, const int32_t* positions, const float* weights,
                    const void* C, int64_t ldc, void* out, int64_t ldo, int64_t rows, int T, int top_k, int N,
                    hipStream_t stream);

/*
 * Gradients of that sum, for dO [T, N]:
 *     dY[positions[t, j]] = weights[t, j] * dO[t], rounded once (optional: dY may be NULL)
 *     dweights[t, j] = sum_n dO[t, n] * Y[positions[t, j], n], 0 without a position
 * Rows of dY that no position names keep what they held. A row may be named once. dY may be Y
 * itself (same stride). All rows of one type; limits as above.
 */
int fp8_moe_combine_backward(const void* dO, int64_t lddo, const void* Y, int64_t ldy, int dtype,
                             const int32_t* positions, const float* weights, void* dY, int64_t lddy, float* dweights,
                             int64_t rows, int T, int top_k, int N, hipStream_t stream);

/*
 * Norm of each head of queries and keys, and rotation by the token's position, in one pass;
 * for a head's D columns x, in FP32 with one rounding at the end:
 *     n = x * rstd * w,  rstd = 1 / sqrt(mean(x^2) + eps)
 *     out = n with the pairs of its first rot_dim columns turned, as by
 *     fp8_rope_append_paged_kv (halves or interleaved)
 *   q, k   [T, Hq, D], [T, Hk, D] BF16 or FP32 (dtype), row strides ldq, ldk, head h at column
 *          h D. Either may be NULL, with its output. q_out, k_out may be q, k (same stride).
 *   qw, kw [D] BF16 or FP32 (w_dtype).
 *   cos_sin  fp32 [max_pos][ld_cs], cosines of rot_dim / 2 angles, then their sines.
 *   positions  int32 [T], clamped to [0, max_pos); NULL: t.
 * D 64, 128 or 256; rot_dim a multiple of 16, 0 .. D (0: no table). Addresses 16-byte aligned,
 * row strides multiples of 16 bytes, ld_cs of 4. T * (Hq + Hk) below 2^31 - 2^18, Hq * D and
 * Hk * D below 2^31.
 */
int fp8_qk_norm_rope(const void* q, int64_t ldq, const void* k, int64_t ldk, int dtype, const void* qw, const void* kw,
                     int w_dtype, const float* cos_sin, int64_t ld_cs, int max_pos, int rot_dim, int interleaved,
                     const int32_t* positions, float eps, void* q_out, int64_t ldqo, void* k_out, int64_t ldko, int T,
                     int Hq, int Hk, int D, hipStream_t stream);

/*
 * Its gradients, for dq and dk that arrive at q_out and k_out: with dn the gradient turned
 * back, g = dn * w and xh = x * rstd,
 *     dx = rstd * (g - xh * mean(g * xh)), rounded once; dw = sum over tokens and heads of dn * xh
 * q, k are the norm's inputs. dq_out, dk_out may be dq, dk or q, k (same stride). dqw, dkw:
 * fp32 [D], overwritten (zero for T == 0).
 *   workspace  fp8_qk_norm_rope_backward_workspace_size(D) bytes, 16-byte aligned; needs no
 *              initial value.
 */
int fp8_qk_norm_rope_backward(const void* dq, int64_t lddq, const void* dk, int64_t lddk, const void* q, int64_t ldq,
                              const void* k, int64_t ldk, int dtype, const void* qw, const void* kw, int w_dtype,
                              const float* cos_sin, int64_t ld_cs, int max_pos, int rot_dim, int interleaved,
                              const int32_t* positions, float eps, void* dq_out, int64_t lddqo, void* dk_out,
                              int64_t lddko, float* dqw, float* dkw, int T, int Hq, int Hk, int D, void* workspace,
                              size_t workspace_bytes, hipStream_t stream);
size_t fp8_qk_norm_rope_backward_workspace_size(int D);

#ifdef __cplusplus
}
#endif

#endif /* FP8MOE_H_ */
