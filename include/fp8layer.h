/*
 * fp8layer.h -- C ABI of the operators around the FP8 GEMMs of a transformer layer, in
 * libfp8gemm.so: the norm that produces a GEMM's 8-bit A operand (with its gradient), and
 * attention over a paged cache held in 8 bits, with the append that fills the cache.
 *
 *   fp8_rmsnorm_quantize_1x128   residual addition, RMS norm, 1x128 quantisation
 *   fp8_rmsnorm_backward         gradients of the norm's input and weight
 *   fp8_rope_append_paged_kv     rotates queries and keys, appends keys and values
 *   fp8_paged_attention          causal attention over the cache, one token or many
 *
 * The conventions of fp8gemm.h hold: device pointers owned by the caller, asynchronous
 * work on `stream`, nothing allocated, freed or synchronised, device memory never read by
 * the host, strides in ELEMENTS, FP8GEMM_* status codes, nothing launched on an argument
 * error, no exception across the ABI. A call may be captured into a graph: grids depend on
 * the host arguments only, and lengths are read on the device.
 *
 * The paged cache of one layer (keys and values alike):
 *   codes   e4m3 [num_pages][Hkv][P][D], contiguous, 16-byte aligned: P token slots of one
 *           page and head lie together. P (the page size) is 16, 32, 64, 128 or 256, D
 *           (the head size) 64, 128 or 256.
 *   scales  fp32 [num_pages][Hkv], contiguous: one power of two per page and head (a UE8M0
 *           value held as FP32; only its exponent is read). A code c of page p and head h
 *           stands for c * scales[p][h].
 * Which pages hold a sequence is its row of the block table:
 *   block_table  int32 [B][ld_bt]: entry j < max_pages is the page of token slots
 *           j P .. j P + P - 1. Entries past a sequence's length are not read. Slots from
 *           max_pages P on have no page: a token there keeps its position, and is not
 *           stored and not seen.
 *   seq_lens     int32 [B]: the sequence's length in the cache, the call's new tokens
 *           included.
 *   cu_q         int32 [B + 1]: rows cu_q[b] .. cu_q[b + 1] - 1 of the call's tokens belong to
 *           sequence b and are the last of its seq_lens[b] tokens; cu_q[0] = 0,
 *           non-decreasing. A sequence may have none.
 * These arrays are device data and are not trusted with addresses: a length below 0 counts
 * as 0, row numbers are clamped to [0, T], slots past the table are never looked up, and a
 * page number outside [0, num_pages) is never followed (the append writes nothing there,
 * attention leaves its keys out). Offsets in cu_q that overlap give rows of no meaning, and
 * no access outside the arrays.
 * A call without rows (M, T or B is 0) does nothing and looks at no pointer to rows or to
 * these arrays. A table without pages (max_pages 0) may be NULL: nothing is stored or seen.
 */
#ifndef FP8LAYER_H_
#define FP8LAYER_H_

#include "fp8gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Residual addition, root-mean-square norm and 1x128 quantisation in one pass, producing
 * the A operand and scales of the GEMM that follows. Per row, in FP32 unless noted:
 *     h = X + R, rounded to X's type (h = X when R is NULL)
 *     rstd = 1 / sqrt(mean(h^2) + eps)
 *     y = (h * rstd) * w
 *     per 128 columns: s = amax(|y|) / 448 (1 if that is 0), q = e4m3_rne(y / s)
 * (the last line as fp8_quantize_1x128). The norm is taken of h as stored, so that a
 * backward pass that reads H sees what was normalised.
 *   X   [M, K] BF16 or FP32 (x_dtype, FP8GEMM_QUANT_*), row stride ldx.
 *   R   optional [M, K] of X's type, row stride ldr (NULL: no addition).
 *   w   [K] BF16 or FP32 (w_dtype).
 *   H   [M, K] of X's type, row stride ldh: h. Required with R (it may be R or X itself,
 *       with the same stride), ignored without.
 *   Y   optional [M, K] BF16, row stride ldy: y rounded to BF16, for readers that take the
 *       norm unquantised (a router).
 *   rstd optional fp32 [M].
 *   Q   e4m3 [M, K], row stride ldq; sa fp32 [K/128][ld_sa] (sa[kb * ld_sa + m]; columns
 *       past M are untouched).
 * K is a multiple of 128 and at most 65536. X, R, H, w are 16-byte aligned with row
 * strides multiples of 16 bytes, likewise Y; Q is 8-byte aligned, ldq % 8 == 0; ld_sa >= M
 * and a multiple of 4. NaN and infinities are outside the contract, as for
 * fp8_quantize_1x128. eps >= 0. M == 0 is a no-op.
 */
int fp8_rmsnorm_quantize_1x128(const void* X, int64_t ldx, const void* R, int64_t ldr, int x_dtype,
                               const void* w, int w_dtype, float eps, void* H, int64_t ldh,
                               void* Y, int64_t ldy, float* rstd, void* Q, int64_t ldq,
                               float* sa, int64_t ld_sa, int M, int K, hipStream_t stream);

/*
 * Gradients of y = h * rstd(h) * w for an arriving gradient dY, all in FP32 with one
 * rounding per output (the quantisation counts as the identity):
 *     g = dY * w,  xhat = H * rstd
 *     dX[m] = rstd[m] * (g[m] - xhat[m] * mean_k(g[m] * xhat[m])) + dH[m]
 *     dW[k] = sum_m dY[m][k] * xhat[m][k]
 * dX is the gradient of X and of R alike; dH, the gradient that arrives at H over the
 * residual stream, is optional.
 *   dY, H, dH, dX  [M, K] of one type (dtype), row strides ld*; dX may be dY or dH itself.
 *   rstd  fp32 [M], as written by the forward call. w [K] (w_dtype).
 *   dW    fp32 [K], overwritten. The rows are summed in an order that is fixed by M, K, dtype,
 *         whether dH is given, the number of compute units (fp8_gemm_set_num_cus), and
 *         whether the memory that dX's rows span meets that of dY's or H's rows: equal
 *         inputs give equal bits in any such call.
 *   workspace  fp8_rmsnorm_backward_workspace_size(M, K) bytes, 16-byte aligned; its
 *         contents need no initial value. FP8GEMM_ERR_WORKSPACE if smaller or NULL.
 * K, alignment and strides as above. M == 0 zeroes dW.
 */
int fp8_rmsnorm_backward(const void* dY, int64_t lddy, const void* H, int64_t ldh, const void* dH, int64_t lddh,
                         int dtype, const float* rstd, const void* w, int w_dtype, void* dX, int64_t lddx,
                         float* dW, int M, int K, void* workspace, size_t workspace_bytes, hipStream_t stream);
size_t fp8_rmsnorm_backward_workspace_size(int M, int K);

/*
 * Rotates the call's queries and keys by their positions and appends keys and values to
 * the cache. Token t of sequence b lands in slot s = seq_lens[b] - (cu_q[b + 1] - t) and is
 * rotated by position positions[t], or s when positions is NULL (clamped to
 * [0, max_pos)). A rotation turns each pair (x1, x2) of the first rot_dim columns by the
 * pair's angle: (x1 cos - x2 sin, x2 cos + x1 sin), each product and the sum rounded in
 * FP32; the other columns pass. Pair i is columns (i, i + rot_dim / 2), or (2 i, 2 i + 1)
 * when interleaved.
 *   q, k, v  BF16, rows ldq / ldk / ldv apart, head h of a row at column h D (views of one
 *            fused projection output will do).
 *   cos_sin  fp32 [max_pos][ld_cs]: cosines of the rot_dim / 2 angles, then their sines.
 *   q_out    BF16 [T, Hq, D], row stride ldqo, rounded once; may be q itself (same
 *            stride). q and q_out may both be NULL: then only the cache is filled.
 * The cache's scales: a page's scale is the smallest power of two (2^-126 at least) by
 * which the largest finite |value| appended to it fits 448. It only grows: when a later
 * append needs a larger one, the page's earlier codes are re-encoded at it (exact but for
 * what falls below the smallest code). A page whose first slot is appended starts afresh,
 * whatever it held. Values are rounded to the nearest code, ties to even; NaN and
 * infinities are stored as the NaN code and do not move the scale.
 * A page that the call appends to must belong to one sequence. Slots below 0 (more new
 * tokens than seq_lens) and past the table (max_pages P and on) are dropped; their queries
 * are rotated like all others. Rows past cu_q[B] are untouched.
 * D, P as above; rot_dim a multiple of 16, 0 .. D. q, k, v, q_out, cos_sin 16-byte
 * aligned, their strides multiples of 8 (BF16) and 4 (cos_sin) elements. T * Hq, T * Hkv,
 * Hq * D, Hkv * D and max_pages * P below 2^31.
 */
int fp8_rope_append_paged_kv(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                             const float* cos_sin, int64_t ld_cs, int max_pos, int rot_dim, int interleaved,
                             const int32_t* positions, const int32_t* block_table, int64_t ld_bt, int max_pages,
                             const int32_t* seq_lens, const int32_t* cu_q, void* q_out, int64_t ldqo,
                             void* k_cache, float* k_scale, void* v_cache, float* v_scale, int num_pages, int P,
                             int B, int T, int Hq, int Hkv, int D, hipStream_t stream);

/*
 * Causal attention of the call's queries over the cache, which already holds the call's
 * own tokens. Row t of sequence b stands at position p = seq_lens[b] - (cu_q[b + 1] - t)
 * and sees the keys j <= p (with window > 0: p - window < j <= p). For query head i and
 * key head i / (Hq / Hkv):
 *     O[t, i] = sum_j softmax_j(softmax_scale * q[t, i] . k[j]) v[j]
 *     lse[t, i] = log sum_j exp(softmax_scale * q[t, i] . k[j])
 * A row that sees no key gives O = 0 and lse = -inf. Rows past cu_q[B] are untouched.
 * Products of BF16 queries and 8-bit keys are exact and summed in FP32; probabilities are
 * rounded to 11 bits for the second product, whose sum is FP32; statistics are FP32.
 *   q    BF16 [T, Hq, D], row stride ldq; O BF16 [T, Hq, D], row stride ldo; lse optional
 *        fp32 [T, Hq], contiguous.
 *   Of the cache's scales only the exponents are read.
 *   workspace  optional, 16-byte aligned: lets long sequences be split over workgroups,
 *        whose results are joined in a fixed order. Its first 64 KiB (arrival counters)
 *        must be zero before its first use, and are zero again when a call completes. Any
 *        size may be given; fp8_paged_attention_workspace_size() suffices for every call.
 *        Calls that may run at the same time must not share it.
 * NaN codes in slots that no row sees change nothing; a row that sees one gives NaN.
 * Hkv divides Hq. q, O 16-byte aligned with strides multiples of 8; T * Hq and Hq * D
 * below 2^31, max_pages * P at most 2^30; window >= 0; num_pages >= 1.
 */
int fp8_paged_attention(const void* q, int64_t ldq, const void* k_cache, const float* k_scale, const void* v_cache,
                        const float* v_scale, int num_pages, int P, const int32_t* block_table, int64_t ld_bt,
                        int max_pages, const int32_t* seq_lens, const int32_t* cu_q, void* O, int64_t ldo,
                        float* lse, float softmax_scale, int window, int B, int T, int Hq, int Hkv, int D,
                        void* workspace, size_t workspace_bytes, hipStream_t stream);
size_t fp8_paged_attention_workspace_size(void);

#ifdef __cplusplus
}
#endif

#endif /* FP8LAYER_H_ */
