// Host side of the layer operators of libfp8gemm (include/fp8layer.h): argument checks,
// the choice among compiled instances, and the launches.
#include "fp8layer.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "attention_kernel.hpp"
#include "host.hpp"
#include "kvcache_kernel.hpp"
#include "rmsnorm_kernel.hpp"

namespace {

// ---------------------------------------------------------------------------- RMS norm

constexpr int kMaxNormCols = 65536;

// Waves that share a row, and most chunks of eight columns a thread. Forward: where rows
// are many, as few waves as keep a row within four chunks a thread (K = 7168: 8 workgroups
// of 4 waves on a CU); where they would not fill the GPU, one chunk a thread, for latency
// (K = 7168, 256 rows: 6.5 us by few waves, 5.0 by many; 700: 10.9 and 10.2; 2048: 22.7 and 24.2).
struct NormShape {
  int waves, chunks;
};
NormShape norm_shape(int M, int K, int cus) {
  const int chunks = K / 8;
  if (M <= 4 * cus) {
    if (chunks <= 64) return {1, 1};
    if (chunks <= 4 * 64) return {4, 1};
    if (chunks <= 16 * 64) return {16, 1};
  }
  for (int ch : {1, 2, 4})
    if (chunks <= 64 * ch) return {1, ch};
  if (chunks <= 4 * 64 * 4) return {4, 4};
  return {16, chunks <= 16 * 64 * 4 ? 4 : 8};
}
// Backward: one chunk a thread up to 16 waves a row.
NormShape norm_grad_shape(int K) {
  const int chunks = K / 8;
  for (int waves : {1, 2, 4, 8})
    if (chunks <= waves * 64) return {waves, 1};
  for (int ch : {1, 2, 4})
    if (chunks <= 16 * 64 * ch) return {16, ch};
  return {16, 8};
}

// Calls f(waves, chunks) with the shape as compile-time values.
template <typename F>
void with_shape(NormShape s, F f) {
  if (s.waves == 1) {
    if (s.chunks == 1) f(Int<1>{}, Int<1>{});
    else if (s.chunks == 2) f(Int<1>{}, Int<2>{});
    else f(Int<1>{}, Int<4>{});
  } else if (s.waves == 4) {
    if (s.chunks == 1) f(Int<4>{}, Int<1>{});
    else f(Int<4>{}, Int<4>{});
  } else if (s.chunks == 1) {
    f(Int<16>{}, Int<1>{});
  } else if (s.chunks == 4) {
    f(Int<16>{}, Int<4>{});
  } else {
    f(Int<16>{}, Int<8>{});
  }
}
// Whether a gradient is taken in one launch, which reads the rows twice: where they are 32 MB
// at most and a row's chunks are one a thread. In two launches and in one, in a graph: FP32
// 16 x 1536 5.7 and 3.5 us, 512 x 2048 8.4 and 6.1, 1024 x 512 6.3 and 4.8, 1024 x 2048 10.5 and
// 10.7, 1024 x 4096 15.4 and 14.6; BF16 256 x 8192 11.5 and 6.7, 1024 x 1024 6.7 and 4.8,
// 1024 x 8192 15.9 and 15.2. But for more than three FP32 rows a CU between those widths the
// second reading costs more than a launch: 1024 x 768 7.2 and 9.2, x 1024 7.8 and 9.7, x 1280
// 8.7 and 11.2, x 1536 9.3 and 10.7 (768 x 1024: 7.1 and 6.8).
bool norm_grad_few(int M, int K, size_t bytes, bool fp32, int cus) {
  if (fp32 && M > 3 * cus && K > 512 && K < 2048) return false;
  return M <= 4 * cus && K <= 8 * 1024 && !streams(M, K, bytes);
}
// Whether rows written to dX lie among those at p: then no workgroup may read what another
// has finished with.
bool rows_meet(const void* dX, int64_t lddx, const void* p, int64_t ld, int M, int K, size_t size) {
  const uintptr_t a = (uintptr_t)dX, b = (uintptr_t)p;
  return a < b + ((size_t)(M - 1) * ld + K) * size && b < a + ((size_t)(M - 1) * lddx + K) * size;
}
template <typename F>
void with_grad_shape(NormShape s, F f) {
  if (s.waves == 1) f(Int<1>{}, Int<1>{});
  else if (s.waves == 2) f(Int<2>{}, Int<1>{});
  else if (s.waves == 4) f(Int<4>{}, Int<1>{});
  else if (s.waves == 8) f(Int<8>{}, Int<1>{});
  else if (s.chunks == 1) f(Int<16>{}, Int<1>{});
  else if (s.chunks == 2) f(Int<16>{}, Int<2>{});
  else if (s.chunks == 4) f(Int<16>{}, Int<4>{});
  else f(Int<16>{}, Int<8>{});
}

int norm_grad_groups(int M, NormShape s, int cus) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(ceil_div(M, 16 / s.waves), cus));
}

// ------------------------------------------------------------------- paged cache, attention

bool cache_shape(int num_pages, int P, int Hkv, int D) {
  return num_pages >= 1 && Hkv >= 1 && (P == 16 || P == 32 || P == 64 || P == 128 || P == 256) &&
         (D == 64 || D == 128 || D == 256);
}
int log2_of(int P) {
  int n = 0;
  while ((1 << n) < P) ++n;
  return n;
}

// Blocks of 16 rows in a tile. One or two where that holds a sequence's rows; otherwise two,
// or the most that registers allow if that takes less time by the padded rows (a row of a
// larger tile costs kLargeTile of one of two blocks: 2 x 2048 prompt tokens over 8192 keys,
// 32 query heads on 8 key heads: D = 64 679 and 752 TFLOP/s, 128 818 and 918, 256 650 and
// 735) and if the tiles are enough to give every CU one (2 x 128 tokens of 16 heads of 64
// over 1000 keys, which are not: 12.3 us in tiles of 32 rows, 15.7 in larger ones).
constexpr int most_row_blocks(int D) { return D == 64 ? 4 : 3; }
constexpr double kLargeTile = 0.9;
constexpr int kFewKeys = 2048;  // for a CU
int attention_row_blocks(int64_t rows, int64_t heads, int D, int cus) {
  if (rows <= 32) return rows <= 16 ? 1 : 2;
  const int64_t most = 16 * most_row_blocks(D), tiles = ceil_div(rows, most);
  return tiles * most * kLargeTile < ceil_div(rows, 32) * 32 && tiles * heads >= cus ? most_row_blocks(D) : 2;
}

fp8layer::Divisor divisor(int d) {
  const int log = d > 1 ? 32 - __builtin_clz(d - 1) : 0;  // ceil(log2 d)
  return {(uint32_t)((((uint64_t)1 << (31 + log)) + d - 1) / d), (uint32_t)(31 + log)};
}

constexpr size_t kAttentionCounterBytes = fp8layer::kCounters * sizeof(int32_t);
constexpr size_t kAttentionPartBytes = (size_t)64 << 20;

}  // namespace

extern "C" {

int fp8_rmsnorm_quantize_1x128(const void* X, int64_t ldx, const void* R, int64_t ldr, int x_dtype, const void* w,
                               int w_dtype, float eps, void* H, int64_t ldh, void* Y, int64_t ldy, float* rstd,
                               void* Q, int64_t ldq, float* sa, int64_t ld_sa, int M, int K, hipStream_t stream) {
  if (!w || (M != 0 && (!X || !Q || !sa || (R && !H)))) return FP8GEMM_ERR_NULL;
  if (M < 0 || K <= 0 || K % 128 != 0 || K > kMaxNormCols || !(eps >= 0.f)) return FP8GEMM_ERR_SHAPE;
  if (!norm_dtype(x_dtype) || !norm_dtype(w_dtype)) return FP8GEMM_ERR_LAYOUT;
  if (M == 0) return FP8GEMM_OK;
  if (!norm_rows(X, ldx, K, x_dtype) || !aligned(w, 16)) return FP8GEMM_ERR_LAYOUT;
  if (R && (!norm_rows(R, ldr, K, x_dtype) || !norm_rows(H, ldh, K, x_dtype))) return FP8GEMM_ERR_LAYOUT;
  if (Y && !norm_rows(Y, ldy, K, FP8GEMM_QUANT_BF16)) return FP8GEMM_ERR_LAYOUT;
  if (!aligned(Q, 8) || ldq < K || ldq % 8 != 0 || !aligned(sa, 4) || ld_sa < M || ld_sa % 4 != 0 || !aligned(rstd, 4))
    return FP8GEMM_ERR_LAYOUT;
  int cus;
  const int st = device(&cus);
  if (st != FP8GEMM_OK) return st;
  fp8layer::NormParams p{X,   R,   w,   H,   Y,   rstd,  static_cast<uint8_t*>(Q), sa, ldx,
                         ldr, ldh, ldy, ldq, ld_sa, eps, M, K, w_dtype == FP8GEMM_QUANT_FP32, 0};
  with_type(x_dtype, [&](auto t) {
    with_flag(streams(M, K, sizeof(t) * (R ? 2 : 1)), [&](auto nt) {
      with_shape(norm_shape(M, K, cus), [&](auto waves, auto chunks) {
        constexpr int kWaves = decltype(waves)::value;
        constexpr int kRows = kWaves > 4 ? 1 : 4 / kWaves, kThreads = kWaves > 4 ? kWaves * 64 : 256;
        in_slices(ceil_div(M, kRows), kThreads, [&](int first, dim3 groups) {
          p.first_group = first;
          hipLaunchKernelGGL((fp8layer::rmsnorm_quantize_kernel<decltype(t), kWaves, decltype(chunks)::value, decltype(nt)::value>),
                             groups, dim3(kThreads), 0, stream, p);
        });
      });
    });
  });
  return launched();
}

size_t fp8_rmsnorm_backward_workspace_size(int M, int K) {
  if (M <= 0 || K <= 0 || K % 128 != 0 || K > kMaxNormCols) return 0;
  int cus;  // without a device: the MI355X's own count
  if (device(&cus) != FP8GEMM_OK) cus = 256;
  return (size_t)norm_grad_groups(M, norm_grad_shape(K), cus) * K * sizeof(float);
}

int fp8_rmsnorm_backward(const void* dY, int64_t lddy, const void* H, int64_t ldh, const void* dH, int64_t lddh,
                         int dtype, const float* rstd, const void* w, int w_dtype, void* dX, int64_t lddx, float* dW,
                         int M, int K, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!w || !dW || (M != 0 && (!dY || !H || !rstd || !dX))) return FP8GEMM_ERR_NULL;
  if (M < 0 || K <= 0 || K % 128 != 0 || K > kMaxNormCols) return FP8GEMM_ERR_SHAPE;
  if (!norm_dtype(dtype) || !norm_dtype(w_dtype)) return FP8GEMM_ERR_LAYOUT;
  if (M != 0 && (!norm_rows(dY, lddy, K, dtype) || !norm_rows(H, ldh, K, dtype) || !norm_rows(dX, lddx, K, dtype) ||
                 (dH && !norm_rows(dH, lddh, K, dtype)) || !aligned(rstd, 4)))
    return FP8GEMM_ERR_LAYOUT;
  if (!aligned(w, 16) || !aligned(dW, 4) || !aligned(workspace, 16)) return FP8GEMM_ERR_LAYOUT;
  int cus;
  const int st = device(&cus);
  if (st != FP8GEMM_OK) return st;
  const NormShape s = norm_grad_shape(K);
  const int groups = M > 0 ? norm_grad_groups(M, s, cus) : 0;
  if (groups > 0 && (!workspace || workspace_bytes < (size_t)groups * K * sizeof(float))) return FP8GEMM_ERR_WORKSPACE;
  float* part = static_cast<float*>(workspace);
  const size_t size = dtype == FP8GEMM_QUANT_BF16 ? 2 : 4, row_bytes = size * (dH ? 3 : 2);
  if (M > 0 && norm_grad_few(M, K, row_bytes, dtype == FP8GEMM_QUANT_FP32, cus) && !rows_meet(dX, lddx, dY, lddy, M, K, size) &&
      !rows_meet(dX, lddx, H, ldh, M, K, size)) {
    const fp8layer::NormGradParams p{dY, H, dH, w, rstd, dX, nullptr, lddy, ldh, lddh, lddx, M, K, w_dtype == FP8GEMM_QUANT_FP32};
    with_type(dtype, [&](auto t) {
      auto go = [&](auto waves) {
        constexpr int kWaves = decltype(waves)::value;
        hipLaunchKernelGGL((fp8layer::rmsnorm_backward_few_kernel<decltype(t), kWaves>),
                           dim3((unsigned)(K * (int)sizeof(t) / 128 + ceil_div(M, 16 / kWaves))), dim3(1024), 0, stream, p, dW);
      };
      const int waves = norm_shape(M, K, cus).waves;
      if (waves == 1) go(Int<1>{});
      else if (waves == 4) go(Int<4>{});
      else go(Int<16>{});
    });
    return launched();
  }
  if (M > 0) {
    const fp8layer::NormGradParams p{dY, H, dH, w, rstd, dX, part, lddy, ldh, lddh, lddx, M, K, w_dtype == FP8GEMM_QUANT_FP32};
    const size_t merge = (size_t)(16 / s.waves - 1) * K * sizeof(float);  // at most 30 KB
    with_type(dtype, [&](auto t) {
      with_flag(streams(M, K, row_bytes), [&](auto nt) {
        with_grad_shape(s, [&](auto waves, auto chunks) {
          hipLaunchKernelGGL(
              (fp8layer::rmsnorm_backward_kernel<decltype(t), decltype(waves)::value, decltype(chunks)::value, decltype(nt)::value>),
              dim3(groups), dim3(1024), merge, stream, p);
        });
      });
    });
    const int rc = launched();
    if (rc != FP8GEMM_OK) return rc;
  }
  hipLaunchKernelGGL(fp8layer::rmsnorm_weight_grad_kernel, dim3((unsigned)(K / 16)), dim3(256), 0, stream, part,
                     groups, K, dW);
  return launched();
}

int fp8_rope_append_paged_kv(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                             const float* cos_sin, int64_t ld_cs, int max_pos, int rot_dim, int interleaved,
                             const int32_t* positions, const int32_t* block_table, int64_t ld_bt, int max_pages,
                             const int32_t* seq_lens, const int32_t* cu_q, void* q_out, int64_t ldqo, void* k_cache,
                             float* k_scale, void* v_cache, float* v_scale, int num_pages, int P, int B, int T, int Hq,
                             int Hkv, int D, hipStream_t stream) {
  if (!k_cache || !k_scale || !v_cache || !v_scale ||
      (T != 0 && B != 0 && (!k || !v || (max_pages > 0 && !block_table) || !seq_lens || !cu_q || (q == nullptr) != (q_out == nullptr) ||
                            (rot_dim > 0 && !cos_sin))))
    return FP8GEMM_ERR_NULL;
  if (!cache_shape(num_pages, P, Hkv, D) || B < 0 || T < 0 || Hq < 1 || max_pages < 0 || rot_dim < 0 || rot_dim > D ||
      rot_dim % 16 != 0 || (rot_dim > 0 && max_pos < 1) || (int64_t)T * std::max(Hq, Hkv) >= INT32_MAX - 256 ||
      (int64_t)std::max(Hq, Hkv) * D > INT32_MAX || (int64_t)max_pages * P > INT32_MAX)
    return FP8GEMM_ERR_SHAPE;
  if (B == 0 || T == 0) return FP8GEMM_OK;
  if (ldk < (int64_t)Hkv * D || ldk % 8 || ldv < (int64_t)Hkv * D || ldv % 8 || ld_bt < max_pages ||
      (q && (ldq < (int64_t)Hq * D || ldq % 8 || ldqo < (int64_t)Hq * D || ldqo % 8)) ||
      (rot_dim > 0 && (ld_cs < rot_dim || ld_cs % 4)))
    return FP8GEMM_ERR_LAYOUT;
  if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(cos_sin, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) ||
      !aligned(positions, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_q, 4))
    return FP8GEMM_ERR_LAYOUT;
  int cus;
  const int st = device(&cus);
  if (st != FP8GEMM_OK) return st;
  // Most pages that T new tokens of B sequences can fall in: whole pages, and an end of a
  // page on either side for each sequence that has any.
  const int64_t pages = std::min<int64_t>(T, ceil_div(T, P) + 2 * (int64_t)std::min(B, T));
  const int64_t units = pages * Hkv * 2;
  // A wave for each unit where its registers hold a sequence's new tokens, or pages are small,
  // and units are many; four otherwise. Heads of 128, one wave and four: 64 users' single
  // tokens 4.5 and 5.3 us, 16 tokens each 6.8 and 8.4, 32 each 11.2 both; 8 users' 16 tokens
  // 5.0 and 4.2; prompts in pages of 16, 32 and 64 40 and 56, 49 and 53, 50 and 47 us.
  const bool small = units > 2 * cus && ((int64_t)T * D <= (int64_t)fp8layer::kHeld * 64 * 16 * B || P * D <= 4096);
  const int64_t unit_groups = small ? ceil_div(units, 4) : units;
  // Queries: a token a workgroup; two where that still leaves several rounds of workgroups,
  // the second's in flight while the first is turned (8636 tokens by 32 heads of 128, with
  // keys and values of 8 heads: 46.5 us by one token, 45.0 by two, 46.4 by four, 51 by eight).
  const int group_tokens = T >= 8 * cus ? 2 : 1;
  const int64_t q_groups = q ? ceil_div(T, group_tokens) : 0;
  if (unit_groups + q_groups > INT32_MAX) return FP8GEMM_ERR_SHAPE;
  fp8layer::AppendParams p{static_cast<const uint16_t*>(q),
                           static_cast<const uint16_t*>(k),
                           static_cast<const uint16_t*>(v),
                           cos_sin,
                           positions,
                           block_table,
                           seq_lens,
                           cu_q,
                           static_cast<uint16_t*>(q_out),
                           static_cast<uint8_t*>(k_cache),
                           static_cast<uint8_t*>(v_cache),
                           k_scale,
                           v_scale,
                           ldq,
                           ldk,
                           ldv,
                           ld_cs,
                           ld_bt,
                           ldqo,
                           max_pos,
                           rot_dim,
                           interleaved ? 1 : 0,
                           max_pages,
                           num_pages,
                           log2_of(P),
                           B,
                           T,
                           Hq,
                           Hkv,
                           (int)unit_groups,
                           group_tokens,
                           0};
  auto go = [&](auto d) {
    constexpr int kD = decltype(d)::value;
    with_flag(streams(T, ((q ? Hq : 0) + 2 * (int64_t)Hkv) * D, sizeof(uint16_t)), [&](auto nt) {
      constexpr bool kStream = decltype(nt)::value;
      in_slices(unit_groups + q_groups, 256, [&](int first, dim3 groups) {
        p.first_group = first;
        if (small)
          hipLaunchKernelGGL((fp8layer::rope_append_kernel<kD, 1, kStream>), groups, dim3(256), 0, stream, p);
        else
          hipLaunchKernelGGL((fp8layer::rope_append_kernel<kD, 4, kStream>), groups, dim3(256), 0, stream, p);
      });
    });
  };
  if (D == 64) go(Int<64>{});
  else if (D == 128) go(Int<128>{});
  else go(Int<256>{});
  return launched();
}

size_t fp8_paged_attention_workspace_size(void) { return kAttentionCounterBytes + kAttentionPartBytes; }

int fp8_paged_attention(const void* q, int64_t ldq, const void* k_cache, const float* k_scale, const void* v_cache,
                        const float* v_scale, int num_pages, int P, const int32_t* block_table, int64_t ld_bt,
                        int max_pages, const int32_t* seq_lens, const int32_t* cu_q, void* O, int64_t ldo, float* lse,
                        float softmax_scale, int window, int B, int T, int Hq, int Hkv, int D, void* workspace,
                        size_t workspace_bytes, hipStream_t stream) {
  if (!k_cache || !k_scale || !v_cache || !v_scale ||
      (T != 0 && B != 0 && (!q || (max_pages > 0 && !block_table) || !seq_lens || !cu_q || !O)))
    return FP8GEMM_ERR_NULL;
  if (!cache_shape(num_pages, P, Hkv, D) || B < 0 || T < 0 || Hq < 1 || Hq % Hkv != 0 || max_pages < 0 || window < 0 ||
      !std::isfinite(softmax_scale) || (int64_t)T * Hq >= INT32_MAX - 256 || (int64_t)Hq * D > INT32_MAX ||
      (int64_t)max_pages * P > fp8layer::kMostKeys)
    return FP8GEMM_ERR_SHAPE;
  if (B == 0 || T == 0) return FP8GEMM_OK;
  if (ldq < (int64_t)Hq * D || ldq % 8 || ldo < (int64_t)Hq * D || ldo % 8 || ld_bt < max_pages) return FP8GEMM_ERR_LAYOUT;
  if (!aligned(q, 16) || !aligned(O, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 4) ||
      !aligned(v_scale, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_q, 4) || !aligned(lse, 4) ||
      !aligned(workspace, 16))
    return FP8GEMM_ERR_LAYOUT;
  int cus;
  const int st = device(&cus);
  if (st != FP8GEMM_OK) return st;
  const int max_len = max_pages * P;
  fp8layer::AttentionParams p{};
  p.q = static_cast<const uint16_t*>(q);
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.cu_q = cu_q;
  p.O = static_cast<uint16_t*>(O);
  p.lse = lse;
  p.ldq = ldq;
  p.ldo = ldo;
  p.ld_bt = ld_bt;
  p.scale_log2 = std::fabs(softmax_scale) * 1.4426950408889634f;
  p.q_sign = softmax_scale < 0.f ? 0x80008000u : 0u;
  p.window = window;
  p.B = B;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.group = Hq / Hkv;
  p.by_group = divisor(p.group);
  p.by_heads = divisor(Hkv);
  p.num_pages = num_pages;
  p.log_p = log2_of(P);
  p.max_pages = max_pages;
  const int64_t rows = ceil_div((int64_t)T * p.group, B);  // that share a key head, on average
  const int blocks = attention_row_blocks(rows, (int64_t)B * Hkv, D, cus);
  const int tile = 16 * blocks;
  const bool stream_kv = rows <= tile;  // the tile is the only reader of its keys and values
  // Most row tiles, times heads. Splitting adds units up to a number that gives every CU
  // a few: that many are wanted, and the workspace has a slot for each unit.
  const int64_t tiles = (std::min(B, T) + (int64_t)T * p.group / tile) * Hkv;
  const size_t slot = (size_t)tile * (D + 1) * sizeof(float);
  const size_t bytes = std::min<size_t>(workspace ? workspace_bytes : 0, (size_t)1 << 30);
  const int64_t slots = bytes > kAttentionCounterBytes ? (int64_t)((bytes - kAttentionCounterBytes) / slot) : 0;
  p.cus = cus;
  // Units that splitting may add: one for each CU where the longest sequences that the table
  // allows are little work, four otherwise (workgroups without a unit end at once, but 512 of
  // them cost a microsecond).
  const int64_t most_keys = tiles * max_len;
  const int64_t rounds = most_keys <= (int64_t)kFewKeys * cus ? 1 : 4;
  const int64_t added = std::min(rounds * cus, std::min<int64_t>(slots, fp8layer::kPartCounters) - tiles);
  int64_t grid = tiles;
  if (tiles <= fp8layer::kTileCounters && added > 0 && max_len > fp8layer::kMinChunk) {
    p.most_units = (int)added;
    p.counters = static_cast<int32_t*>(workspace);
    p.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + kAttentionCounterBytes);
    grid = std::min(tiles + added, tiles * ceil_div(max_len, fp8layer::kMinChunk));
  }
  if (grid > INT32_MAX) return FP8GEMM_ERR_SHAPE;
  auto go = [&](auto d) {
    constexpr int kD = decltype(d)::value;
    constexpr int kMost = most_row_blocks(kD);
    in_slices(grid, 256, [&](int first, dim3 groups) {
      p.first_unit = first;
      if (blocks == 1) {
        hipLaunchKernelGGL((fp8layer::attention_kernel<kD, 1, true, false>), groups, dim3(256), 0, stream, p);
      } else if (stream_kv) {
        hipLaunchKernelGGL((fp8layer::attention_kernel<kD, 2, true, false>), groups, dim3(256), 0, stream, p);
      } else {
        with_flag(P >= 32, [&](auto w) {
          constexpr bool kWide = decltype(w)::value;
          if (blocks == 2) hipLaunchKernelGGL((fp8layer::attention_kernel<kD, 2, false, kWide>), groups, dim3(256), 0, stream, p);
          else hipLaunchKernelGGL((fp8layer::attention_kernel<kD, kMost, false, kWide>), groups, dim3(256), 0, stream, p);
        });
      }
    });
  };
  if (D == 64) go(Int<64>{});
  else if (D == 128) go(Int<128>{});
  else go(Int<256>{});
  return launched();
}

}  // extern "C"
