// Host side of the expert and head operators of libfp8gemm (include/fp8moe.h): argument checks,
// the choice among compiled instances, and the launches.
#include "fp8moe.h"

#include <cmath>

#include "host.hpp"
#include "combine_kernel.hpp"
#include "dispatch_kernel.hpp"
#include "heads_kernel.hpp"
#include "route_kernel.hpp"

namespace {

using fp8moe::kAlign;
using fp8moe::kMaxExperts;
using fp8moe::kPiece;

constexpr int kMaxChoices = 64;               // of a token: a lane holds one
constexpr int64_t kMost = INT32_MAX - (1 << 18);  // choices and rows, so that segments' ends fit 32 bits

// Weights are scaled by scale / (sum of scores + 1e-20), which has to be a number.
bool route_scale(float scale) { return std::fabs(scale) <= 0x1p60f; }
bool route_shape(int T, int E, int top_k) { return T >= 0 && E >= 1 && E <= kMaxExperts && top_k >= 1 && top_k <= std::min(E, kMaxChoices); }
bool rows_dtype(int t) { return norm_dtype(t); }
// row stride of a [.., E] array of `size`-byte elements that are read one by one
bool narrow_rows(const void* p, int64_t ld, int E, size_t size) { return aligned(p, size) && ld >= E; }
size_t size_of(int dtype) { return dtype == FP8GEMM_QUANT_BF16 ? 2 : 4; }

// Calls f with the first of some counts in rising order that is not below n, or the last, as a
// compile-time value.
template <int V, int... MORE, typename F>
void with_count(int n, F f) {
  if constexpr (sizeof...(MORE) > 0) {
    if (n > V) return with_count<MORE...>(n, f);
  }
  f(Int<V>{});
}

}  // namespace

extern "C" {

int fp8_moe_route(const void* logits, int64_t ldl, int dtype, const float* bias, int scoring, int groups, int top_groups,
                  int group_best, int renormalize, float scale, int32_t* ids, float* weights, float* scores, int64_t lds,
                  int T, int E, int top_k, hipStream_t stream) {
  if (T != 0 && (!logits || !ids || !weights)) return FP8GEMM_ERR_NULL;
  if (!route_shape(T, E, top_k) || groups < 1 || groups > 64 || E % groups != 0 || top_groups < 1 || top_groups > groups ||
      (group_best != 1 && group_best != 2) || !route_scale(scale))
    return FP8GEMM_ERR_SHAPE;
  if (!rows_dtype(dtype) || (scoring != FP8MOE_SOFTMAX && scoring != FP8MOE_SIGMOID)) return FP8GEMM_ERR_LAYOUT;
  if (T == 0) return FP8GEMM_OK;
  if (!narrow_rows(logits, ldl, E, size_of(dtype)) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4) ||
      (scores && !narrow_rows(scores, lds, E, 4)))
    return FP8GEMM_ERR_LAYOUT;
  int cus;
  const int st = device(&cus);
  if (st != FP8GEMM_OK) return st;
  int log_groups = 0;
  while ((1 << log_groups) < groups) ++log_groups;
  const int log_lanes = 6 - log_groups, size = E / groups, each = (int)ceil_div(size, 1 << log_lanes);
  fp8moe::RouteParams p{logits, bias,       ids,        weights,    scores,      ldl,         lds,  scale,     T,    E,
                        top_k,  groups,     top_groups, group_best, scoring == FP8MOE_SIGMOID, renormalize != 0, size, log_lanes, each,
                        0,      0,          0};
  // Experts of a lane where 16 lanes hold a row, and a group some of them. A wave for four rows
  // shares most instructions among them, and needs many rows to fill the GPU; there has to be a
  // lane for each choice and one more. For four rows and for one, FP32 logits of deviation 1.5 that the
  // caches hold, sigmoid with a bias, calls of a graph, us: 16 experts, 1 token 2.3 and 2.6, 16384 3.3
  // and 8.1; 32, 1 token 2.9 and 2.6, 16384 7.5 and 9.2, in 4 groups 4096 7.0 and 5.1, 16384 7.2 and
  // 10.3; 64, 4096 5.0 and 4.8, 8192 5.1 and 6.5, 16384 6.2 and 9.0, 65536 13.9 and 26.7; 256, 8192
  // 8.2 and 7.1, 16384 10.5 and 11.1, 65536 26.8 and 33.7, in 8 groups 8192 8.4 and 8.4, 16384 11.6
  // and 13.7, 65536 33.4 and 44.1. Cold logits of 16384 x 256: 12.3 and 12.1, in 8 groups 14.6 and 15.0.
  // Other rows, of which FP32 leaves others open, move these by up to 3.
  const int of_16 = log_groups <= 4 ? (int)ceil_div(size, 1 << (log_lanes - 2)) : 0;
  const bool four_rows = of_16 == 1 || (of_16 == 2 && T > 32 * cus) ||
                         (of_16 > 2 && of_16 <= 16 && top_k <= 15 && T >= (of_16 <= 4 ? 32 : 64) * cus);
  with_type(dtype, [&](auto t) {
    if (four_rows) {
      with_count<1, 2, 4, 8, 16>(of_16, [&](auto count) {
        constexpr int kCount = decltype(count)::value;
        p.even = size == (kCount + 3) / 4 << log_lanes && groups == 1 << log_groups;
        p.even_16 = size == kCount << (log_lanes - 2) && groups == 1 << log_groups;
        in_slices(ceil_div(T, 16), 256, [&](int first, dim3 grid) {
          p.first_group = first;
          hipLaunchKernelGGL((fp8moe::route_rows_kernel<decltype(t), kCount>), grid, dim3(256), 0, stream, p);
        });
      });
      return;
    }
    with_count<1, 2, 3, 4, 6, 8, 16, 32>(each, [&](auto count) {
      p.even = size == decltype(count)::value << log_lanes && groups == 1 << log_groups;
      in_slices(ceil_div(T, 4), 256, [&](int first, dim3 grid) {
        p.first_group = first;
        hipLaunchKernelGGL((fp8moe::route_kernel<decltype(t), decltype(count)::value>), grid, dim3(256), 0, stream, p);
      });
    });
  });
  return launched();
}

int fp8_moe_route_backward(const float* dweights, const void* logits, int64_t ldl, int dtype, const int32_t* ids, int scoring,
                           int renormalize, float scale, const float* dscores, int64_t ldds, void* dlogits, int64_t lddl,
                           int T, int E, int top_k, hipStream_t stream) {
  if (T != 0 && (!dweights || !logits || !ids || !dlogits)) return FP8GEMM_ERR_NULL;
  if (!route_shape(T, E, top_k) || !route_scale(scale)) return FP8GEMM_ERR_SHAPE;
  if (!rows_dtype(dtype) || (scoring != FP8MOE_SOFTMAX && scoring != FP8MOE_SIGMOID)) return FP8GEMM_ERR_LAYOUT;
  if (T == 0) return FP8GEMM_OK;
  if (!narrow_rows(logits, ldl, E, size_of(dtype)) || !narrow_rows(dlogits, lddl, E, size_of(dtype)) || !aligned(ids, 4) ||
      !aligned(dweights, 4) || (dscores && !narrow_rows(dscores, ldds, E, 4)))
    return FP8GEMM_ERR_LAYOUT;
  int cus;
  const int st = device(&cus);
  if (st != FP8GEMM_OK) return st;
  fp8moe::RouteGradParams p{dweights, dscores, logits, ids, dlogits, ldl, ldds, lddl, scale, T, E, top_k, scoring == FP8MOE_SIGMOID,
                            renormalize != 0, 0};
  with_type(dtype, [&](auto t) {
    auto go = [&](auto count, auto lanes) {
      constexpr int kLanes = decltype(lanes)::value;
      in_slices(ceil_div(T, 256 / kLanes), 256, [&](int first, dim3 grid) {
        p.first_group = first;
        hipLaunchKernelGGL((fp8moe::route_backward_kernel<decltype(t), decltype(count)::value, kLanes>), grid, dim3(256), 0, stream, p);
      });
    };
    // A lane holds a choice: four rows a wave where 16 lanes are enough for that and for a few experts.
    // With 16 lanes a row and with 64, BF16 softmax and a gradient of the scores, us: 16 experts, 1000
    // rows 2.5 and 2.6, 16384 3.2 and 6.0; 64, 1000 2.7 and 2.5, 16384 3.7 and 6.1, 65536 9.1 and 20.0; 96,
    // 1000 3.0 and 2.5, 10007 3.8 and 4.6; 160, 4096 3.7 and 3.3, 10007 4.8 and 5.2, 65536 17.0 and 23.5;
    // 256, 4096 4.3 and 3.8, 16384 7.6 and 8.6. Past 64 experts 16 lanes lose on few rows; what they gain
    // on many is not taken.
    if (E <= 64 && top_k <= 16) with_count<1, 2, 4>((int)ceil_div(E, 16), [&](auto count) { go(count, Int<16>{}); });
    else with_count<1, 2, 3, 4, 6, 8, 12, 16>((int)ceil_div(E, 64), [&](auto count) { go(count, Int<64>{}); });
  });
  return launched();
}

int64_t fp8_moe_rows(int T, int top_k, int E) {
  if (T < 0 || top_k < 1 || top_k > kMaxChoices || E < 1 || E > kMaxExperts) return 0;
  const int64_t n = (int64_t)T * top_k;
  return n > kMost ? 0 : (n + std::min<int64_t>(n, E) * (kAlign - 1)) / kAlign * kAlign;
}

}  // extern "C"

namespace {

// Choices up to which every placing workgroup counts them all itself, and the counting launch
// and the one that adds up are saved.
constexpr int kCountedByAll = 65536;
// Whether layout and rows are one launch, in which every workgroup counts all choices for itself
// and copies the rows of a token or a few. In one and in two: 600 tokens of 8 choices and 1024
// columns 8.4 and 11.0 us, 1000 of 7168 columns 20.1 and 19.9; 2000 of 4 choices 9.0 and 8.4, 5453
// of one 12.1 and 10.5.
bool few_choices(int T, int n) { return n <= 4096 || (n <= 8192 && T <= 1024); }
constexpr int kFewGroups = 512;  // that their tokens are cut into

bool gather_layout(const void* Q, int64_t ldq, const float* sa, int64_t ld_sa, const float* weights, const void* Qx, int64_t ldqx,
                   const float* sax, int64_t ld_sax, int64_t rows, int max_m, int T, int K) {
  const int64_t columns = max_m ? max_m : rows;
  return aligned(Q, 16) && ldq >= K && ldq % 16 == 0 && aligned(sa, 4) && ld_sa >= T && ld_sa % 4 == 0 && aligned(weights, 4) &&
         aligned(Qx, 16) && ldqx >= K && ldqx % 16 == 0 && aligned(sax, 4) && ld_sax >= columns && ld_sax % 4 == 0;
}
bool dispatch_shape(int64_t rows, int max_m, int T, int top_k, int E) {
  return T >= 0 && top_k >= 1 && top_k <= kMaxChoices && (int64_t)T * top_k <= kMost && rows >= 0 && rows <= kMost && max_m >= 0 &&
         (max_m ? E >= 1 && E <= kMaxExperts && rows == (int64_t)E * max_m : rows % kAlign == 0);
}
bool gather_cols(int K) { return K >= 128 && K % 128 == 0 && K <= 65536; }

fp8moe::GatherParams gather_params(const void* Q, int64_t ldq, const float* sa, int64_t ld_sa, const float* weights, void* Qx,
                                   int64_t ldqx, float* sax, int64_t ld_sax, const int32_t* positions, const int32_t* sources,
                                   int64_t rows, int max_m, int T, int top_k, int E, int K) {
  return {static_cast<const uint8_t*>(Q), sa, weights, static_cast<uint8_t*>(Qx), sax, positions, sources, ldq, ld_sa,
          ldqx, ld_sax, rows, max_m, T, top_k, E, K, (int)ceil_div(K, fp8moe::kSlice), 0, (int)ceil_div(max_m ? max_m : rows, 64), 0};
}
int gather(fp8moe::GatherParams p, hipStream_t stream) {
  auto go = [&](auto lanes) -> int {
    constexpr int kLanes = decltype(lanes)::value;
    p.code_groups = kLanes < 64 ? ceil_div(p.T, 256 / kLanes) : ceil_div((int64_t)p.T * p.slices, 4);
    const int64_t scale_units = (p.max_m ? p.E : 1) * (int64_t)p.row_groups * ceil_div(p.K / 128, fp8moe::kScaleBlocks);
    const int64_t all = p.code_groups + ceil_div(scale_units, 4);
    if (all > INT32_MAX) return FP8GEMM_ERR_SHAPE;
    in_slices(all, 256, [&](int first, dim3 grid) {
      p.first_group = first;
      hipLaunchKernelGGL(fp8moe::gather_kernel<kLanes>, grid, dim3(256), 0, stream, p);
    });
    return launched();
  };
  // lanes of 16 bytes: as many as a row has, where a wave can take several rows
  if (p.K <= 128) return go(Int<8>{});
  if (p.K <= 256) return go(Int<16>{});
  if (p.K <= 512) return go(Int<32>{});
  return go(Int<64>{});
}

}  // namespace

extern "C" {

size_t fp8_moe_dispatch_workspace_size(int T, int top_k, int E) {
  if (T < 0 || top_k < 1 || top_k > kMaxChoices || E < 1 || E > kMaxExperts) return 0;
  const int64_t n = (int64_t)T * top_k;
  return n <= kCountedByAll || n > kMost ? 0 : (size_t)(ceil_div(n, kPiece) + 1) * E * sizeof(int32_t);
}

int fp8_moe_dispatch(const void* Q, int64_t ldq, const float* sa, int64_t ld_sa, const int32_t* ids, const float* weights, void* Qx,
                     int64_t ldqx, float* sax, int64_t ld_sax, int32_t* positions, int32_t* sources, int32_t* m_indices,
                     int32_t* counts, int64_t rows, int max_m, int T, int top_k, int E, int K, void* workspace,
                     size_t workspace_bytes, hipStream_t stream) {
  if (!counts || (T != 0 && (!ids || !positions)) || (rows != 0 && (!sources || (max_m == 0 && !m_indices))) ||
      (Q && T != 0 && rows != 0 && (!sa || !Qx || !sax)))
    return FP8GEMM_ERR_NULL;
  if (E < 1 || E > kMaxExperts || !dispatch_shape(rows, max_m, T, top_k, E) || (Q && !gather_cols(K))) return FP8GEMM_ERR_SHAPE;
  if (!aligned(ids, 4) || !aligned(positions, 4) || !aligned(sources, 4) || !aligned(m_indices, 4) || !aligned(counts, 4) ||
      !aligned(workspace, 16))
    return FP8GEMM_ERR_LAYOUT;
  const bool moves = Q && T != 0 && rows != 0;
  if (moves && !gather_layout(Q, ldq, sa, ld_sa, weights, Qx, ldqx, sax, ld_sax, rows, max_m, T, K)) return FP8GEMM_ERR_LAYOUT;
  int cus;
  const int st = device(&cus);
  if (st != FP8GEMM_OK) return st;
  const size_t need = fp8_moe_dispatch_workspace_size(T, top_k, E);
  if (need && (!workspace || workspace_bytes < need)) return FP8GEMM_ERR_WORKSPACE;
  const int n = T * top_k;
  int bits = 0;
  while ((1 << bits) < E) ++bits;
  const fp8moe::LayoutParams p{ids,  static_cast<int32_t*>(workspace), positions, sources, m_indices, counts, rows, n, E, bits, max_m,
                               std::max(1, (int)ceil_div(n, kPiece))};
  const fp8moe::GatherParams copy =
      gather_params(Q, ldq, sa, ld_sa, weights, Qx, ldqx, sax, ld_sax, positions, sources, rows, max_m, T, top_k, E, moves ? K : 0);
  if (moves && few_choices(T, n)) {  // then a group's tokens have at most kFewChoices
    fp8moe::FewParams f{p, copy, (int)ceil_div(T, kFewGroups), 1, K};
    const int groups = (int)ceil_div(T, f.tokens);
    // slices of 4096 columns (16 a thread) where that gives more CUs a part
    f.slices = (int)std::min<int64_t>(ceil_div(K, 4096), std::max(1, kFewGroups / groups));
    f.slice = (int)ceil_div(ceil_div(K, f.slices), 128) * 128;
    hipLaunchKernelGGL(fp8moe::dispatch_few_kernel, dim3(groups * f.slices), dim3(256), 0, stream, f);
    return launched();
  }
  if (need) {
    hipLaunchKernelGGL(fp8moe::count_kernel, dim3(p.pieces), dim3(kPiece), 0, stream, p);
    hipLaunchKernelGGL(fp8moe::scan_kernel, dim3((unsigned)ceil_div(E, 64)), dim3(1024), 0, stream, p);
    hipLaunchKernelGGL(fp8moe::place_kernel<false>, dim3(p.pieces), dim3(kPiece), 0, stream, p);
  } else {
    hipLaunchKernelGGL(fp8moe::place_kernel<true>, dim3(p.pieces), dim3(kPiece), 0, stream, p);
  }
  const int rc = launched();
  return rc != FP8GEMM_OK || !moves ? rc : gather(copy, stream);
}

int fp8_moe_gather(const void* Q, int64_t ldq, const float* sa, int64_t ld_sa, const float* weights, void* Qx, int64_t ldqx,
                   float* sax, int64_t ld_sax, const int32_t* positions, const int32_t* sources, int64_t rows, int max_m, int T,
                   int top_k, int E, int K, hipStream_t stream) {
  if (T != 0 && rows != 0 && (!Q || !sa || !Qx || !sax || !positions || !sources)) return FP8GEMM_ERR_NULL;
  if (!dispatch_shape(rows, max_m, T, top_k, E) || !gather_cols(K)) return FP8GEMM_ERR_SHAPE;
  if (T == 0 || rows == 0) return FP8GEMM_OK;
  if (!aligned(positions, 4) || !aligned(sources, 4) ||
      !gather_layout(Q, ldq, sa, ld_sa, weights, Qx, ldqx, sax, ld_sax, rows, max_m, T, K))
    return FP8GEMM_ERR_LAYOUT;
  int cus;
  const int st = device(&cus);
  if (st != FP8GEMM_OK) return st;
  return gather(gather_params(Q, ldq, sa, ld_sa, weights, Qx, ldqx, sax, ld_sax, positions, sources, rows, max_m, T, top_k, E, K), stream);
}

}  // extern "C"

namespace {

bool combine_shape(int64_t rows, int T, int top_k, int N) {
  return T >= 0 && top_k >= 1 && top_k <= kMaxChoices && rows >= 0 && rows <= INT32_MAX && N >= 8 && N % 8 == 0;
}

}  // namespace

extern "C" {

int fp8_moe_combine(const void* Y, int64_t ldy, int dtype, const int32_t* positions, const float* weights, const void* C, int64_t ldc,
                    void* out, int64_t ldo, int64_t rows, int T, int top_k, int N, hipStream_t stream) {
  if (T != 0 && ((rows != 0 && !Y) || !positions || !out)) return FP8GEMM_ERR_NULL;
  if (!combine_shape(rows, T, top_k, N)) return FP8GEMM_ERR_SHAPE;
  if (!rows_dtype(dtype)) return FP8GEMM_ERR_LAYOUT;
  if (T == 0) return FP8GEMM_OK;
  if ((rows != 0 && !norm_rows(Y, ldy, N, dtype)) || !norm_rows(out, ldo, N, dtype) || (C && !norm_rows(C, ldc, N, dtype)) ||
      !aligned(positions, 4) || !aligned(weights, 4))
    return FP8GEMM_ERR_LAYOUT;
  int cus;
  const int st = device(&cus);
  if (st != FP8GEMM_OK) return st;
  fp8moe::CombineParams p{Y, C, out, positions, weights, ldy, ldc, ldo, rows, T, top_k, N, (int)ceil_div(N, 512), 0};
  const int64_t groups = ceil_div((int64_t)T * p.slices, 4);
  if (groups > INT32_MAX) return FP8GEMM_ERR_SHAPE;
  with_type(dtype, [&](auto t) {
    with_flag(streams(T, (int64_t)N * top_k, sizeof(t)), [&](auto nt) {
      in_slices(groups, 256, [&](int first, dim3 grid) {
        p.first_group = first;
        hipLaunchKernelGGL((fp8moe::combine_kernel<decltype(t), decltype(nt)::value>), grid, dim3(256), 0, stream, p);
      });
    });
  });
  return launched();
}

int fp8_moe_combine_backward(const void* dO, int64_t lddo, const void* Y, int64_t ldy, int dtype, const int32_t* positions,
                             const float* weights, void* dY, int64_t lddy, float* dweights, int64_t rows, int T, int top_k, int N,
                             hipStream_t stream) {
  if (T != 0 && (!dO || (rows != 0 && !Y) || !positions || !weights || !dweights)) return FP8GEMM_ERR_NULL;
  if (!combine_shape(rows, T, top_k, N)) return FP8GEMM_ERR_SHAPE;
  if (!rows_dtype(dtype)) return FP8GEMM_ERR_LAYOUT;
  if (T == 0) return FP8GEMM_OK;
  if (!norm_rows(dO, lddo, N, dtype) || (rows != 0 && !norm_rows(Y, ldy, N, dtype)) ||
      (dY && rows != 0 && !norm_rows(dY, lddy, N, dtype)) || !aligned(positions, 4) || !aligned(weights, 4) || !aligned(dweights, 4))
    return FP8GEMM_ERR_LAYOUT;
  int cus;
  const int st = device(&cus);
  if (st != FP8GEMM_OK) return st;
  fp8moe::CombineGradParams p{dO, Y, dY, positions, weights, dweights, lddo, ldy, lddy, rows, T, top_k, N, 0};
  with_type(dtype, [&](auto t) {
    with_flag(streams(T, (int64_t)N * top_k, sizeof(t)), [&](auto nt) {
      with_flag(N > 512, [&](auto wide) {
        constexpr int kWaves = decltype(wide)::value ? 4 : 1;
        in_slices(T, kWaves * 64, [&](int first, dim3 grid) {
          p.first_group = first;
          hipLaunchKernelGGL((fp8moe::combine_backward_kernel<decltype(t), kWaves, decltype(nt)::value>), grid, dim3(kWaves * 64), 0,
                             stream, p);
        });
      });
    });
  });
  return launched();
}

}  // extern "C"

namespace {

// Workgroups of a gradient, at most: their sums are what the workspace holds.
constexpr int kHeadGroups = 1024;

bool heads_shape(int T, int Hq, int Hk, int D, int max_pos, int rot_dim) {
  return T >= 0 && Hq >= 0 && Hk >= 0 && (D == 64 || D == 128 || D == 256) && rot_dim >= 0 && rot_dim <= D && rot_dim % 16 == 0 &&
         (rot_dim == 0 || max_pos >= 1) && (int64_t)T * ((int64_t)Hq + Hk) <= kMost && (int64_t)std::max(Hq, Hk) * D <= INT32_MAX;
}
// of rows of H heads; a single row may carry any stride
bool head_rows(const void* p, int64_t ld, int64_t columns, int dtype) {
  return aligned(p, 16) && ld >= columns && ld % (dtype == FP8GEMM_QUANT_BF16 ? 8 : 4) == 0;
}
template <typename F>
void with_dim(int D, F f) {
  if (D == 64) f(Int<64>{});
  else if (D == 128) f(Int<128>{});
  else f(Int<256>{});
}

}  // namespace

extern "C" {

int fp8_qk_norm_rope(const void* q, int64_t ldq, const void* k, int64_t ldk, int dtype, const void* qw, const void* kw, int w_dtype,
                     const float* cos_sin, int64_t ld_cs, int max_pos, int rot_dim, int interleaved, const int32_t* positions,
                     float eps, void* q_out, int64_t ldqo, void* k_out, int64_t ldko, int T, int Hq, int Hk, int D,
                     hipStream_t stream) {
  if (Hq == 0) q = q_out = nullptr;  // no heads have no address
  if (Hk == 0) k = k_out = nullptr;
  if (T != 0 && ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr) || (q && !qw) || (k && !kw) ||
                 (rot_dim > 0 && !cos_sin)))
    return FP8GEMM_ERR_NULL;
  if (!q) Hq = 0;
  if (!k) Hk = 0;
  if (!heads_shape(T, Hq, Hk, D, max_pos, rot_dim) || !(eps >= 0.f)) return FP8GEMM_ERR_SHAPE;
  if (!norm_dtype(dtype) || !norm_dtype(w_dtype)) return FP8GEMM_ERR_LAYOUT;
  if (T == 0 || Hq + Hk == 0) return FP8GEMM_OK;
  if ((q && (!head_rows(q, ldq, (int64_t)Hq * D, dtype) || !head_rows(q_out, ldqo, (int64_t)Hq * D, dtype) || !aligned(qw, 16))) ||
      (k && (!head_rows(k, ldk, (int64_t)Hk * D, dtype) || !head_rows(k_out, ldko, (int64_t)Hk * D, dtype) || !aligned(kw, 16))) ||
      (rot_dim > 0 && (ld_cs < rot_dim || ld_cs % 4 || !aligned(cos_sin, 16))) || !aligned(positions, 4))
    return FP8GEMM_ERR_LAYOUT;
  int cus;
  const int st = device(&cus);
  if (st != FP8GEMM_OK) return st;
  fp8moe::HeadsParams p{q, k, qw, kw, q_out, k_out, cos_sin, positions, ldq, ldk, ldqo, ldko, ld_cs, eps, T, Hq, Hk,
                        w_dtype == FP8GEMM_QUANT_FP32, max_pos, rot_dim, interleaved != 0, 0};
  with_type(dtype, [&](auto t) {
    with_dim(D, [&](auto dim) {
      constexpr int kD = decltype(dim)::value;
      with_flag(streams(T, ((int64_t)Hq + Hk) * D, sizeof(t)), [&](auto nt) {
        in_slices(ceil_div((int64_t)T * (Hq + Hk), 256 * 16 / kD), 256, [&](int first, dim3 grid) {
          p.first_group = first;
          hipLaunchKernelGGL((fp8moe::heads_kernel<decltype(t), kD, decltype(nt)::value>), grid, dim3(256), 0, stream, p);
        });
      });
    });
  });
  return launched();
}

size_t fp8_qk_norm_rope_backward_workspace_size(int D) {
  return D == 64 || D == 128 || D == 256 ? (size_t)(kHeadGroups + 2) * D * sizeof(float) : 0;
}

int fp8_qk_norm_rope_backward(const void* dq, int64_t lddq, const void* dk, int64_t lddk, const void* q, int64_t ldq, const void* k,
                              int64_t ldk, int dtype, const void* qw, const void* kw, int w_dtype, const float* cos_sin,
                              int64_t ld_cs, int max_pos, int rot_dim, int interleaved, const int32_t* positions, float eps,
                              void* dq_out, int64_t lddqo, void* dk_out, int64_t lddko, float* dqw, float* dkw, int T, int Hq,
                              int Hk, int D, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const bool queries = dqw != nullptr, keys = dkw != nullptr;
  if (!queries) Hq = 0;
  if (!keys) Hk = 0;
  if (!queries && !keys) return FP8GEMM_ERR_NULL;
  if (T != 0 && ((Hq != 0 && (!dq || !q || !qw || !dq_out)) || (Hk != 0 && (!dk || !k || !kw || !dk_out)) || (rot_dim > 0 && !cos_sin)))
    return FP8GEMM_ERR_NULL;
  if (!heads_shape(T, Hq, Hk, D, max_pos, rot_dim) || !(eps >= 0.f)) return FP8GEMM_ERR_SHAPE;
  if (!norm_dtype(dtype) || !norm_dtype(w_dtype) || !aligned(dqw, 4) || !aligned(dkw, 4) || !aligned(workspace, 16))
    return FP8GEMM_ERR_LAYOUT;
  if (T != 0 &&
      ((Hq != 0 && (!head_rows(dq, lddq, (int64_t)Hq * D, dtype) || !head_rows(q, ldq, (int64_t)Hq * D, dtype) ||
                    !head_rows(dq_out, lddqo, (int64_t)Hq * D, dtype) || !aligned(qw, 16))) ||
       (Hk != 0 && (!head_rows(dk, lddk, (int64_t)Hk * D, dtype) || !head_rows(k, ldk, (int64_t)Hk * D, dtype) ||
                 !head_rows(dk_out, lddko, (int64_t)Hk * D, dtype) || !aligned(kw, 16))) ||
       (rot_dim > 0 && (ld_cs < rot_dim || ld_cs % 4 || !aligned(cos_sin, 16))) || !aligned(positions, 4)))
    return FP8GEMM_ERR_LAYOUT;
  int cus;
  const int st = device(&cus);
  if (st != FP8GEMM_OK) return st;
  // Every workgroup takes the same number of turns, of 4096 / D heads each; four workgroups a CU.
  const int64_t per_turn = 256 * 16 / D, q_turns = ceil_div((int64_t)T * Hq, per_turn), k_turns = ceil_div((int64_t)T * Hk, per_turn);
  const int64_t turns = std::max<int64_t>(1, ceil_div(q_turns + k_turns, std::min(4 * cus, kHeadGroups)));
  const int q_groups = (int)ceil_div(q_turns, turns), k_groups = (int)ceil_div(k_turns, turns);
  const int groups = q_groups + k_groups;
  if (groups && (!workspace || workspace_bytes < (size_t)groups * D * sizeof(float))) return FP8GEMM_ERR_WORKSPACE;
  float* part = static_cast<float*>(workspace);
  if (groups) {
    const fp8moe::HeadsGradParams p{dq,   dk,   q,    k,     qw,    kw,    dq_out, dk_out, cos_sin, positions, part,
                                    lddq, lddk, ldq,  ldk,   lddqo, lddko, ld_cs,  eps,    T,       Hq,        Hk,
                                    w_dtype == FP8GEMM_QUANT_FP32, max_pos, rot_dim, interleaved != 0, q_groups};
    with_type(dtype, [&](auto t) {
      with_dim(D, [&](auto dim) {
        hipLaunchKernelGGL((fp8moe::heads_backward_kernel<decltype(t), decltype(dim)::value>), dim3(groups), dim3(256), 0, stream, p);
      });
    });
    const int rc = launched();
    if (rc != FP8GEMM_OK) return rc;
  }
  hipLaunchKernelGGL(fp8moe::heads_weight_grad_kernel, dim3(2 * D / 16), dim3(1024), 0, stream, part, q_groups, groups, D, dqw,
                     dkw);
  return launched();
}

}  // extern "C"
