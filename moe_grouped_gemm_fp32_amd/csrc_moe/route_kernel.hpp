// Device code of routing to experts: scores, the choice of experts and their weights, and
// the gradient of the logits.
#pragma once

#include "common.hpp"

namespace fp8moe {

using namespace fp8layer;

constexpr float kNone = -__builtin_huge_valf();
constexpr float kNanKey = -1e30f;  // below every key that is a number of any use
constexpr float kTiny = 1e-20f;    // what a sum of chosen scores is divided with at least

// exp(x) for x <= 0 or so: 2^(x log2 e) with the product's rounding error put back, which
// would otherwise be |x| 2^-24 of the result.
__device__ __forceinline__ float exp_near(float x) {
  constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLow = 1.92596299112661746887e-8f;
  const float t = x * kLog2e;
  const float r = __builtin_fmaf(x, kLog2eLow, __builtin_fmaf(x, kLog2e, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return t > -126.f && t < 127.f ? __builtin_fmaf(e, r * 0.693147180559945309f, e) : e;  // r is NaN or meaningless out there
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + exp_near(-x)); }

// A wave's maximum of doubles, in every lane (a rare path: through shuffles).
__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmax(v, __shfl_xor(v, off, 64));
  return v;
}
using fp8layer::wave_max;
__device__ __forceinline__ float lane_value(float v, int lane) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane)); }
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t u = __double_as_longlong(v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane), hi = __builtin_amdgcn_readlane((int)(u >> 32), lane);
  return __longlong_as_double((int64_t)(((uint64_t)hi << 32) | lo));
}

__device__ __forceinline__ float logit(const float* p) { return *p; }
__device__ __forceinline__ float logit(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ void set_logit(float* p, float x) { *p = x; }
__device__ __forceinline__ void set_logit(uint16_t* p, float x) { *p = (uint16_t)pack_bf16(x, x); }

struct RouteParams {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float *weights, *scores;
  int64_t ldl, lds;
  float scale;
  int T, E, top_k, groups, top_groups, group_best, sigmoid, renormalize;
  int size;       // experts of a group
  int log_lanes;  // lanes of a group: 64 over the power of two that is not below `groups`
  int each;       // experts of a lane, at most VPL
  int first_group;  // the launch's first workgroup of the call's
};

// Which experts a row's keys choose. A lane holds `count` experts in a row, from `base` on,
// `key` -inf where there is none; lanes follow each other in the order of experts, so the
// lower index of equal keys is the first lane's first key. Lane i < top_k gets the i-th
// choice (id -1 where none is left) and its logit. With `tell`, the return value says
// whether every decision was wider than what FP32 leaves open: `slack` + 2^-22 of a key.
template <int VPL, typename K>
__device__ __forceinline__ bool choose(const RouteParams& p, K (&key)[VPL], const float (&x)[VPL], int base, int lane, bool tell, float slack,
                                       const float* bias, int& id, float& chosen_x) {
  bool sure = true;
  const K none = (K)kNone;
  if (p.top_groups < p.groups) {
    K best = none, second = none;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      second = fmax(second, fmin(best, key[j]));
      best = fmax(best, key[j]);
    }
    for (int off = 1; off < 1 << p.log_lanes; off <<= 1) {
      const K b = __shfl_xor(best, off, 64), s = __shfl_xor(second, off, 64);
      second = fmax(fmax(second, s), fmin(best, b));
      best = fmax(best, b);
    }
    const K score = p.group_best == 2 && second > none ? best + second : best;
    const int mine = lane >> p.log_lanes;
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const K other = lane_value(score, g << p.log_lanes);
      rank += other > score || (other == score && g < mine);
    }
    const bool kept = rank < p.top_groups;
    if (tell && (bias != nullptr || p.group_best == 2)) {
      const K least = -wave_max(kept && score > none ? -score : none), most = wave_max(!kept ? score : none);
      // without a group that is left out, or with too few groups that have anyone, nothing was decided
      if (most > none && !(least - most > (K)2 * (K)(slack + 0x1p-22f * (float)fabs(most)))) sure = false;
    }
    if (!kept) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) key[j] = none;
    }
  }
  K top = key[0];
  int at = 0;
  float top_x = x[0];
#pragma unroll
  for (int j = 1; j < VPL; ++j)
    if (key[j] > top) top = key[j], at = j, top_x = x[j];
  id = -1;
  chosen_x = 0.f;
  K before = none;
  const int rounds = p.top_k + (tell && bias ? 1 : 0);  // one more: the first that was not chosen
  int last = -1;
  for (int i = 0; i < rounds; ++i) {
    const K m = wave_max(top);
    if (!(m > none)) break;
    const int from = __ffsll((unsigned long long)__ballot(top == m)) - 1;
    const int e = __builtin_amdgcn_readlane(base + at, from);
    if (tell && bias && i > 0 && !(before - m > (K)(slack + 0x1p-22f * (float)fabs(m)))) {
      // equal keys of equal logits and biases are no question
      const float xb = lane_value(chosen_x, i - 1), xm = lane_value(top_x, from);
      if (!(xb == xm && bias[last] == bias[e])) {
        sure = false;
        break;
      }
    }
    before = m, last = e;
    const float xe = lane_value(top_x, from);
    if (lane == i) id = e, chosen_x = xe;
    if (lane == from) {
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (j == at) key[j] = none;
      top = key[0], at = 0, top_x = x[0];
#pragma unroll
      for (int j = 1; j < VPL; ++j)
        if (key[j] > top) top = key[j], at = j, top_x = x[j];
    }
  }
  if (lane >= p.top_k) id = -1;  // the round that only looked
  return sure;
}

// One row a wave. The keys stay in registers, a group's in neighbouring lanes; a choice is a
// maximum over the lanes, of which only the winner's then changes. Keys are FP32; a row with
// a decision that FP32 leaves open (0.5% of rows of 256 sigmoid scores with a bias) is
// decided again in FP64. Without a bias experts are compared by their logits, exactly.
template <typename T, int VPL>
__global__ void __launch_bounds__(256) route_kernel(const RouteParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t row = ((int64_t)p.first_group + blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (row >= p.T) return;
  const T* logits = static_cast<const T*>(p.logits) + row * p.ldl;
  const int group = lane >> p.log_lanes, sub = lane & ((1 << p.log_lanes) - 1);
  const int begin = sub * p.each;                                                  // within the group
  const int count = group < p.groups ? min(max(p.size - begin, 0), p.each) : 0;
  const int base = group * p.size + begin;
  float x[VPL], key[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) x[j] = j < count ? logit(logits + base + j) : kNone;
  float top = kNone, total = 0.f;
  if (!p.sigmoid) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) top = fmaxf(top, x[j]);
    top = wave_max(top);
    if (!(top > kNone)) top = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) total += j < count ? exp_near(x[j] - top) : 0.f;
    total = wave_sum(total);
  }
  const float inverse = 1.0f / total;
  auto score = [&](float v) {
    if (p.sigmoid) return sigmoid(v);
    return total == 0.f ? 0.f : exp_near(v - top) * inverse;
  };
  float largest = kNone;  // score
  if (p.bias || p.scores || (p.group_best == 2 && p.top_groups < p.groups)) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      if (j >= count) {
        key[j] = kNone;
        continue;
      }
      const float s = score(x[j]);
      largest = fmaxf(largest, s);
      if (p.scores) p.scores[row * p.lds + base + j] = s;
      const float k = p.bias ? s + p.bias[base + j] : s;
      key[j] = x[j] == kNone ? kNone : k == k ? k : kNanKey;
    }
    largest = wave_max(largest);
  }
  const bool by_score = p.bias || (p.group_best == 2 && p.top_groups < p.groups);
  if (!by_score) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = x[j] == x[j] ? x[j] : kNanKey;
  }
  int id;
  float chosen;
  // The scores' error: the exponential, the sum's (common to a row) and the reciprocal.
  const float slack = (p.sigmoid ? 0x1p-18f : 0x1p-17f) * largest;
  const bool sure = choose<VPL, float>(p, key, x, base, lane, by_score, slack, p.bias, id, chosen);
  if (!sure) {
    double wide[VPL], sum = 0.0;
    if (!p.sigmoid) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) sum += j < count ? exp((double)x[j] - (double)top) : 0.0;
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      wide[j] = (double)kNone;
      if (j >= count || x[j] == kNone) continue;
      const double s = p.sigmoid ? 1.0 / (1.0 + exp(-(double)x[j])) : exp((double)x[j] - (double)top) / sum;
      const double k = p.bias ? s + (double)p.bias[base + j] : s;
      wide[j] = k == k ? k : (double)kNanKey;
    }
    choose<VPL, double>(p, wide, x, base, lane, false, 0.f, p.bias, id, chosen);
  }
  if (lane >= p.top_k) return;
  const float s = id >= 0 ? score(chosen) : 0.f;
  float w = s;
  if (p.renormalize) {
    float sum = 0.f;
    for (int i = 0; i < p.top_k; ++i) sum += lane_value(s, i);
    w = s / (sum + kTiny);
  }
  const int64_t out = row * p.top_k + lane;
  p.ids[out] = id;
  p.weights[out] = w * p.scale;
}

struct RouteGradParams {
  const float *dweights, *dscores;
  const void* logits;
  const int32_t* ids;
  void* dlogits;
  int64_t ldl, ldds, lddl;
  float scale;
  int T, E, top_k, sigmoid, renormalize;
  int first_group;
};

// One row a wave; expert lane + 64 j is a lane's j-th. The few gradients of the chosen scores
// are spread to their experts through LDS.
template <typename T, int VPL>
__global__ void __launch_bounds__(256) route_backward_kernel(const RouteGradParams p) {
  __shared__ float spread[4][64 * VPL];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = ((int64_t)p.first_group + blockIdx.x) * 4 + wave;
  const bool live = row < p.T;  // barriers below are for whole workgroups
  const T* logits = static_cast<const T*>(p.logits) + row * p.ldl;
  float x[VPL], ds[VPL];
  int id = -1;
  float g = 0.f, xi = 0.f;
  if (live) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) x[j] = lane + 64 * j < p.E ? logit(logits + lane + 64 * j) : kNone;
    if (lane < p.top_k) {
      id = p.ids[row * p.top_k + lane];
      if ((unsigned)id >= (unsigned)p.E) id = -1;
      if (id >= 0) {
        g = p.dweights[row * p.top_k + lane] * p.scale;
        xi = logit(logits + id);
      }
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      ds[j] = p.dscores && lane + 64 * j < p.E ? p.dscores[row * p.ldds + lane + 64 * j] : 0.f;
      spread[wave][lane + 64 * j] = 0.f;
    }
  }
  __syncthreads();
  float top = kNone, total = 0.f;
  if (live && !p.sigmoid) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) top = fmaxf(top, x[j]);
    top = wave_max(top);
    if (!(top > kNone)) top = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) total += lane + 64 * j < p.E ? exp_near(x[j] - top) : 0.f;
    total = wave_sum(total);
  }
  const float inverse = 1.0f / total;
  auto score = [&](float v) {
    if (p.sigmoid) return sigmoid(v);
    return total == 0.f ? 0.f : exp_near(v - top) * inverse;
  };
  if (live) {
    const float s = id >= 0 ? score(xi) : 0.f;
    if (p.renormalize) {
      const float sum = wave_sum(s) + kTiny, dot = wave_sum(g * s);
      g = (g - dot / sum) / sum;
    }
    if (id >= 0) atomicAdd(&spread[wave][id], g);
  }
  __syncthreads();
  if (!live) return;
  T* out = static_cast<T*>(p.dlogits) + row * p.lddl;
  float dot = 0.f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    ds[j] += spread[wave][lane + 64 * j];
    if (!p.sigmoid) {
      x[j] = lane + 64 * j < p.E ? score(x[j]) : 0.f;
      dot += ds[j] * x[j];
    }
  }
  if (!p.sigmoid) dot = wave_sum(dot);
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = lane + 64 * j;
    if (e >= p.E) continue;
    if (p.sigmoid) {
      // 1 - s without the subtraction's cancellation
      set_logit(out + e, ds[j] == 0.f ? 0.f : ds[j] * sigmoid(x[j]) * sigmoid(-x[j]));
    } else {
      set_logit(out + e, x[j] * (ds[j] - dot));
    }
  }
}

}  // namespace fp8moe
