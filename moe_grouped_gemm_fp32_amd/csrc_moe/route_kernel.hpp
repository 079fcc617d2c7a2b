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

// 1 / x to an ulp or so, for 1 <= x.
__device__ __forceinline__ float reciprocal(float x) {
  const float r = __builtin_amdgcn_rcpf(x);
  return x < 0x1p100f ? __builtin_fmaf(__builtin_fmaf(-x, r, 1.0f), r, r) : r;  // a step would turn 1 / inf into NaN
}
__device__ __forceinline__ float sigmoid(float x) { return reciprocal(1.0f + exp_near(-x)); }

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

// What the wave's lanes have written to LDS is there for its other lanes.
__device__ __forceinline__ void own_lds() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}
// A lane of the wave gets what the lane before it has; lane 0 its own.
template <typename V>
__device__ __forceinline__ V from_before(V v) {
  return dpp<0x138>(v, v);
}
// v as an integer of the same order, and back.
__device__ __forceinline__ int ordered(float v) {
  const int i = __float_as_int(v);
  return i ^ ((i >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float ordered_back(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7FFFFFFF)); }
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ float uniform(float v) { return __int_as_float(uniform(__float_as_int(v))); }

// Leaves the keys of the best groups, the others become -inf. A group's lanes are neighbours.
// False where FP32 leaves open which groups are best (`tell`: keys are off by `slack`, as
// described at choose()).
template <int VPL, typename K>
__device__ __forceinline__ bool keep_groups(const RouteParams& p, K (&key)[VPL], int lane, bool tell, float slack) {
  const K none = (K)kNone;
  K best = none, second = none;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    second = fmax(second, fmin(best, key[j]));
    best = fmax(best, key[j]);
  }
  auto join = [&](K b, K s) {
    second = fmax(fmax(second, s), fmin(best, b));
    best = fmax(best, b);
  };
  if constexpr (sizeof(K) == 4) {
    // halves and rows are mirrored where the lanes below agree already
    if (p.log_lanes > 0) join(dpp<kSwap1>(best, best), dpp<kSwap1>(second, second));
    if (p.log_lanes > 1) join(dpp<kSwap2>(best, best), dpp<kSwap2>(second, second));
    if (p.log_lanes > 2) join(dpp<kHalfMirror>(best, best), dpp<kHalfMirror>(second, second));
    if (p.log_lanes > 3) join(dpp<kMirror>(best, best), dpp<kMirror>(second, second));
    if (p.log_lanes > 4) join(__shfl_xor(best, 16, 64), __shfl_xor(second, 16, 64));
  } else {
    for (int off = 1; off < 1 << p.log_lanes; off <<= 1) join(__shfl_xor(best, off, 64), __shfl_xor(second, off, 64));
  }
  const K score = p.group_best == 2 && second > none ? best + second : best;
  const int mine = lane >> p.log_lanes;
  int rank = 0;
  for (int g = 0; g < p.groups; ++g) {
    const K other = lane_value(score, g << p.log_lanes);
    rank += other > score || (other == score && g < mine);
  }
  const bool kept = rank < p.top_groups;
#pragma unroll
  for (int j = 0; j < VPL; ++j) key[j] = kept ? key[j] : none;
  if (!tell) return true;
  const K least = -wave_max(kept && score > none ? -score : none), most = wave_max(!kept ? score : none);
  // without a group that is left out, or with too few groups that have anyone, nothing was decided
  return !(most > none) || least - most > (K)2 * (K)(slack + 0x1p-22f * (float)fabs(most));
}

// Which experts a row's keys choose, one maximum over the wave after another, in FP64: lane i <
// top_k gets the i-th choice, -1 where none is left. A lane's experts are `base` and those
// after it, so the lower index of equal keys is the first lane's first key.
template <int VPL>
__device__ __forceinline__ int choose_slowly(const RouteParams& p, double (&key)[VPL], int base, int lane) {
  const double none = (double)kNone;
  if (p.top_groups < p.groups) keep_groups<VPL, double>(p, key, lane, false, 0.f);
  int id = -1;
  for (int i = 0; i < p.top_k; ++i) {
    double top = key[0];
    int at = 0;
#pragma unroll
    for (int j = 1; j < VPL; ++j)
      if (key[j] > top) top = key[j], at = j;
    const double m = wave_max(top);
    if (!(m > none)) break;
    const int from = __ffsll((unsigned long long)__ballot(top == m)) - 1;
    const int e = __builtin_amdgcn_readlane(base + at, from);
    if (lane == i) id = e;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (lane == from && j == at) key[j] = none;
  }
  return id;
}

constexpr int kEnough = 8;  // candidates beyond those needed that are ranked rather than searched on

// The same in FP32, by a threshold that a few more keys than needed reach: those become
// candidates, one a lane, and each counts the larger ones. Returns whether every decision was
// wider than what FP32 leaves open, `slack` + 2^-22 of a key (0: the keys are exact); equal
// keys of equal logits and biases are no question. `place`: LDS for 64 keys and numbers.
template <int VPL, typename T>
__device__ __forceinline__ bool choose(const RouteParams& p, float (&key)[VPL], int base, int lane, bool tell, float slack, const T* logits,
                                       uint2* place, int& id, float& chosen) {
  id = -1;
  int live = 0;
  float top = kNone;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    live += __popcll(__ballot(key[j] > kNone));
    top = fmaxf(top, key[j]);
  }
  live = uniform(live);
  if (live == 0) return true;
  const int need = min(p.top_k + (tell ? 1 : 0), live);  // one more: the first that is not chosen
  if (need > 64) return false;
  // Every run of lanes that has a key has one that reaches the least of the runs' maxima: the
  // longest runs, of up to 16 lanes, of which there are enough.
  float run = top, least;
  {
    auto low = [&](float v) { return -wave_max(v > kNone ? -v : kNone); };
    auto enough = [&](float v, int log) { return __popcll(__ballot(v > kNone)) >> log >= need; };
    const float r1 = fmaxf(top, dpp<kSwap1>(top, top)), r2 = fmaxf(r1, dpp<kSwap2>(r1, r1));
    const float r3 = fmaxf(r2, dpp<kHalfMirror>(r2, r2)), r4 = fmaxf(r3, dpp<kMirror>(r3, r3));
    if (enough(r4, 4)) run = r4;
    else if (enough(r3, 3)) run = r3;
    else if (enough(r2, 2)) run = r2;
    else if (enough(r1, 1)) run = r1;
    least = enough(run, 0) ? low(run) : -__builtin_huge_valf();
  }
  auto reach = [&](float t) {
    int n = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) n += __popcll(__ballot(key[j] >= t));
    return uniform(n);
  };
  // ``low`` is reached by enough, ``high`` by too few
  int low = least > kNone ? ordered(least) : ordered(kNone) + 1, high = ordered(wave_max(top)) + 1;
  int count = least > kNone ? reach(least) : live;
  while (count > min(need + kEnough, 64) && (int64_t)high - low > 1) {
    const int mid = (int)(((int64_t)low + high) >> 1);
    const int n = reach(ordered_back(mid));
    if (n >= need) low = mid, count = n;
    else high = mid;
  }
  const float threshold = ordered_back(low);
  // Candidates in the order of experts. More than 64 are left only where no number lies between
  // the threshold and what too few reach: fewer than 64 keys are above it, and the first of
  // those that equal it come after them.
  int mine = 0, first = 0;
  if (count <= 64) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) mine += key[j] >= threshold;
    first = wave_scan(mine) - mine;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (key[j] >= threshold) place[first++] = make_uint2(__float_as_uint(key[j]), base + j);
  } else {
    int equal = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) mine += key[j] > threshold, equal += key[j] == threshold;
    const int scan = wave_scan(mine);
    first = scan - mine;
    int next = last_lane(scan) + wave_scan(equal) - equal;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      if (key[j] > threshold) place[first++] = make_uint2(__float_as_uint(key[j]), base + j);
      if (key[j] == threshold && next < 64) place[next] = make_uint2(__float_as_uint(key[j]), base + j);
      next += key[j] == threshold;
    }
    count = 64;
  }
  own_lds();
  uint2 own = lane < count ? place[lane] : make_uint2(__float_as_uint(kNone), 0);
  const float value = __uint_as_float(own.x);
  int rank = 0;
  for (int c = 0; c < count; ++c) rank += lane_value(value, c) > value;
  if (lane >= count) rank = 0;
  // the ranks of different keys sum up to this; equal ones go by their order
  if (last_lane(wave_scan(rank)) != count * (count - 1) / 2) {
    for (int c = 0; c < count; ++c) rank += c < lane && lane_value(value, c) == value;
  }
  if (lane >= count) rank = lane;
  const float sorted = __int_as_float(__builtin_amdgcn_ds_permute(rank * 4, __float_as_int(value)));
  const int e = __builtin_amdgcn_ds_permute(rank * 4, (int)own.y);
  id = lane < min(p.top_k, need) ? e : -1;
  chosen = sorted;
  if (!tell) return true;
  const float before = from_before(sorted);
  const int last = from_before(e);
  bool open = lane > 0 && lane < need && !(before - sorted > slack + 0x1p-22f * fabsf(sorted));
  if (__ballot(open) == 0) return true;
  if (open) open = !(logit(logits + last) == logit(logits + e) && (!p.bias || p.bias[last] == p.bias[e]));
  return __ballot(open) == 0;
}

// One row a wave. The keys stay in registers, a group's in neighbouring lanes. Keys are FP32; a
// row with a decision that FP32 leaves open (0.5% of rows of 256 sigmoid scores with a bias)
// is decided again in FP64. Without a bias experts are compared by their logits, exactly.
template <typename T, int VPL>
__global__ void __launch_bounds__(256) route_kernel(const RouteParams p) {
  __shared__ uint2 places[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = ((int64_t)p.first_group + blockIdx.x) * 4 + wave;
  if (row >= p.T) return;
  const T* logits = static_cast<const T*>(p.logits) + row * p.ldl;
  const int group = lane >> p.log_lanes, sub = lane & ((1 << p.log_lanes) - 1);
  const int begin = sub * p.each;  // within the group
  const int count = group < p.groups ? min(max(p.size - begin, 0), p.each) : 0;
  const int base = group * p.size + begin;
  const bool limited = p.top_groups < p.groups;
  const bool by_score = p.bias || (p.group_best == 2 && limited);  // else the logits' order is the scores'
  float x[VPL], key[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    x[j] = j < count ? logit(logits + base + j) : kNone;
    key[j] = p.bias && j < count ? p.bias[base + j] : 0.f;
  }
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
  const float inverse = total == 0.f ? 0.f : 1.0f / total;
  auto score = [&](float v) { return p.sigmoid ? sigmoid(v) : exp_near(v - top) * inverse; };
  float largest = kNone;
  if (by_score || p.scores) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const float s = score(x[j]);
      if (j < count) {
        largest = fmaxf(largest, s);
        if (p.scores) p.scores[row * p.lds + base + j] = s;
      }
      const float k = s + key[j];
      key[j] = x[j] == kNone ? kNone : k == k ? k : kNanKey;
    }
  }
  if (!by_score) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = x[j] == x[j] ? x[j] : kNanKey;
  }
  // The scores' error: the exponential, the sum's (common to a row) and the reciprocal.
  const float slack = by_score ? (p.sigmoid ? 0x1p-18f : 0x1p-17f) * wave_max(largest) : 0.f;
  int id;
  float chosen;
  bool sure = !limited || keep_groups<VPL, float>(p, key, lane, by_score, slack);
  if (sure) sure = choose<VPL>(p, key, base, lane, by_score, slack, logits, places[wave], id, chosen);
  if (!sure) {
    double wide[VPL], sum = 0.0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      x[j] = j < count ? logit(logits + base + j) : kNone;
      if (!p.sigmoid) sum += j < count ? exp((double)x[j] - (double)top) : 0.0;
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      double k = x[j];
      if (by_score) {
        k = p.sigmoid ? 1.0 / (1.0 + exp(-(double)x[j])) : exp((double)x[j] - (double)top) / sum;
        if (p.bias && j < count) k += (double)p.bias[base + j];
      }
      wide[j] = x[j] == kNone ? (double)kNone : k == k ? k : (double)kNanKey;
    }
    id = choose_slowly<VPL>(p, wide, base, lane);
  }
  float s = 0.f;
  if (id >= 0) s = score(sure && !by_score && chosen > kNanKey ? chosen : logit(logits + id));
  float w = s;
  if (p.renormalize) w = s / (wave_sum(s) + kTiny);
  if (lane >= p.top_k) return;
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
  if (row >= p.T) return;
  const T* logits = static_cast<const T*>(p.logits) + row * p.ldl;
  float x[VPL], ds[VPL];
  int id = -1;
  float g = 0.f, xi = 0.f;
  if (lane < p.top_k) {
    id = p.ids[row * p.top_k + lane];
    g = p.dweights[row * p.top_k + lane] * p.scale;
  }
#pragma unroll
  for (int j = 0; j < VPL; ++j) x[j] = lane + 64 * j < p.E ? logit(logits + lane + 64 * j) : kNone;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    ds[j] = p.dscores && lane + 64 * j < p.E ? p.dscores[row * p.ldds + lane + 64 * j] : 0.f;
    spread[wave][lane + 64 * j] = 0.f;
  }
  if ((unsigned)id >= (unsigned)p.E) id = -1, g = 0.f;
  if (id >= 0) xi = logit(logits + id);
  float top = kNone, total = 0.f;
  if (!p.sigmoid) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) top = fmaxf(top, x[j]);
    top = wave_max(top);
    if (!(top > kNone)) top = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      x[j] = exp_near(x[j] - top);  // 0 past the experts
      total += x[j];
    }
    total = wave_sum(total);
  }
  const float inverse = total == 0.f ? 0.f : 1.0f / total;
  const float s = id < 0 ? 0.f : p.sigmoid ? sigmoid(xi) : exp_near(xi - top) * inverse;
  if (p.renormalize) {
    const float sum = wave_sum(s) + kTiny, dot = wave_sum(g * s);
    g = (g - dot / sum) / sum;
  }
  own_lds();
  if (id >= 0) atomicAdd(&spread[wave][id], g);
  own_lds();
  T* out = static_cast<T*>(p.dlogits) + row * p.lddl;
  float dot = 0.f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    ds[j] += spread[wave][lane + 64 * j];
    if (!p.sigmoid) {
      x[j] *= inverse;
      dot += ds[j] * x[j];
    }
  }
  if (!p.sigmoid) dot = wave_sum(dot);
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = lane + 64 * j;
    float dx;
    if (p.sigmoid) dx = ds[j] == 0.f ? 0.f : ds[j] * sigmoid(x[j]) * sigmoid(-x[j]);  // 1 - s without a cancellation
    else dx = x[j] * (ds[j] - dot);
    if (e < p.E) set_logit(out + e, dx);
  }
}

}  // namespace fp8moe
