// Device code of routing to experts: scores, the choice of experts and their weights, and
// the gradient of the logits.
#pragma once

#include <type_traits>

#include "common.hpp"

namespace fp8moe {

using namespace fp8layer;

constexpr float kNone = -__builtin_huge_valf();
constexpr float kLargest = 3.40282346638528859812e38f;
// Of a NaN, below every number: in FP32 it meets the last of them, and FP64 decides.
constexpr float kNanKey = -kLargest;
constexpr double kNanExactly = -1e300;
constexpr float kTiny = 1e-20f;    // what a sum of chosen scores is divided with at least

// exp(x): 2^(x log2 e) with the product's rounding error put back, which would otherwise be
// |x| 2^-24 of the result.
__device__ __forceinline__ float exp_near(float x) {
  constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLow = 1.92596299112661746887e-8f;
  const float t = x * kLog2e;
  const float r = __builtin_fmaf(x, kLog2eLow, __builtin_fmaf(x, kLog2e, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return fabsf(t) < 126.f ? __builtin_fmaf(e, r * 0.693147180559945309f, e) : e;  // r is meaningless out there
}
// Within 3 ulp: the exponential, the sum, the reciprocal.
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + exp_near(-x)); }
// For keys: off by s (3 + 2 |x| (1 - s)) 2^-24.
__device__ __forceinline__ float sigmoid_for_order(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.44269502162933349609375f));
}

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
  int even;       // whether every lane has VPL
  int even_16;    // and where 16 lanes hold a row
  int first_group;  // the launch's first workgroup of the call's
};

// What the wave's lanes have written to LDS is there for its other lanes.
__device__ __forceinline__ void own_lds() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}
// A lane of the wave gets what the lane before it has; lane 0 its own.
__device__ __forceinline__ int from_before(int v) { return dpp<0x138>(v, v); }

// Keys are compared as integers of the floats' order (0 has one sign): the wave's data-parallel
// maxima are single instructions then.
__device__ __forceinline__ int ordered(float v) {
  const int i = __float_as_int(v + 0.f);
  return i ^ ((i >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float value_of(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7FFFFFFF)); }
constexpr int kNoKey = (int)0x807FFFFF;  // of -inf
constexpr int kLowest = (int)0x80000000;
constexpr int kInfinite = 0x7F800000;    // of +inf

// Of experts that their logits alone order. Where a row of the wave has a NaN, numbers make room for
// it above what is never chosen.
template <int VPL>
__device__ __forceinline__ void logit_keys(const float (&x)[VPL], int (&key)[VPL]) {
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    key[j] = ordered(x[j]);
    sum += x[j];
  }
  if (__ballot(sum != sum) != 0) {  // or has infinities of both signs, or sums to them
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = x[j] != x[j] ? kNoKey + 1 : key[j] + (key[j] > kNoKey);
  }
}

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ int max_with(int v) {
  // all rows: every lane has a source
  return max(v, __builtin_amdgcn_update_dpp(kLowest, v, CTRL, ROWS, 0xF, ROWS == 0xF));
}
template <int CTRL>
__device__ __forceinline__ int moved(int v) {
  return __builtin_amdgcn_update_dpp(kLowest, v, CTRL, 0xF, 0xF, true);
}
__device__ __forceinline__ int wave_max(int v) {
  v = max_with<kMirror>(max_with<kHalfMirror>(max_with<kSwap2>(max_with<kSwap1>(v))));
  return last_lane(max_with<kLast31, 0xC>(max_with<kLast15, 0xA>(v)));
}
// The row's largest logit that is a number; 0 where there is none above -inf.
template <int VPL>
__device__ __forceinline__ float largest_number(const float (&x)[VPL]) {
  float top = kNone;
#pragma unroll
  for (int j = 0; j < VPL; ++j) top = fmaxf(top, x[j]);
  const int most = wave_max(ordered(top));
  return most > kNoKey ? value_of(most) : 0.f;
}
__device__ __forceinline__ int lane_value(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int lanes_of(bool b) { return __popcll(__ballot(b)); }

// A group's score, kNoKey without experts. A sum past FP32's numbers becomes the last of them, so
// that a group with experts has no empty one's score; such groups meet there, and FP64 decides.
__device__ __forceinline__ int group_score(int best, int second, bool two) {
  if (!two) return best;
  return min(max(ordered(value_of(best) + value_of(second)), kNoKey + 1), max(best, kInfinite - 1));
}
// What a group's score is off by at most: the errors of its scores, and 2^-24 of each key and of
// their sum, which may be far smaller than they are. Twice over, like the slack.
__device__ __forceinline__ float group_off(int best, int second, bool two, float slack) {
  float off = __builtin_fmaf(0x1p-22f, fabsf(value_of(best)), slack);
  if (two) off = __builtin_fmaf(0x1p-22f, fabsf(value_of(second)), off);
  return off;
}

// Whether the lane's group is among the best. A group's lanes are neighbours. `sure` becomes
// false where FP32 leaves that open (`tell`: keys are off by `slack`, as described at
// choose()): where a group that is kept need not be better than every one that is not.
template <int VPL>
__device__ __forceinline__ bool best_groups(const RouteParams& p, const int (&key)[VPL], int lane, bool tell, float slack, bool& sure) {
  int best = key[0], second = kNoKey;
#pragma unroll
  for (int j = 1; j < VPL; ++j) {
    second = max(second, min(best, key[j]));
    best = max(best, key[j]);
  }
  auto join = [&](int b, int s) {
    second = max(max(second, s), min(best, b));
    best = max(best, b);
  };
  // halves and rows are mirrored where the lanes below agree already
  if (p.log_lanes > 0) join(moved<kSwap1>(best), moved<kSwap1>(second));
  if (p.log_lanes > 1) join(moved<kSwap2>(best), moved<kSwap2>(second));
  if (p.log_lanes > 2) join(moved<kHalfMirror>(best), moved<kHalfMirror>(second));
  if (p.log_lanes > 3) join(moved<kMirror>(best), moved<kMirror>(second));
  if (p.log_lanes > 4) join(__shfl_xor(best, 16, 64), __shfl_xor(second, 16, 64));
  const bool two = p.group_best == 2 && second > kNoKey;
  const int score = group_score(best, second, two);
  const float off = tell ? group_off(best, second, two, slack) : 0.f;
  const int mine = lane >> p.log_lanes;
  const bool there = mine < p.groups;
  int rank = 0;
  for (int g = 0; g < p.groups; ++g) rank += lane_value(score, g << p.log_lanes) > score;
  // the ranks of different scores sum up to this; of equal ones the first groups are better
  if (last_lane(wave_scan(there ? rank : 0)) >> p.log_lanes != p.groups * (p.groups - 1) / 2) {
    for (int g = 0; g < p.groups; ++g) rank += lane_value(score, g << p.log_lanes) == score && g < mine;
  }
  if (tell) {
    const bool kept = there && rank < p.top_groups;
    const int most = wave_max(there && !kept && score > kNoKey ? ordered(value_of(score) + off) : kNoKey);
    // where nobody is left out, nothing was decided
    sure = most == kNoKey || __ballot(kept && !(value_of(score) - off > value_of(most))) == 0;
  }
  return there && rank < p.top_groups;
}

// The same of keys in FP64.
template <int VPL>
__device__ __forceinline__ bool best_groups(const RouteParams& p, const double (&key)[VPL], int lane) {
  const double none = (double)kNone;
  double best = none, second = none;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    second = fmax(second, fmin(best, key[j]));
    best = fmax(best, key[j]);
  }
  for (int off = 1; off < 1 << p.log_lanes; off <<= 1) {
    const double b = __shfl_xor(best, off, 64), s = __shfl_xor(second, off, 64);
    second = fmax(fmax(second, s), fmin(best, b));
    best = fmax(best, b);
  }
  const double score = p.group_best == 2 && second > none ? best + second : best;
  const int mine = lane >> p.log_lanes;
  int rank = 0;
  for (int g = 0; g < p.groups; ++g) {
    const double other = lane_value(score, g << p.log_lanes);
    rank += other > score || (other == score && g < mine);
  }
  return mine < p.groups && rank < p.top_groups;
}

// A row's keys in FP64.
struct Exactly {
  bool sigmoid;
  double top, sum;  // of the softmax
  template <int VPL>
  __device__ __forceinline__ Exactly(bool sigmoid, float top, const float (&x)[VPL], int lanes = 64)
      : sigmoid(sigmoid), top(top), sum(0.0) {
    if (sigmoid) return;
#pragma unroll
    for (int j = 0; j < VPL; ++j) sum += exp((double)x[j] - this->top);
    for (int off = lanes / 2; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
  }
  __device__ __forceinline__ double key(float x, float bias) const {
    if (x == kNone) return (double)kNone;
    const double k = (sigmoid ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - top) / sum) + (double)bias;
    return k == k ? k : kNanExactly;
  }
};

// Which experts a row's keys choose, one maximum over the wave after another, in FP64: lane i <
// top_k gets the i-th choice, -1 where none is left. A lane's experts are `base` and those
// after it, so the lower index of equal keys is the first lane's first key.
template <int VPL>
__device__ __forceinline__ int choose_slowly(const RouteParams& p, double (&key)[VPL], int base, int lane) {
  const double none = (double)kNone;
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
    const int e = lane_value(base + at, from);
    if (lane == i) id = e;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (lane == from && j == at) key[j] = none;
  }
  return id;
}

// Whether any of the lane's keys that FP32 cannot tell from the first one that is not chosen,
// `edge`, is another than that, by its logit and bias. Equal keys at the edge of the choice go by
// their numbers if it holds for no lane: what is further off was decided, whatever its place.
template <int VPL, typename T>
__device__ __forceinline__ bool others_near(const RouteParams& p, const int (&key)[VPL], const float (&x)[VPL], int base, int2 edge, float slack,
                                            const T* logits) {
  const float v = value_of(edge.x), off = slack + 0x1p-22f * fabsf(v), x0 = logit(logits + edge.y), b0 = p.bias[edge.y];
  bool other = false;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const float k = value_of(key[j]);
    if (key[j] > kNoKey && !(fabsf(k - v) > off)) other = other || !(x[j] == x0 && p.bias[base + j] == b0);
  }
  return other;
}

constexpr int kEnough = 8;  // candidates beyond those needed that are ranked rather than searched on

// The same in FP32, by a threshold that a few more keys than needed reach: those become
// candidates, one a lane, and each counts the larger ones. A decision is sure where two keys
// are further apart than FP32 leaves open, `slack` + 2^-22 of a key (without `tell` the keys
// are exact), or have equal logits and biases. Otherwise the candidates, and whatever could
// be among them, are ranked in FP64; false if they are too many for that. That is so for each row
// of more than 64 experts with a bias of which 64 are chosen, since the first that is not would be
// the 65th: 4096 rows of 256 take 42 us, and 13 with 63 chosen; one row 25 and 4.2. `place`: LDS
// for 64 keys and numbers.
template <int VPL, typename T>
__device__ __forceinline__ bool choose(const RouteParams& p, const int (&key)[VPL], const float (&x)[VPL], int base, int lane, bool tell,
                                       float slack, float top_logit, const T* logits, int2* place, int& id) {
  id = -1;
  int live = 0, top = key[0];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    live += lanes_of(key[j] > kNoKey);
    top = max(top, key[j]);
  }
  if (live == 0) return true;
  const int need = min(p.top_k + (int)tell, live);  // one more: the first that is not chosen
  if (need > 64) return false;
  // Every run of lanes that has a key has one that reaches the least of the runs' maxima: the
  // longest runs, of up to 16 lanes, of which there are enough.
  const int r1 = max_with<kSwap1>(top), r2 = max_with<kSwap2>(r1), r3 = max_with<kHalfMirror>(r2), r4 = max_with<kMirror>(r3);
  int run = top;
  if (lanes_of(r4 > kNoKey) >> 4 >= need) run = r4;
  else if (lanes_of(r3 > kNoKey) >> 3 >= need) run = r3;
  else if (lanes_of(r2 > kNoKey) >> 2 >= need) run = r2;
  else if (lanes_of(r1 > kNoKey) >> 1 >= need) run = r1;
  // `low` is reached by enough, `high` by too few
  int low = kNoKey + 1, high = last_lane(max_with<kLast31, 0xC>(max_with<kLast15, 0xA>(r4))) + 1, count = live;
  auto reach = [&](int t) {
    int n = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) n += lanes_of(key[j] >= t);
    return n;
  };
  const int limit = min(need + kEnough, 64);
  if (count > limit) {
    if (lanes_of(run > kNoKey) >= need) {
      low = ~wave_max(run > kNoKey ? ~run : kLowest);  // ~ turns the order of integers
      count = reach(low);
    }
    while (count > limit && (unsigned)high - (unsigned)low > 1) {
      const int mid = low + (int)(((unsigned)high - (unsigned)low) >> 1);
      const int n = reach(mid);
      if (n >= need) low = mid, count = n;
      else high = mid;
    }
  }
  // Candidates in the order of experts. More than 64 are left only where no number lies between
  // the threshold and what too few reach: fewer than 64 keys are above it, and the first of
  // those that equal it come after them.
  auto candidates = [&](int t) {
    int mine = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) mine += key[j] >= t;
    int first = wave_scan(mine) - mine;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (key[j] >= t) place[first++] = make_int2(key[j], base + j);
  };
  if (count <= 64) {
    candidates(low);
  } else {
    int mine = 0, equal = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) mine += key[j] > low, equal += key[j] == low;
    const int scan = wave_scan(mine);
    int first = scan - mine, next = last_lane(scan) + wave_scan(equal) - equal;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      if (key[j] > low) place[first++] = make_int2(key[j], base + j);
      if (key[j] == low && next < 64) place[next] = make_int2(key[j], base + j);
      next += key[j] == low;
    }
    count = 64;
  }
  own_lds();
  int2 own = place[lane];
  if (lane >= count) own.x = kLowest;
  int rank = 0;
  for (int c = 0; c < count; c += 4) {  // four at a time, at most 64; the lanes past the candidates are larger than none
#pragma unroll
    for (int i = 0; i < 4; ++i) rank += lane_value(own.x, c + i) > own.x;
  }
  // the ranks of different keys sum up to this; equal ones go by their order
  if (last_lane(wave_scan(lane < count ? rank : 0)) != count * (count - 1) / 2) {
    for (int c = 0; c < count; ++c) rank += c < lane && lane_value(own.x, c) == own.x;
  }
  if (lane >= count) rank = lane;
  int e = __builtin_amdgcn_ds_permute(rank * 4, own.y);
  const int chosen = min(p.top_k, need);
  if (tell) {
    const int sorted = __builtin_amdgcn_ds_permute(rank * 4, own.x);
    const float v = value_of(sorted), before = value_of(from_before(sorted));
    bool open = lane > 0 && lane < need && !(before - v > slack + 0x1p-22f * fabsf(v));
    if (__ballot(open) != 0) {
      const int last = from_before(e);
      if (open) open = !(logit(logits + last) == logit(logits + e) && p.bias[last] == p.bias[e]);
      if (need > p.top_k) {  // what follows equal keys at the edge could be larger than they are
        const int2 edge = make_int2(lane_value(sorted, p.top_k), lane_value(e, p.top_k));
        if (!(value_of(lane_value(sorted, p.top_k - 1)) - value_of(edge.x) > slack + 0x1p-22f * fabsf(value_of(edge.x))))
          open = open || others_near(p, key, x, base, edge, slack, logits);
      }
      if (__ballot(open) != 0) {
        const float t = value_of(low);
        low = min(low, ordered(t - (slack + 0x1p-22f * fabsf(t))));  // what does not reach this is less than those that are
        count = low > kNoKey ? reach(low) : live;                    // needed; of keys of +inf it is no number, of either sign
        if (count > 64) return false;
        candidates(max(low, kNoKey + 1));
        own_lds();
        const Exactly exactly(p.sigmoid, top_logit, x);
        e = lane < count ? place[lane].y : 0;
        const double k = lane < count ? exactly.key(logit(logits + e), p.bias[e]) : (double)kNone;
        rank = 0;
        for (int c = 0; c < count; ++c) {
          const double other = lane_value(k, c);
          rank += other > k || (other == k && c < lane);
        }
        if (lane >= count) rank = lane;
        e = __builtin_amdgcn_ds_permute(rank * 4, e);
      }
    }
  }
  id = lane < chosen ? e : -1;
  return true;
}

__device__ __forceinline__ int row16_max(int v) { return max_with<kMirror>(max_with<kHalfMirror>(max_with<kSwap2>(max_with<kSwap1>(v)))); }
template <typename V>
__device__ __forceinline__ V row16_sum(V v) {
  v += dpp<kSwap1>(v, v);
  v += dpp<kSwap2>(v, v);
  v += dpp<kHalfMirror>(v, v);
  return v + dpp<kMirror>(v, v);
}
// The sum of the chosen scores, lane i's the i-th. Up to 16, in the order in which a row of 16 lanes
// adds them; two experts a lane or fewer are added in the experts' order there, and all scores of a
// softmax lane by lane, so weights' last bits may depend on the kernel.
__device__ __forceinline__ float sum_of_chosen(float s) {
  const float row = row16_sum(s);
  return lane_value(row, 0) + lane_value(row, 16) + lane_value(row, 32) + lane_value(row, 48);
}

// How far two keys' errors come to, twice over, for a row's largest score, whose bits have the
// order of what is not negative. Sigmoids: s |x| (1 - s) grows up to s = 1/4 and then stays below
// 0.28, and |x| < 0.7 (e + 1) for a largest score of 2^-e. Softmax: three roundings and the
// exponent's, and the sum's, common to a row, of up to 38 terms and levels. Scores below 2^-126 are
// computed as 0.
__device__ __forceinline__ float slack_of(int largest, int sigmoid) {
  const float relative = sigmoid ? 0x1p-19f + 0x1p-21f * (float)(127 - (largest >> 23)) : 0x1p-17f;
  return fmaxf(__int_as_float(largest) * relative, 0x1p-124f);
}

// One row, by a wave. The keys stay in registers, a group's in neighbouring lanes. Keys are FP32;
// what they leave open (in 2 of 1000 rows of 256 sigmoid scores with a bias) is decided in FP64.
// Without a bias experts are compared by their logits, exactly, and only groups by scores. Bound by vector instructions:
// 16384 rows of 256 experts in 8 groups, 8 chosen, 388 a row, 14.2 us (their bytes take 3.7);
// without groups and bias 9.7; one row 3.5 us, most of it the launch and one chain; 512 experts in 8
// groups 17.7, 1024 27.9, a softmax of 1024 without groups and bias 21.0.
template <typename T, int VPL>
__device__ __forceinline__ void route_row(const RouteParams& p, int64_t row, int lane, int2* place) {
  const T* logits = static_cast<const T*>(p.logits) + row * p.ldl;
  const int group = lane >> p.log_lanes, sub = lane & ((1 << p.log_lanes) - 1);
  const int begin = sub * p.each;  // within the group
  const int count = group < p.groups ? min(max(p.size - begin, 0), p.each) : 0;
  const int base = group * p.size + begin;
  const bool limited = p.top_groups < p.groups;
  const bool by_score = p.bias || (p.group_best == 2 && limited);  // else the logits' order is the scores'
  const bool tell = p.bias;  // experts without a bias go by their logits, however their groups are found
  float x[VPL], bias[VPL] = {};
  int key[VPL];
  if (p.even) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) x[j] = logit(logits + base + j);
    if (p.bias) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) bias[j] = p.bias[base + j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j) x[j] = logit(logits + min(base + j, p.E - 1));
    if (p.bias) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) bias[j] = p.bias[min(base + j, p.E - 1)];
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) x[j] = j < count ? x[j] : kNone;
  }
  float top = 0.f, inverse = 0.f, slack = 0.f;
  float s[VPL];  // scores
  if (!p.sigmoid) {
    top = largest_number(x);
    float total = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      s[j] = exp_near(x[j] - top);  // 0 past the experts
      total += s[j];
    }
    total = wave_sum(total);
    inverse = total == 0.f ? 0.f : 1.0f / total;
#pragma unroll
    for (int j = 0; j < VPL; ++j) s[j] *= inverse;
  } else if (p.scores) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) s[j] = sigmoid(x[j]);
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j) s[j] = sigmoid_for_order(x[j]);
  }
  if (p.scores) {
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (j < count) p.scores[row * p.lds + base + j] = s[j];
  }
  if (by_score) {
    float largest = 0.f, sum = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      largest = fmaxf(largest, s[j]);
      s[j] += bias[j];
    }
    slack = slack_of(wave_max(__float_as_int(largest)), p.sigmoid);
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      key[j] = x[j] == kNone ? kNoKey : ordered(s[j]);
      sum += s[j];
    }
    if (__ballot(sum != sum) != 0) {
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (s[j] != s[j] && x[j] != kNone) key[j] = ordered(kNanKey);
    }
  } else {
    logit_keys(x, key);
  }
  auto exact_keys = [&](double (&wide)[VPL]) {
    const Exactly exactly(p.sigmoid, top, x);
#pragma unroll
    for (int j = 0; j < VPL; ++j) wide[j] = exactly.key(x[j], p.bias ? p.bias[min(base + j, p.E - 1)] : 0.f);
  };
  if (limited) {
    bool sure = true, kept = best_groups<VPL>(p, key, lane, by_score, slack, sure);
    if (!sure) {
      double wide[VPL];
      exact_keys(wide);
      kept = best_groups<VPL>(p, wide, lane);
    }
    if (by_score && !tell) {
      if constexpr (VPL > 8) {  // loaded again: kept over FP64's groups, 16 are 15 registers and a wave a SIMD
        float y[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) y[j] = j < count ? logit(logits + min(base + j, p.E - 1)) : kNone;
        logit_keys(y, key);
      } else {
        logit_keys(x, key);
      }
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = kept ? key[j] : kNoKey;
  }
  int id;
  if (!choose<VPL>(p, key, x, base, lane, tell, slack, top, logits, place, id)) {
    double wide[VPL];
    exact_keys(wide);
#pragma unroll
    for (int j = 0; j < VPL; ++j) wide[j] = key[j] == kNoKey ? (double)kNone : wide[j];
    id = choose_slowly<VPL>(p, wide, base, lane);
  }
  float w = 0.f;
  if (id >= 0) {
    const float v = logit(logits + id);
    w = p.sigmoid ? sigmoid(v) : exp_near(v - top) * inverse;
  }
  const float over = p.renormalize ? p.scale / (sum_of_chosen(w) + kTiny) : p.scale;
  if (lane < p.top_k) {
    const int64_t out = row * p.top_k + lane;
    p.ids[out] = id;
    p.weights[out] = w * over;
  }
}

// What the lanes of a row of 16 hold comes by every lane of it in turn: f(values, turn).
template <int D>
__device__ __forceinline__ int turned(int v) {
  if constexpr (D == 0) return v;
  else return moved<kTurn + D>(v);
}
template <int D = 0, int VPL, typename F>
__device__ __forceinline__ void each_turn(const int (&key)[VPL], F f) {
  int other[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) other[j] = turned<D>(key[j]);
  f(other, std::integral_constant<int, D>{});
  if constexpr (D < 15) each_turn<D + 1>(key, f);
}
template <typename T, int VPL>
__global__ void __launch_bounds__(256) route_kernel(const RouteParams p) {
  __shared__ int2 places[4][64];
  const int wave = uniform(threadIdx.x >> 6);
  const int64_t row = ((int64_t)p.first_group + blockIdx.x) * 4 + wave;
  if (row < p.T) route_row<T, VPL>(p, row, threadIdx.x & 63, places[wave]);
}

// Four rows a wave: 16 lanes hold a row, VPL experts each. Up to two each, every key counts the
// larger ones of its row as they come by; more are searched for a threshold that 16 at most
// reach, one a lane, which then count each other. What FP32 leaves open, or equal keys make too
// many, is done again by route_row(), up to 16 near keys of more than 32 experts in place. Vector
// instructions a row of 256 experts in 8 groups 258, a wave's own row 388: 65536 rows 31.9 and
// 44.0 us; of 16384, four waves a SIMD, whose chains bind it, 13.4 and 14.2 (cold, 14.6). What
// route_row() and FP64 need lives beside the fast path: 96 registers, and 46 scalars spilled to
// lanes. 16384 rows of 16 experts (sigmoid, bias) 3.3 to 6.3 us, of 64 6.4.
template <typename T, int VPL>
__global__ void __launch_bounds__(256) route_rows_kernel(const RouteParams p) {
  __shared__ int2 places[4][64];
  __shared__ int2 order[4][4][VPL <= 2 ? 16 * VPL : 32];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), sub16 = lane & 15, mine = lane >> 4;
  const int64_t first_row = (((int64_t)p.first_group + blockIdx.x) * 4 + wave) * 4;
  if (first_row >= p.T) return;
  const int64_t row = min(first_row + mine, (int64_t)p.T - 1);  // rows past the last are done and not written
  const bool there = first_row + mine < p.T;
  const int log_lanes = p.log_lanes - 2, each = (p.size + (1 << log_lanes) - 1) >> log_lanes;
  const T* logits = static_cast<const T*>(p.logits) + row * p.ldl;
  const int group = sub16 >> log_lanes, begin = (sub16 & ((1 << log_lanes) - 1)) * each;
  const int count = group < p.groups ? min(max(p.size - begin, 0), each) : 0;
  const int base = group * p.size + begin;
  const bool limited = p.top_groups < p.groups;
  const bool by_score = p.bias || (p.group_best == 2 && limited), tell = p.bias;
  float x[VPL], s[VPL];
  int key[VPL];
  if (p.even_16) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) x[j] = logit(logits + base + j);
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j) x[j] = logit(logits + min(base + j, p.E - 1));
#pragma unroll
    for (int j = 0; j < VPL; ++j) x[j] = j < count ? x[j] : kNone;
  }
  float top = 0.f, inverse = 0.f, slack = 0.f;
  if (p.sigmoid && VPL > 2 && !p.scores) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) s[j] = sigmoid_for_order(x[j]);
  } else if (p.sigmoid) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) s[j] = sigmoid(x[j]);
  } else {
    float most = kNone, total = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) most = fmaxf(most, x[j]);
    const int bits = row16_max(ordered(most));
    top = bits > kNoKey ? value_of(bits) : 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      s[j] = exp_near(x[j] - top);
      total += s[j];
    }
    total = row16_sum(total);
    inverse = total == 0.f ? 0.f : 1.0f / total;
#pragma unroll
    for (int j = 0; j < VPL; ++j) s[j] *= inverse;
  }
  if (p.scores && there) {
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (j < count) p.scores[row * p.lds + base + j] = s[j];
  }
  if (by_score) {
    float largest = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) largest = fmaxf(largest, s[j]);
    float bias[VPL] = {};
    if (p.bias) {
      if (p.even_16) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) bias[j] = p.bias[base + j];
      } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) bias[j] = p.bias[min(base + j, p.E - 1)];
      }
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const float k = s[j] + bias[j];
      key[j] = x[j] == kNone ? kNoKey : ordered(k == k ? k : kNanKey);
    }
    slack = slack_of(row16_max(__float_as_int(largest)), p.sigmoid);
  } else {
    logit_keys(x, key);
  }
  bool open = false;
  if (limited) {
    int best = key[0], second = kNoKey;
#pragma unroll
    for (int j = 1; j < VPL; ++j) {
      second = max(second, min(best, key[j]));
      best = max(best, key[j]);
    }
    auto join = [&](int b, int t) {
      second = max(max(second, t), min(best, b));
      best = max(best, b);
    };
    if (log_lanes > 0) join(moved<kSwap1>(best), moved<kSwap1>(second));
    if (log_lanes > 1) join(moved<kSwap2>(best), moved<kSwap2>(second));
    if (log_lanes > 2) join(moved<kHalfMirror>(best), moved<kHalfMirror>(second));
    const bool two = p.group_best == 2 && second > kNoKey;
    const int score[1] = {group_score(best, second, two)}, number[1] = {group};
    const float off = by_score ? group_off(best, second, two, slack) : 0.f;
    int rank = 0;  // in lanes
    each_turn(score, [&](const int (&other)[1], auto) { rank += other[0] > score[0]; });
    const bool is = group < p.groups;
    if (__ballot(row16_sum(is ? rank : 0) != p.groups * (p.groups - 1) / 2 << 2 * log_lanes) != 0) {
      each_turn(number, [&](const int (&other)[1], auto d) {
        rank += turned<decltype(d)::value>(score[0]) == score[0] && other[0] < group;
      });
    }
    rank >>= log_lanes;
    if (by_score) {
      const bool kept = is && rank < p.top_groups;
      const int most = row16_max(is && !kept && score[0] > kNoKey ? ordered(value_of(score[0]) + off) : kNoKey);
      open = kept && most != kNoKey && !(value_of(score[0]) - off > value_of(most));
    }
    if (by_score && !tell) logit_keys(x, key);
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = is && rank < p.top_groups ? key[j] : kNoKey;
  }
  int live = 0;
#pragma unroll
  for (int j = 0; j < VPL; ++j) live += key[j] > kNoKey;
  live = row16_sum(live);
  uint64_t left;
  if constexpr (VPL <= 2) {
    int rank[VPL] = {}, sum = 0;
    each_turn(key, [&](const int (&other)[VPL], auto) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
#pragma unroll
        for (int j = 0; j < VPL; ++j) rank[j] += other[i] > key[j];
    });
#pragma unroll
    for (int j = 0; j < VPL; ++j) sum += key[j] > kNoKey ? rank[j] : 0;
    if (__ballot(row16_sum(sum) != live * (live - 1) / 2) != 0) {  // equal keys go by their numbers
      int number[1] = {base};
      each_turn(number, [&](const int (&other)[1], auto d) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const int theirs = turned<decltype(d)::value>(key[i]);
#pragma unroll
          for (int j = 0; j < VPL; ++j) rank[j] += theirs == key[j] && other[0] + i < base + j;
        }
      });
    }
    if (tell) {
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (key[j] > kNoKey) order[wave][mine][rank[j]] = make_int2(key[j], base + j);
      own_lds();
      bool edge = false;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        if (key[j] == kNoKey || rank[j] >= p.top_k || rank[j] + 1 >= live) continue;
        const int2 next = order[wave][mine][rank[j] + 1];
        const float v = value_of(key[j]), after = value_of(next.x);
        if (v - after > slack + 0x1p-22f * fabsf(after)) continue;
        open = open || !(x[j] == logit(logits + next.y) && p.bias[base + j] == p.bias[next.y]);
        edge = edge || rank[j] + 1 == p.top_k;
      }
      const bool at_edge = (__ballot(edge) >> (lane & 48) & 0xFFFF) != 0;
      if (at_edge) open = open || others_near(p, key, x, base, order[wave][mine][p.top_k], slack, logits);
    }
    left = __ballot(open && there);
    const bool again = (left >> (lane & 48) & 0xFFFF) != 0;
    float w[VPL], total = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      w[j] = key[j] > kNoKey && rank[j] < p.top_k ? s[j] : 0.f;
      total += w[j];
    }
    const float over = p.renormalize ? p.scale / (row16_sum(total) + kTiny) : p.scale;
    if (there && !again) {
      const int64_t out = row * p.top_k;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        if (key[j] == kNoKey || rank[j] >= p.top_k) continue;
        p.ids[out + rank[j]] = base + j;
        p.weights[out + rank[j]] = w[j] * over;
      }
      for (int i = live + sub16; i < p.top_k; i += 16) p.ids[out + i] = -1, p.weights[out + i] = 0.f;
    }
  } else {
    const int need = min(p.top_k + (int)tell, live);  // at most 16
    // Of the lanes' largest keys, or their two largest, there are enough that reach the least of
    // them; `low` is reached by enough, `high` by too few.
    int best = key[0], second = kNoKey;
#pragma unroll
    for (int j = 1; j < VPL; ++j) {
      second = max(second, min(best, key[j]));
      best = max(best, key[j]);
    }
    int low = kNoKey + 1, high = row16_max(best) + 1;
    if (row16_sum((int)(best > kNoKey)) >= need) low = ~row16_max(best > kNoKey ? ~best : kLowest);
    else if (2 * row16_sum((int)(second > kNoKey)) >= need) low = ~row16_max(second > kNoKey ? ~second : kLowest);
    auto reach = [&](int t) {
      int n = 0;
#pragma unroll
      for (int j = 0; j < VPL; ++j) n += key[j] >= t;
      return row16_sum(n);
    };
    int found = reach(low);
    while (__ballot(found > 16 && (unsigned)high - (unsigned)low > 1) != 0) {
      const int mid = low + (int)(((unsigned)high - (unsigned)low) >> 1);
      const int n = reach(mid);
      if (found > 16 && (unsigned)high - (unsigned)low > 1) {
        if (n >= need) low = mid, found = n;
        else high = mid;
      }
    }
    open = open || found > 16;  // then this is another's work
    int2* const line = order[wave][mine];
    // The keys that reach t, in the order of experts, one for each of the first lanes.
    auto candidates = [&](int t) {
      int take = 0;
#pragma unroll
      for (int j = 0; j < VPL; ++j) take += key[j] >= t;
      int at = take;  // inclusive over the row's lanes
      at += dpp<kShift + 1>(0, at);
      at += dpp<kShift + 2>(0, at);
      at += dpp<kShift + 4>(0, at);
      at += dpp<kShift + 8>(0, at);
      at -= take;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        if (key[j] >= t && at < 16) line[at] = make_int2(key[j], base + j);
        at += key[j] >= t;
      }
      own_lds();
      return line[sub16];
    };
    // What is handed over comes to the lane of its rank.
    auto sorted = [&](int2 own, int rank, bool is) {
      if (is) line[16 + rank] = own;
      own_lds();
      return line[16 + sub16];
    };
    const int some = min(found, 16);
    int2 own = candidates(low);
    if (sub16 >= some) own.x = kNoKey;
    const int value[1] = {own.x}, number[1] = {sub16};
    int rank = 0;
    each_turn(value, [&](const int (&other)[1], auto) { rank += other[0] > own.x; });
    if (__ballot(row16_sum(sub16 < some ? rank : 0) != some * (some - 1) / 2) != 0) {  // equal keys go by their numbers
      each_turn(number, [&](const int (&other)[1], auto d) { rank += turned<decltype(d)::value>(own.x) == own.x && other[0] < sub16; });
    }
    int2 best_of = sorted(own, rank, sub16 < some);  // the row's sub16-th
    if (tell) {
      const int before = dpp<kShift + 1>(best_of.x, best_of.x), last = dpp<kShift + 1>(best_of.y, best_of.y);
      bool near = false;
      if (found <= 16 && sub16 > 0 && sub16 < need) {
        const float v = value_of(best_of.x);
        if (!(value_of(before) - v > slack + 0x1p-22f * fabsf(v)))
          near = true;
      }
      if (__ballot(near) != 0) {
        const bool at_edge = (__ballot(near && sub16 == p.top_k) >> (lane & 48) & 0xFFFF) != 0;
        if (near) near = !(logit(logits + last) == logit(logits + best_of.y) && p.bias[last] == p.bias[best_of.y]);
        if (at_edge) near = near || others_near(p, key, x, base, line[16 + p.top_k], slack, logits);
      }
      const uint64_t nears = __ballot(near);
      if (nears != 0) {  // ranked in FP64, with whatever could be among them
        const float t = value_of(low);
        const int lower = max(min(low, ordered(t - (slack + 0x1p-22f * fabsf(t)))), kNoKey + 1), more = reach(lower);
        const bool mend = (nears >> (lane & 48) & 0xFFFF) != 0;
        open = open || (mend && more > 16);
        const int2 other = candidates(lower);
        const Exactly exactly(p.sigmoid, top, x, 16);
        const bool is = mend && sub16 < more && more <= 16;
        const double k = is ? exactly.key(logit(logits + other.y), p.bias[other.y]) : (double)kNone;
        const uint64_t bits = __double_as_longlong(k);
        const int low_half[1] = {(int)(uint32_t)bits}, high_half[1] = {(int)(bits >> 32)};
        int place = 0;
        each_turn(low_half, [&](const int (&theirs)[1], auto d) {
          const uint64_t upper = (uint32_t)turned<decltype(d)::value>(high_half[0]);
          const double v = __longlong_as_double((int64_t)(upper << 32 | (uint32_t)theirs[0]));
          const int number = turned<decltype(d)::value>(sub16);  // by all lanes: those that are off have nothing to give
          place += v > k || (v == k && number < sub16);
        });
        const int2 exact = sorted(other, place, is);
        if (mend) best_of = exact;
      }
    }
    const bool chosen = sub16 < min(p.top_k, need) && found <= 16;
    left = __ballot(open && there);
    const bool again = (left >> (lane & 48) & 0xFFFF) != 0;
    float w = 0.f;
    if (chosen) {
      const float v = logit(logits + best_of.y);
      w = p.sigmoid ? sigmoid(v) : exp_near(v - top) * inverse;
    }
    const float over = p.renormalize ? p.scale / (row16_sum(w) + kTiny) : p.scale;
    if (there && !again && sub16 < p.top_k) {
      p.ids[row * p.top_k + sub16] = chosen ? best_of.y : -1;
      p.weights[row * p.top_k + sub16] = w * over;
    }
  }
  while (left != 0) {
    const int which = uniform((__ffsll((unsigned long long)left) - 1) >> 4);
    left &= ~(0xFFFFull << 16 * which);
    route_row<T, (VPL + 3) / 4>(p, first_row + which, lane, places[wave]);
  }
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

// Over the lanes of a row, 16 or the wave.
template <int LANES>
__device__ __forceinline__ float row_sum_of(float v) {
  if constexpr (LANES == 16) return row16_sum(v);
  else return wave_sum(v);
}

// LANES lanes hold a row, 16 or 64; expert lane + LANES j is a lane's j-th. The few gradients of
// the chosen scores are spread to their experts through LDS. 10007 rows of 160 experts in BF16 with
// a gradient of the scores 6.2 us (their bytes take 2.8): 217 vector instructions a row, and the
// latency of one; 16384 x 256 FP32 11.6 us, 4.3 TB/s.
template <typename T, int VPL, int LANES>
__global__ void __launch_bounds__(256) route_backward_kernel(const RouteGradParams p) {
  constexpr int kRows = 256 / LANES;
  __shared__ float spread[kRows][LANES * VPL];
  const int lane = threadIdx.x % LANES, at = LANES == 64 ? uniform(threadIdx.x / LANES) : threadIdx.x / LANES;
  const int64_t first = ((int64_t)p.first_group + blockIdx.x) * kRows;
  // rows past the last are done and not written, in a wave that has any before it
  if (first + (threadIdx.x & ~63) / LANES >= p.T) return;
  const int64_t row = LANES == 64 ? first + at : min(first + at, (int64_t)p.T - 1);
  const T* logits = static_cast<const T*>(p.logits) + row * p.ldl;
  float x[VPL], ds[VPL];
  int id = -1;
  float g = 0.f, xi = 0.f;
  if (lane < p.top_k) {
    id = p.ids[row * p.top_k + lane];
    g = p.dweights[row * p.top_k + lane] * p.scale;
  }
#pragma unroll
  for (int j = 0; j < VPL; ++j) x[j] = logit(logits + min(lane + LANES * j, p.E - 1));
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    ds[j] = p.dscores ? p.dscores[row * p.ldds + min(lane + LANES * j, p.E - 1)] : 0.f;
    spread[at][lane + LANES * j] = 0.f;
  }
#pragma unroll
  for (int j = 0; j < VPL; ++j) x[j] = lane + LANES * j < p.E ? x[j] : kNone;
  if ((unsigned)id >= (unsigned)p.E) id = -1, g = 0.f;
  if (id >= 0) xi = logit(logits + id);
  float top = 0.f, inverse = 0.f;
  if (!p.sigmoid) {
    float most = kNone, total = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) most = fmaxf(most, x[j]);
    const int bits = LANES == 16 ? row16_max(ordered(most)) : wave_max(ordered(most));
    top = bits > kNoKey ? value_of(bits) : 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      x[j] = exp_near(x[j] - top);  // 0 past the experts
      total += x[j];
    }
    total = row_sum_of<LANES>(total);
    inverse = total == 0.f ? 0.f : 1.0f / total;
  }
  const float s = id < 0 ? 0.f : p.sigmoid ? sigmoid(xi) : exp_near(xi - top) * inverse;
  if (p.renormalize) {
    const float over = 1.0f / (row_sum_of<LANES>(s) + kTiny);
    g = (g - row_sum_of<LANES>(g * s) * over) * over;
  }
  own_lds();
  if (id >= 0) atomicAdd(&spread[at][id], g);
  own_lds();
  T* out = static_cast<T*>(p.dlogits) + row * p.lddl;
  float dot = 0.f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    ds[j] += spread[at][lane + LANES * j];
    if (!p.sigmoid) {
      x[j] *= inverse;
      dot += ds[j] * x[j];
    }
  }
  if (!p.sigmoid) dot = row_sum_of<LANES>(dot);
  if (first + at >= p.T) return;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = lane + LANES * j;
    float dx;
    if (p.sigmoid) dx = ds[j] == 0.f ? 0.f : ds[j] * sigmoid(x[j]) * sigmoid(-x[j]);  // 1 - s without a cancellation
    else dx = x[j] * (ds[j] - dot);
    if (e < p.E) set_logit(out + e, dx);
  }
}

}  // namespace fp8moe
