// Device code of the norm of queries and keys for each head with their rotation, and of its
// gradients.
//
// D / 16 lanes hold a head, each two groups of eight of its columns that hold whole pairs: of
// halves, both members of eight pairs; interleaved, four pairs in each group. So neither the
// rotation nor the norm needs another lane's columns, only the sum of squares (or the gradient's
// dot product) goes over the lanes. The first groups of neighbouring lanes are neighbours, and so
// are the second ones: a load reads 64 bytes or more in a piece.
#pragma once

#include "common.hpp"

namespace fp8moe {

using namespace fp8layer;

// The first columns of a lane's two groups, and whether they turn.
struct Columns {
  int lo, hi;
  bool lo_turns, hi_turns;
};
template <int D>
__device__ __forceinline__ Columns columns_of(int i, int rot_dim, int interleaved) {
  if (interleaved) return {8 * i, D / 2 + 8 * i, 8 * i < rot_dim, D / 2 + 8 * i < rot_dim};
  if (16 * i < rot_dim) return {8 * i, (rot_dim >> 1) + 8 * i, true, true};
  const int rest = rot_dim + 8 * (i - (rot_dim >> 4));
  return {rest, rest + ((D - rot_dim) >> 1), false, false};
}

// Cosines and sines of a lane's pairs; interleaved, four of each group.
struct Angles {
  float c[8], s[8];
  __device__ __forceinline__ void load(const float* row, const Columns& at, int rot_dim, int interleaved) {
    const float* sines = row + (rot_dim >> 1);
    if (!interleaved) {
      if (!at.lo_turns) return;
      load8(row + at.lo, c);
      load8(sines + at.lo, s);
      return;
    }
    auto four = [](const float* from, float* to) {
      const float4 v = *reinterpret_cast<const float4*>(from);
      to[0] = v.x, to[1] = v.y, to[2] = v.z, to[3] = v.w;
    };
    if (at.lo_turns) four(row + at.lo / 2, c), four(sines + at.lo / 2, s);
    if (at.hi_turns) four(row + at.hi / 2, c + 4), four(sines + at.hi / 2, s + 4);
  }
  // Turns the pairs of a and b (BACK: by the angles' negatives).
  template <bool BACK>
  __device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const Columns& at, int interleaved) const {
    auto pair = [](float& x1, float& x2, float cosine, float sine) {
      const float y = BACK ? -sine : sine, x = x1;
      x1 = x * cosine - x2 * y;
      x2 = x2 * cosine + x * y;
    };
    if (!interleaved) {
      if (!at.lo_turns) return;
#pragma unroll
      for (int j = 0; j < 8; ++j) pair(a[j], b[j], c[j], s[j]);
      return;
    }
    if (at.lo_turns) {
#pragma unroll
      for (int j = 0; j < 4; ++j) pair(a[2 * j], a[2 * j + 1], c[j], s[j]);
    }
    if (at.hi_turns) {
#pragma unroll
      for (int j = 0; j < 4; ++j) pair(b[2 * j], b[2 * j + 1], c[4 + j], s[4 + j]);
    }
  }
};

// Sum over LANES (4, 8 or 16) neighbouring lanes, in every one of them.
template <int LANES>
__device__ __forceinline__ float head_sum(float v) {
  v += dpp<kSwap1>(v, v);
  v += dpp<kSwap2>(v, v);
  if constexpr (LANES >= 8) v += dpp<kHalfMirror>(v, v);
  if constexpr (LANES >= 16) v += dpp<kMirror>(v, v);
  return v;
}

__device__ __forceinline__ void head_weight(const void* w, int w_fp32, int c, float (&x)[8]) {
  if (w_fp32) load8(static_cast<const float*>(w) + c, x);
  else load8(static_cast<const uint16_t*>(w) + c, x);
}

struct HeadsParams {
  const void *q, *k, *qw, *kw;
  void *q_out, *k_out;
  const float* cos_sin;
  const int32_t* positions;
  int64_t ldq, ldk, ldqo, ldko, ld_cs;
  float eps;
  int T, Hq, Hk, w_fp32, max_pos, rot_dim, interleaved;
  int first_group;  // the launch's first workgroup of the call's
};

// One head for D / 16 lanes. Bound by memory: 8192 tokens of 40 heads of 128 BF16 columns 37 us,
// 4.6 TB/s; 64 tokens 3.5 us.
template <typename T, int D, bool STREAM>
__global__ void __launch_bounds__(256) heads_kernel(const HeadsParams p) {
  constexpr int kLanes = D / 16, kHeads = 256 / kLanes;
  const int64_t item = ((int64_t)p.first_group + blockIdx.x) * kHeads + threadIdx.x / kLanes;
  const int i = threadIdx.x % kLanes, heads = p.Hq + p.Hk;
  const int token = (int)((uint32_t)item / (uint32_t)heads);
  if (token >= p.T) return;
  int h = (int)item - token * heads;
  const bool key = h >= p.Hq;
  if (key) h -= p.Hq;
  const Columns at = columns_of<D>(i, p.rot_dim, p.interleaved);
  const T* x = key ? static_cast<const T*>(p.k) + token * p.ldk + h * D : static_cast<const T*>(p.q) + token * p.ldq + h * D;
  T* y = key ? static_cast<T*>(p.k_out) + token * p.ldko + h * D : static_cast<T*>(p.q_out) + token * p.ldqo + h * D;
  float a[8], b[8], wa[8], wb[8];
  Angles angles;
  load8<STREAM>(x + at.lo, a);
  load8<STREAM>(x + at.hi, b);
  if (at.lo_turns) {  // where the second group turns, the first does
    const int position = min(max(p.positions ? p.positions[token] : token, 0), p.max_pos - 1);
    angles.load(p.cos_sin + position * p.ld_cs, at, p.rot_dim, p.interleaved);
  }
  const void* w = key ? p.kw : p.qw;
  head_weight(w, p.w_fp32, at.lo, wa);
  head_weight(w, p.w_fp32, at.hi, wb);
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) ss += a[j] * a[j] + b[j] * b[j];
  const float rstd = 1.0f / sqrtf(head_sum<kLanes>(ss) * (1.0f / D) + p.eps);
#pragma unroll
  for (int j = 0; j < 8; ++j) a[j] *= rstd * wa[j], b[j] *= rstd * wb[j];
  angles.turn<false>(a, b, at, p.interleaved);
  store8(y + at.lo, a);
  store8(y + at.hi, b);
}

struct HeadsGradParams {
  const void *dq, *dk, *q, *k, *qw, *kw;
  void *dq_out, *dk_out;
  const float* cos_sin;
  const int32_t* positions;
  float* part;  // [gridDim.x][D]: each workgroup's sums for its weight's gradient
  int64_t lddq, lddk, ldq, ldk, lddqo, lddko, ld_cs;
  float eps;
  int T, Hq, Hk, w_fp32, max_pos, rot_dim, interleaved;
  int q_groups;  // workgroups of queries; the others take keys
};

// A workgroup takes heads of queries, or of keys, and keeps its sums for dw in registers over
// all of them. Loading the next heads while the present ones are worked on changed nothing
// (5003 x 32 heads of 64: 19.2 us with, 18.9 without, both launches). Bound by memory where heads
// are many (6000 x 80 of 64 40.8 us with the launch below, 4.5 TB/s); 5003 x 32 15.2 us, and 4 below.
template <typename T, int D>
__global__ void __launch_bounds__(256) heads_backward_kernel(const HeadsGradParams p) {
  constexpr int kLanes = D / 16, kHeads = 256 / kLanes;
  __shared__ __align__(16) float sums[16][D];  // a row of 16 lanes each
  const bool key = (int)blockIdx.x >= p.q_groups;
  const int heads = key ? p.Hk : p.Hq;
  const int group = key ? blockIdx.x - p.q_groups : blockIdx.x, groups = key ? gridDim.x - p.q_groups : p.q_groups;
  const int i = threadIdx.x % kLanes;
  const Columns at = columns_of<D>(i, p.rot_dim, p.interleaved);
  const T* dy = static_cast<const T*>(key ? p.dk : p.dq);
  const T* x = static_cast<const T*>(key ? p.k : p.q);
  T* dx = static_cast<T*>(key ? p.dk_out : p.dq_out);
  const int64_t lddy = key ? p.lddk : p.lddq, ldx = key ? p.ldk : p.ldq, lddx = key ? p.lddko : p.lddqo;
  float wa[8], wb[8], da[8] = {}, db[8] = {};
  const void* w = key ? p.kw : p.qw;
  head_weight(w, p.w_fp32, at.lo, wa);
  head_weight(w, p.w_fp32, at.hi, wb);
  const int64_t items = (int64_t)p.T * heads, step = (int64_t)groups * kHeads;
  for (int64_t item = (int64_t)group * kHeads + threadIdx.x / kLanes; item < items; item += step) {
    const int token = (int)((uint32_t)item / (uint32_t)heads), h = (int)item - token * heads;
    float ga[8], gb[8], xa[8], xb[8];
    load8(dy + token * lddy + h * D + at.lo, ga);
    load8(dy + token * lddy + h * D + at.hi, gb);
    load8(x + token * ldx + h * D + at.lo, xa);
    load8(x + token * ldx + h * D + at.hi, xb);
    T* to = dx + token * lddx + h * D;
    if (at.lo_turns) {
      Angles angles;
      const int position = p.positions ? p.positions[token] : token;
      angles.load(p.cos_sin + min(max(position, 0), p.max_pos - 1) * p.ld_cs, at, p.rot_dim, p.interleaved);
      angles.turn<true>(ga, gb, at, p.interleaved);
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss += xa[j] * xa[j] + xb[j] * xb[j];
    const float rstd = 1.0f / sqrtf(head_sum<kLanes>(ss) * (1.0f / D) + p.eps);
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      xa[j] *= rstd, xb[j] *= rstd;
      da[j] += ga[j] * xa[j], db[j] += gb[j] * xb[j];
      ga[j] *= wa[j], gb[j] *= wb[j];
      dot += ga[j] * xa[j] + gb[j] * xb[j];
    }
    const float mean = head_sum<kLanes>(dot) * (1.0f / D);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      ga[j] = rstd * (ga[j] - xa[j] * mean);
      gb[j] = rstd * (gb[j] - xb[j] * mean);
    }
    store8(to + at.lo, ga);
    store8(to + at.hi, gb);
  }
  // over the heads of a row of lanes, then over the rows
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (kLanes <= 8) da[j] += dpp<kTurn + 8>(da[j], da[j]), db[j] += dpp<kTurn + 8>(db[j], db[j]);
    if constexpr (kLanes <= 4) da[j] += dpp<kTurn + 4>(da[j], da[j]), db[j] += dpp<kTurn + 4>(db[j], db[j]);
  }
  if ((threadIdx.x & 15) < kLanes) {
    store8(&sums[threadIdx.x >> 4][at.lo], da);
    store8(&sums[threadIdx.x >> 4][at.hi], db);
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < 16; ++v) sum += sums[v][threadIdx.x];
    p.part[(int64_t)blockIdx.x * D + threadIdx.x] = sum;
  }
}

// dw of queries, then of keys: the sums of their workgroups, in a fixed order, 16 columns a
// workgroup by 64 slices of the parts.
__global__ void __launch_bounds__(1024) heads_weight_grad_kernel(const float* __restrict__ part, int q_groups, int groups, int D,
                                                                 float* dqw, float* dkw) {
  __shared__ float waves[16][16];
  const bool key = (int)blockIdx.x * 16 >= D;
  float* to = key ? dkw : dqw;
  if (!to) return;
  const int column = blockIdx.x * 16 - (key ? D : 0) + (threadIdx.x & 15), slice = threadIdx.x >> 4;
  const int first = key ? q_groups : 0, last = key ? groups : q_groups;
  float sum = 0.f;
#pragma unroll 16
  for (int g = first + slice; g < last; g += 64) sum += part[(int64_t)g * D + column];
  sum += __shfl_xor(sum, 16, 64);
  sum += __shfl_xor(sum, 32, 64);
  if ((threadIdx.x & 63) < 16) waves[threadIdx.x >> 6][threadIdx.x & 15] = sum;
  __syncthreads();
  if (threadIdx.x >= 16) return;
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < 16; ++w) sum += waves[w][threadIdx.x];
  to[column] = sum;
}

}  // namespace fp8moe
