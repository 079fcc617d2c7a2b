// Device code of the way back from experts to tokens: the weighted sum of a token's rows, and
// its gradients.
#pragma once

#include "common.hpp"

namespace fp8moe {

using namespace fp8layer;

struct CombineParams {
  const void *Y, *C;
  void* out;
  const int32_t* positions;
  const float* weights;
  int64_t ldy, ldc, ldo, rows;
  int T, top_k, N;
  int slices;       // of a row, 512 columns each
  int first_group;  // the launch's first workgroup of the call's
};

// A wave takes 512 columns of one token, eight a thread, and has the rows of eight choices in
// flight at once. Bound by memory: 4096 tokens of 8 rows of 7168 BF16 columns, added to C, 101 us,
// 5.8 TB/s; 64 tokens 3.8 us.
template <typename T, bool STREAM>
__global__ void __launch_bounds__(256) combine_kernel(const CombineParams p) {
  const int64_t unit = ((int64_t)p.first_group + blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t token = unit / p.slices;
  if (token >= p.T) return;
  const int column = (int)(unit - token * p.slices) * 512 + (threadIdx.x & 63) * 8;
  if (column >= p.N) return;
  float sum[8] = {};
  if (p.C) load8<STREAM>(static_cast<const T*>(p.C) + token * p.ldc + column, sum);
  const T* Y = static_cast<const T*>(p.Y) + column;
  for (int first = 0; first < p.top_k; first += 8) {
    Eight<T> y[8];
    float w[8];
    bool there[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      there[j] = false;
      if (first + j >= p.top_k) continue;
      const int64_t row = p.positions[token * p.top_k + first + j];
      there[j] = row >= 0 && row < p.rows;
      w[j] = p.weights ? p.weights[token * p.top_k + first + j] : 1.0f;
      if (there[j]) y[j].template load<STREAM>(Y + row * p.ldy);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!there[j]) continue;
      float v[8];
      y[j].get(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(w[j], v[i], sum[i]);
    }
  }
  store8(static_cast<T*>(p.out) + token * p.ldo + column, sum);
}

struct CombineGradParams {
  const void *dO, *Y;
  void* dY;
  const int32_t* positions;
  const float* weights;
  float* dweights;
  int64_t lddo, ldy, lddy, rows;
  int T, top_k, N;
  int first_group;
};

// A workgroup of WAVES waves takes one token: its gradient is read once for eight choices,
// whose rows are read, multiplied with it and written as the choice's gradient in one pass. Bound by
// memory: 4096 tokens of 8 rows of 7168 BF16 columns 205 us, 4.9 TB/s.
template <typename T, int WAVES, bool STREAM>
__global__ void __launch_bounds__(WAVES * 64) combine_backward_kernel(const CombineGradParams p) {
  __shared__ float part[WAVES][8];
  const int64_t token = (int64_t)p.first_group + blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const T* dO = static_cast<const T*>(p.dO) + token * p.lddo;
  for (int first = 0; first < p.top_k; first += 8) {
    int64_t row[8];
    float w[8], dot[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dot[j] = 0.f, row[j] = -1;
      if (first + j >= p.top_k) continue;
      row[j] = p.positions[token * p.top_k + first + j];
      if (row[j] >= p.rows) row[j] = -1;
      w[j] = p.weights[token * p.top_k + first + j];
    }
    for (uint32_t column = threadIdx.x * 8; column < (uint32_t)p.N; column += WAVES * 512) {  // past the last one below 2^32
      Eight<T> y[8];
      float g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (row[j] >= 0) y[j].template load<STREAM>(static_cast<const T*>(p.Y) + row[j] * p.ldy + column);
      load8(dO + column, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (row[j] < 0) continue;
        float v[8];
        y[j].get(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot[j] = __builtin_fmaf(g[i], v[i], dot[j]);
        if (p.dY) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = w[j] * g[i];
          store8(static_cast<T*>(p.dY) + row[j] * p.lddy + column, v);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) dot[j] = wave_sum(dot[j]);
    if (first > 0) __syncthreads();  // the last eight choices' sums have been read
    if (lane == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) part[wave][j] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < 8 && first + (int)threadIdx.x < p.top_k) {
      float sum = 0.f;
      for (int v = 0; v < WAVES; ++v) sum += part[v][threadIdx.x];
      p.dweights[token * p.top_k + first + threadIdx.x] = sum;
    }
  }
}

}  // namespace fp8moe
