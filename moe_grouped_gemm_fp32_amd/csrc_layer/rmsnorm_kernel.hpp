// Device code of the residual RMS norm with 8-bit output, and of its gradient.
//
// A row is held in registers from its one read to its last write. A thread owns chunks of
// eight consecutive columns, chunk i of thread t at column 8 (t + i * threads), so that a
// wave reads and writes whole lines and the 16 lanes of one 128-column quantisation block
// are neighbours. WPR waves share a row.
#pragma once

#include "common.hpp"

namespace fp8layer {

// A row of K columns over WPR waves: at most CH chunks a thread.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* part, int wave) {
  v = wave_sum(v);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) part[wave] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) v += part[i];
  }
  return v;
}

struct NormParams {
  const void *X, *R, *w;
  void *H, *Y;
  float* rstd;
  uint8_t* Q;
  float* sa;
  int64_t ldx, ldr, ldh, ldy, ldq, ld_sa;
  float eps;
  int M, K;
};

// Forward: sum of squares, then y = (h * rstd) * w in FP32, its maximum over the 16 lanes
// of a block, and the codes by a correctly rounded division (the quantiser's).
template <typename T, typename W, int WPR, int CH>
__global__ void __launch_bounds__(WPR > 4 ? WPR * 64 : 256) rmsnorm_quantize_kernel(const NormParams p) {
  constexpr int kRows = WPR > 4 ? 1 : 4 / WPR;  // rows of a workgroup
  __shared__ float part[WPR];
  const int wave = threadIdx.x >> 6;
  const int t = WPR > 1 ? threadIdx.x : threadIdx.x & 63;
  const int row = blockIdx.x * kRows + (WPR > 1 ? 0 : wave);
  if (row >= p.M) return;  // whole rows only: no wave of a shared row leaves
  const T* X = static_cast<const T*>(p.X) + (int64_t)row * p.ldx;
  const int chunks = p.K >> 3;
  float h[CH][8], w[CH][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + i * WPR * 64;
    if (c < chunks) {
      load8(X + c * 8, h[i]);
      if (p.R) {
        float r[8];
        load8(static_cast<const T*>(p.R) + (int64_t)row * p.ldr + c * 8, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = rounded<T>(h[i][j] + r[j]);
        store8(static_cast<T*>(p.H) + (int64_t)row * p.ldh + c * 8, h[i]);
      }
      load8(static_cast<const W*>(p.w) + c * 8, w[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += h[i][j] * h[i][j];
    }
  }
  ss = row_sum<WPR>(ss, part, wave);
  const float rstd = 1.0f / sqrtf(ss / (float)p.K + p.eps);
  if (p.rstd && t == 0) p.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + i * WPR * 64;
    if (c < chunks) {
      float y[8], amax = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = h[i][j] * rstd * w[i][j];
        amax = fmaxf(amax, fabsf(y[j]));
      }
      if (p.Y) store8(static_cast<uint16_t*>(p.Y) + (int64_t)row * p.ldy + c * 8, y);
      amax = row_max(amax);
      float s = amax / kE4m3Max;
      if (!(s > 0.f)) s = 1.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] /= s;
      *reinterpret_cast<uint2*>(p.Q + (int64_t)row * p.ldq + c * 8) = pack_e4m3(y);
      if ((c & 15) == 0) p.sa[(int64_t)(c >> 4) * p.ld_sa + row] = s;
    }
  }
}

struct NormGradParams {
  const void *dY, *H, *dH, *w;
  const float* rstd;
  void* dX;
  float* part;  // [gridDim.x][K]: each workgroup's sums for dW
  int64_t lddy, ldh, lddh, lddx;
  int M, K;
};

// Backward: each workgroup takes every gridDim.x-th row (WPR == 1: group of four rows) and
// keeps its columns' part of dW in registers over them.
template <typename T, typename W, int WPR, int CH>
__global__ void __launch_bounds__(WPR > 4 ? WPR * 64 : 256) rmsnorm_backward_kernel(const NormGradParams p) {
  constexpr int kRows = WPR > 4 ? 1 : 4 / WPR;
  __shared__ float part[2][WPR];
  __shared__ float merge[WPR == 1 ? 3 * CH * 512 : 1];
  const int wave = threadIdx.x >> 6;
  const int t = WPR > 1 ? threadIdx.x : threadIdx.x & 63;
  const int chunks = p.K >> 3;
  float w[CH][8], dw[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + i * WPR * 64;
    if (c < chunks) load8(static_cast<const W*>(p.w) + c * 8, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  }
  int turn = 0;
  for (int row = blockIdx.x * kRows + (WPR > 1 ? 0 : wave); row < p.M; row += gridDim.x * kRows, turn ^= 1) {
    const float rstd = p.rstd[row];
    float dy[CH][8], xh[CH][8];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + i * WPR * 64;
      if (c < chunks) {
        load8(static_cast<const T*>(p.dY) + (int64_t)row * p.lddy + c * 8, dy[i]);
        load8(static_cast<const T*>(p.H) + (int64_t)row * p.ldh + c * 8, xh[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          xh[i][j] *= rstd;
          dw[i][j] += dy[i][j] * xh[i][j];
          dy[i][j] *= w[i][j];
          dot += dy[i][j] * xh[i][j];
        }
      }
    }
    // the parts of successive rows alternate, so that one barrier a row is enough
    dot = row_sum<WPR>(dot, part[turn], wave);
    const float mean = dot / (float)p.K;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + i * WPR * 64;
      if (c < chunks) {
        float dx[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) dx[j] = rstd * (dy[i][j] - xh[i][j] * mean);
        if (p.dH) {
          float dh[8];
          load8(static_cast<const T*>(p.dH) + (int64_t)row * p.lddh + c * 8, dh);
#pragma unroll
          for (int j = 0; j < 8; ++j) dx[j] += dh[j];
        }
        store8(static_cast<T*>(p.dX) + (int64_t)row * p.lddx + c * 8, dx);
      }
    }
  }
  if constexpr (WPR == 1) {  // the four waves hold the same columns: add them up in wave 0
    if (wave > 0) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) merge[((wave - 1) * CH * 8 + i * 8 + j) * 64 + t] = dw[i][j];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] += merge[(k * CH * 8 + i * 8 + j) * 64 + t];
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + i * WPR * 64;
    if (c < chunks) store8(p.part + (int64_t)blockIdx.x * p.K + c * 8, dw[i]);
  }
}

// dW[k] = sum of the workgroups' parts, in a fixed order: 16 column quads by 16 slices of
// the parts a workgroup.
__global__ void __launch_bounds__(256) rmsnorm_weight_grad_kernel(const float* __restrict__ part, int parts, int K,
                                                                  float* __restrict__ dW) {
  __shared__ float4 slice[16][16];
  const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
  const int k = (blockIdx.x * 16 + x) * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (k < K) {
    for (int g = y; g < parts; g += 16) {
      const float4 v = *reinterpret_cast<const float4*>(part + (int64_t)g * K + k);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
  }
  slice[y][x] = s;
  __syncthreads();
  if (y == 0 && k < K) {
    for (int i = 1; i < 16; ++i) {
      const float4 v = slice[i][x];
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    dW[k] = s.x, dW[k + 1] = s.y, dW[k + 2] = s.z, dW[k + 3] = s.w;
  }
}

}  // namespace fp8layer
