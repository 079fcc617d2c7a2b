// Device code of the residual RMS norm with 8-bit output, and of its gradient.
//
// A row is held in registers, as it is in memory, from its one read to its last write. A
// thread owns chunks of eight consecutive columns, chunk i of thread t at column
// 8 (t + i * threads), so that a wave reads and writes whole lines and the 16 lanes of one
// 128-column quantisation block are neighbours. WPR waves share a row, at most CH chunks a
// thread.
#pragma once

#include "common.hpp"

namespace fp8layer {

// Sum over a row's waves: `part` has a place for each wave of the workgroup.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* part, int wave) {
  v = wave_sum(v);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) part[wave] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) v += part[wave / WPR * WPR + i];
  }
  return v;
}

// Weights are BF16 or FP32, whatever the rows are.
__device__ __forceinline__ void load_weight(const void* w, int w_fp32, int c, float (&x)[8]) {
  if (w_fp32) load8(static_cast<const float*>(w) + c * 8, x);
  else load8(static_cast<const uint16_t*>(w) + c * 8, x);
}

struct NormParams {
  const void *X, *R, *w;
  void *H, *Y;
  float* rstd;
  uint8_t* Q;
  float* sa;
  int64_t ldx, ldr, ldh, ldy, ldq, ld_sa;
  float eps;
  int M, K, w_fp32;
  int first_group;  // the launch's first workgroup of the call's
};

// y / s for a scale s and r = 1 / s (rounded): one step of Markstein's division, which
// rounds correctly where r does; three instructions where a division takes ten.
__device__ __forceinline__ float quotient(float y, float s, float r) {
  const float q = y * r;
  return __builtin_fmaf(__builtin_fmaf(-q, s, y), r, q);
}

// Forward: sum of squares, then y = (h * rstd) * w in FP32, its maximum over the 16 lanes
// of a block, and the codes. Bound by memory: 4096 x 7168 BF16 with the residual 40.4 us,
// 5.1 TB/s (a large copy reaches 4.8 to 5.3); 1537 x 2048 FP32 6.8 us; one row of 7168
// 3.2 us, most of it the launch.
template <typename T, int WPR, int CH, bool STREAM>
__global__ void __launch_bounds__(WPR > 4 ? WPR * 64 : 256) rmsnorm_quantize_kernel(const NormParams p) {
  constexpr int kRows = WPR > 4 ? 1 : 4 / WPR;  // rows of a workgroup
  __shared__ float part[WPR > 4 ? WPR : 4];
  const int wave = threadIdx.x >> 6;
  const int t = WPR > 1 ? threadIdx.x : threadIdx.x & 63;
  const int row = (p.first_group + (int)blockIdx.x) * kRows + (WPR > 1 ? 0 : wave);
  if (row >= p.M) return;  // whole rows only: no wave of a shared row leaves
  const T* X = static_cast<const T*>(p.X) + (int64_t)row * p.ldx;
  const int chunks = p.K >> 3;
  Eight<T> h[CH];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + i * WPR * 64;
    if (c < chunks) h[i].template load<STREAM>(X + c * 8);
  }
  if (p.R) {
    const T* R = static_cast<const T*>(p.R) + (int64_t)row * p.ldr;
    T* H = static_cast<T*>(p.H) + (int64_t)row * p.ldh;
    Eight<T> r[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + i * WPR * 64;
      if (c < chunks) r[i].template load<STREAM>(R + c * 8);
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + i * WPR * 64;
      if (c < chunks) {
        float a[8], b[8];
        h[i].get(a);
        r[i].get(b);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] += b[j];
        h[i].set(a);  // rounded: what is normalised is what is stored
        h[i].store(H + c * 8);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    if (t + i * WPR * 64 < chunks) {
      float a[8];
      h[i].get(a);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += a[j] * a[j];
    }
  }
  ss = row_sum<WPR>(ss, part, wave);
  const float rstd = 1.0f / sqrtf(ss / (float)p.K + p.eps);
  if (p.rstd && t == 0) p.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + i * WPR * 64;
    if (c < chunks) {
      float y[8], w[8], amax = 0.f;
      h[i].get(y);
      load_weight(p.w, p.w_fp32, c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = y[j] * rstd * w[j];
        amax = fmaxf(amax, fabsf(y[j]));
      }
      if (p.Y) store8(static_cast<uint16_t*>(p.Y) + (int64_t)row * p.ldy + c * 8, y);
      amax = row_max(amax);
      float s = amax / kE4m3Max;
      if (!(s > 0.f)) s = 1.0f;
      const float r = 1.0f / s;
      if (s > 0x1p-100f && s < 0x1p100f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = quotient(y[j], s, r);
      } else {  // where r, or a product with it, could leave the normal range
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] /= s;
      }
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
  int M, K, w_fp32;
};

// Backward: workgroups of 16 waves, 16 / WPR rows at a time, one workgroup a CU, so that
// few hold partial sums of dW (in registers over all rows of the workgroup; 256 parts of
// 28 KB for 4096 rows of 7168 columns, against 235 MB read and written). The next rows are
// loaded before the present ones are reduced. Bound by memory: 4096 x 7168 BF16 with the
// residual stream's gradient 45.6 us with the sums' reduction, 5.1 TB/s.
template <typename T, int WPR, int CH, bool STREAM>
__global__ void __launch_bounds__(1024) rmsnorm_backward_kernel(const NormGradParams p) {
  constexpr int kRows = 16 / WPR;
  __shared__ float part[2][16];
  extern __shared__ float merge[];  // kRows > 1: [kRows - 1][K]
  const int wave = threadIdx.x >> 6, sub = wave / WPR;  // sub: which of the rows
  const int t = threadIdx.x & (WPR * 64 - 1);
  const int chunks = p.K >> 3;
  const int stride = gridDim.x * kRows;
  float w[CH][8], dw[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + i * WPR * 64;
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f, w[i][j] = 0.f;
    if (c < chunks) load_weight(p.w, p.w_fp32, c, w[i]);
  }
  Eight<T> dy[CH], h[CH], dh[CH];
  float rstd = 0.f;
  auto fetch = [&](int row) {
    if (row >= p.M) return;
    rstd = p.rstd[row];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + i * WPR * 64;
      if (c < chunks) {
        dy[i].template load<STREAM>(static_cast<const T*>(p.dY) + (int64_t)row * p.lddy + c * 8);
        h[i].template load<STREAM>(static_cast<const T*>(p.H) + (int64_t)row * p.ldh + c * 8);
        if (p.dH) dh[i].template load<STREAM>(static_cast<const T*>(p.dH) + (int64_t)row * p.lddh + c * 8);
      }
    }
  };
  int turn = 0;
  fetch(blockIdx.x * kRows + sub);
  // all rows of the workgroup take part in each turn's barrier, also where one is past M
  for (int first = blockIdx.x * kRows; first < p.M; first += stride, turn ^= 1) {
    const int row = first + sub;
    const bool live = row < p.M;
    Eight<T> dy0[CH], h0[CH], dh0[CH];
    const float r0 = rstd;
#pragma unroll
    for (int i = 0; i < CH; ++i) dy0[i] = dy[i], h0[i] = h[i], dh0[i] = dh[i];
    fetch(row + stride);
    float dot = 0.f;
    if (live) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        if (t + i * WPR * 64 < chunks) {
          float g[8], x[8];
          dy0[i].get(g);
          h0[i].get(x);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[j] *= r0;
            dw[i][j] += g[j] * x[j];
            dot += g[j] * w[i][j] * x[j];
          }
        }
      }
    }
    // the parts of successive turns alternate, so that one barrier a turn is enough
    dot = row_sum<WPR>(dot, part[turn], wave);
    const float mean = dot / (float)p.K;
    if (live) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = t + i * WPR * 64;
        if (c < chunks) {
          float g[8], x[8];
          dy0[i].get(g);
          h0[i].get(x);
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] = r0 * (g[j] * w[i][j] - x[j] * r0 * mean);
          if (p.dH) {
            dh0[i].get(x);
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] += x[j];
          }
          store8(static_cast<T*>(p.dX) + (int64_t)row * p.lddx + c * 8, g);
        }
      }
    }
  }
  if constexpr (kRows > 1) {  // the rows' sums, added in their order
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + i * WPR * 64;
      if (sub > 0 && c < chunks) store8(merge + (sub - 1) * p.K + c * 8, dw[i]);
    }
    __syncthreads();
    if (sub > 0) return;
    for (int k = 0; k < kRows - 1; ++k)
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = t + i * WPR * 64;
        if (c < chunks) {
          float x[8];
          load8(merge + k * p.K + c * 8, x);
#pragma unroll
          for (int j = 0; j < 8; ++j) dw[i][j] += x[j];
        }
      }
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + i * WPR * 64;
    if (c < chunks) store8(p.part + (int64_t)blockIdx.x * p.K + c * 8, dw[i]);
  }
}

// Backward of few rows, in one launch, for a dX that is not in dY's place (both are read by
// other workgroups while it is written): neither result needs the other, as rstd is given. The
// first workgroups sum dW of 128 bytes of columns each, a thread eight columns over every
// 128th (FP32: 256th) row; the others take 16 / WPR rows each for dX. The rows are read twice, by
// workgroups that are mostly on different XCDs: the second time from the last-level cache. 333 x 2048 FP32 4.9 us, 64 x 7168 BF16 3.7, where the kernels above
// take 7.4 and 7.6 and cost the host two launches.
template <typename T, int WPR>
__global__ void __launch_bounds__(1024) rmsnorm_backward_few_kernel(const NormGradParams p, float* dW) {
  constexpr int kWaves = 16, kRows = kWaves / WPR;
  constexpr int kLanes = 16 / sizeof(T), kCols = 8 * kLanes;  // of a slice: 128 bytes of a row
  __shared__ float part[kWaves];
  __shared__ __align__(16) float sums[kWaves][kCols];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int slices = p.K / kCols;
  if ((int)blockIdx.x < slices) {
    const int at = lane % kLanes * 8, c = blockIdx.x * kCols + at;
    float dw[8] = {};
#pragma unroll 4
    for (int row = threadIdx.x / kLanes; row < p.M; row += kWaves * 64 / kLanes) {
      float g[8], x[8];
      load8(static_cast<const T*>(p.dY) + row * p.lddy + c, g);
      load8(static_cast<const T*>(p.H) + row * p.ldh + c, x);
      const float r = p.rstd[row];
#pragma unroll
      for (int j = 0; j < 8; ++j) dw[j] += g[j] * (x[j] * r);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)  // over the wave's rows
#pragma unroll
      for (int off = kLanes; off < 64; off <<= 1) dw[j] += __shfl_xor(dw[j], off, 64);
    if (lane < kLanes) store8(&sums[wave][at], dw);
    __syncthreads();
    if (threadIdx.x < kCols) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) sum += sums[w][threadIdx.x];
      dW[blockIdx.x * kCols + threadIdx.x] = sum;
    }
    return;
  }
  const int row = ((int)blockIdx.x - slices) * kRows + wave / WPR;
  const int c = threadIdx.x & (WPR * 64 - 1);
  const bool live = row < p.M && c < p.K >> 3;  // the barrier below is for whole rows
  Eight<T> dy, h, dh;
  float w[8], r = 0.f, dot = 0.f;
  if (live) {
    r = p.rstd[row];
    dy.load(static_cast<const T*>(p.dY) + row * p.lddy + c * 8);
    h.load(static_cast<const T*>(p.H) + row * p.ldh + c * 8);
    if (p.dH) dh.load(static_cast<const T*>(p.dH) + row * p.lddh + c * 8);
    load_weight(p.w, p.w_fp32, c, w);
    float g[8], x[8];
    dy.get(g);
    h.get(x);
#pragma unroll
    for (int j = 0; j < 8; ++j) dot += g[j] * w[j] * (x[j] * r);
  }
  dot = row_sum<WPR>(dot, part, wave);
  if (!live) return;
  const float mean = dot / (float)p.K;
  float g[8], x[8];
  dy.get(g);
  h.get(x);
#pragma unroll
  for (int j = 0; j < 8; ++j) g[j] = r * (g[j] * w[j] - x[j] * r * mean);
  if (p.dH) {
    dh.get(x);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] += x[j];
  }
  store8(static_cast<T*>(p.dX) + row * p.lddx + c * 8, g);
}

// dW[k] = sum of the workgroups' parts, in a fixed order: four column quads by 64 slices of
// the parts a workgroup.
__global__ void __launch_bounds__(256) rmsnorm_weight_grad_kernel(const float* __restrict__ part, int parts, int K,
                                                                  float* __restrict__ dW) {
  __shared__ float4 slice[64][4];
  const int x = threadIdx.x & 3, y = threadIdx.x >> 2;
  const int k = (blockIdx.x * 4 + x) * 4;  // K is a multiple of 16
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int g = y; g < parts; g += 64) {
    const float4 v = *reinterpret_cast<const float4*>(part + (int64_t)g * K + k);
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  slice[y][x] = s;
  __syncthreads();
  if (threadIdx.x < 16) {  // one column each
    const float* column = reinterpret_cast<const float*>(slice) + threadIdx.x;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 64; ++i) sum += column[i * 16];
    dW[blockIdx.x * 16 + threadIdx.x] = sum;
  }
}

}  // namespace fp8layer
