// Small device helpers shared by the layer operators' kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8layer {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr float kE4m3Max = 448.0f;

// Eight consecutive elements as they are in memory (BF16 bits or FP32), 16-byte aligned.
template <typename T>
struct Eight {
  uint4 v[sizeof(T) / 2];
  // STREAM: with the hint that the lines are read once.
  template <bool STREAM = false>
  __device__ __forceinline__ void load(const T* src) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      if constexpr (STREAM) v[i] = __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const v4u*>(src) + i));
      else v[i] = reinterpret_cast<const uint4*>(src)[i];
    }
  }
  __device__ __forceinline__ void store(T* dst) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(dst)[i] = v[i];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (sizeof(T) == 2) {
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
      x[0] = __uint_as_float(v[0].x), x[1] = __uint_as_float(v[0].y), x[2] = __uint_as_float(v[0].z), x[3] = __uint_as_float(v[0].w);
      x[4] = __uint_as_float(v[1].x), x[5] = __uint_as_float(v[1].y), x[6] = __uint_as_float(v[1].z), x[7] = __uint_as_float(v[1].w);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8]);
};

template <bool STREAM = false, typename T>
__device__ __forceinline__ void load8(const T* src, float (&x)[8]) {
  Eight<T> e;
  e.template load<STREAM>(src);
  e.get(x);
}

// Two FP32 values rounded to nearest even BF16, packed.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{a, b}, v2bf));
}

// Rounds eight FP32 values to T.
template <typename T>
__device__ __forceinline__ void Eight<T>::set(const float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    v[0] = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  } else {
    v[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    v[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* dst, const float (&x)[8]) {
  Eight<T> e;
  e.set(x);
  e.store(dst);
}

// Eight FP32 values to e4m3 codes, round to nearest even.
__device__ __forceinline__ uint2 pack_e4m3(const float (&x)[8]) {
  int a = 0, b = 0;
  a = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], a, false);
  a = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], a, true);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], b, false);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], b, true);
  return make_uint2((uint32_t)a, (uint32_t)b);
}

// Reductions and prefix sums over the wave's lanes, by data-parallel primitives (a few
// cycles a step, where a shuffle goes through LDS). Within a row of 16 lanes: quad
// permutations, then mirrored halves and rows; over rows: the last lane of a row
// broadcast into the next ones.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ int dpp(int old, int v) {
  return __builtin_amdgcn_update_dpp(old, v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float dpp(float old, float v) {
  return __int_as_float(dpp<CTRL, ROWS>(__float_as_int(old), __float_as_int(v)));
}
constexpr int kSwap1 = 0xB1, kSwap2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;  // of a row's lanes
constexpr int kShift = 0x110, kLast15 = 0x142, kLast31 = 0x143;

// Inclusive prefix sum.
template <typename T>
__device__ __forceinline__ T wave_scan(T v) {
  v += dpp<kShift + 1>(T(0), v);
  v += dpp<kShift + 2>(T(0), v);
  v += dpp<kShift + 4>(T(0), v);
  v += dpp<kShift + 8>(T(0), v);
  v += dpp<kLast15, 0xA>(T(0), v);
  v += dpp<kLast31, 0xC>(T(0), v);
  return v;
}

__device__ __forceinline__ float last_lane(float v) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63)); }
__device__ __forceinline__ int last_lane(int v) { return __builtin_amdgcn_readlane(v, 63); }

__device__ __forceinline__ float wave_sum(float v) { return last_lane(wave_scan(v)); }

// Maximum over the lane's row of 16, in every lane of it.
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, dpp<kSwap1>(v, v));
  v = fmaxf(v, dpp<kSwap2>(v, v));
  v = fmaxf(v, dpp<kHalfMirror>(v, v));
  return fmaxf(v, dpp<kMirror>(v, v));
}

// Maximum over the wave.
__device__ __forceinline__ float wave_max(float v) {
  v = row_max(v);
  v = fmaxf(v, dpp<kLast15, 0xA>(v, v));
  v = fmaxf(v, dpp<kLast31, 0xC>(v, v));
  return last_lane(v);
}

// The part of a sequence that a call concerns, from its device arrays, clamped to what
// the call's host arguments allow (nothing read from these arrays becomes an address
// unchecked). Only what is held is clamped to the table, not where the rows stand: a row
// past the table's slots has its own position and no slot.
struct Sequence {
  int row0;   // its first row among the call's tokens
  int rows;   // its number of rows
  int start;  // position of the first row: below 0 for more rows than the sequence is long
  int len;    // its slots that the table can hold
};
__device__ __forceinline__ Sequence sequence(const int32_t* cu_q, const int32_t* seq_lens, int b, int T, int max_len) {
  const int q0 = min(max(cu_q[b], 0), T);
  const int q1 = min(max(cu_q[b + 1], q0), T);
  const int len = max(seq_lens[b], 0);
  return {q0, q1 - q0, len - (q1 - q0), min(len, max_len)};
}

}  // namespace fp8layer
