// What the host sides of the layer operators share: checks of arguments, the device, launches,
// and the step from run-time to compile-time choices.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "fp8gemm.h"

namespace {

constexpr int kMaxDevices = 64;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// FP8GEMM_OK and the current device's compute units if it is a gfx950. The units are capped
// by fp8_gemm_set_num_cus, like those of the GEMMs' grids.
int device(int* cus) {
  struct Info {
    int status = 1, cus = 0;
  };
  static Info infos[kMaxDevices];
  static std::mutex mutex;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return FP8GEMM_ERR_DEVICE;
  std::lock_guard<std::mutex> lock(mutex);
  Info& d = infos[dev];
  if (d.status == 1) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return FP8GEMM_ERR_DEVICE;
    d.cus = prop.multiProcessorCount;
    d.status = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? FP8GEMM_OK : FP8GEMM_ERR_DEVICE;
  }
  const int cap = fp8_gemm_get_num_cus();
  *cus = cap > 0 ? std::min(cap, d.cus) : d.cus;
  return d.status;
}

// Launches so many workgroups in slices: a launch takes less than 2^32 threads, and those past
// that are left out without an error. f(first, groups) launches one slice.
template <typename F>
void in_slices(int64_t groups, int threads, F f) {
  const int64_t most = UINT32_MAX / threads;
  for (int64_t first = 0; first < groups; first += most) f((int)first, dim3((unsigned)std::min(most, groups - first)));
}
int launched() { return hipGetLastError() == hipSuccess ? FP8GEMM_OK : FP8GEMM_ERR_LAUNCH; }

bool norm_dtype(int t) { return t == FP8GEMM_QUANT_BF16 || t == FP8GEMM_QUANT_FP32; }
// row stride of a [.., K] array of x_dtype elements whose rows are read 16 bytes at a time
bool norm_rows(const void* p, int64_t ld, int K, int dtype) {
  return aligned(p, 16) && ld >= K && ld % (dtype == FP8GEMM_QUANT_BF16 ? 8 : 4) == 0;
}

// Whether M rows of K columns, `bytes` each, are read with the hint that they are read once:
// above 32 MB, the sum of the eight L2 caches, each of which gets its own workgroups' rows. 4096
// x 7168 BF16, without and with: norm 46.0 and 40.5 us, gradient 49.0 and 45.6; the gradient of
// 333 x 2048 FP32, 5 MB: 7.3 and 8.0.
bool streams(int M, int64_t K, size_t bytes) { return (size_t)M * K * bytes > ((size_t)32 << 20); }

// Calls f(T{}) with the rows' type; values and flags as compile-time arguments.
template <int N>
using Int = std::integral_constant<int, N>;
template <typename F>
void with_type(int dtype, F f) {
  if (dtype == FP8GEMM_QUANT_BF16) f(uint16_t{});
  else f(float{});
}
template <typename F>
void with_flag(bool flag, F f) {
  if (flag) f(std::true_type{});
  else f(std::false_type{});
}

}  // namespace
