// Device code of the dispatch of tokens to experts: a stable counting sort of the choices by
// expert, and the copy of the tokens' 8-bit rows and scales to their places.
//
// The choices are cut into pieces of kPiece, a workgroup each. Counting: a histogram of each
// piece. Placing: each workgroup adds up the histograms before its own and all of them, which
// gives every expert's segment and the first place of its own choices in it; equal experts
// among 64 choices are found by comparing the bits of their numbers across the wave, so a
// place depends on the order of choices alone, not on that of any atomics.
#pragma once

#include "common.hpp"

namespace fp8moe {

using namespace fp8layer;

constexpr int kMaxExperts = 1024;
constexpr int kPiece = 1024;   // choices of a counting or placing workgroup
constexpr int kAlign = 128;    // rows that a segment of the contiguous layout begins at multiples of

struct LayoutParams {
  const int32_t* ids;
  int32_t* counted;  // [pieces][E]
  int32_t *positions, *sources, *m_indices, *counts;
  int64_t rows;
  int n, E, bits, max_m, pieces;
};

// Histogram of a piece.
__global__ void __launch_bounds__(256) count_kernel(const LayoutParams p) {
  __shared__ int32_t histogram[kMaxExperts];
  for (int e = threadIdx.x; e < p.E; e += 256) histogram[e] = 0;
  __syncthreads();
  const int first = blockIdx.x * kPiece, last = min(first + kPiece, p.n);
  for (int i = first + threadIdx.x; i < last; i += 256) {
    const int id = p.ids[i];
    if ((unsigned)id < (unsigned)p.E) atomicAdd(&histogram[id], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += 256) p.counted[(int64_t)blockIdx.x * p.E + e] = histogram[e];
}

// Exclusive prefix sums of value(e), e < E, into out[0 .. E]; all 256 threads, at most 4 experts each.
template <typename F>
__device__ __forceinline__ void prefix(int E, int32_t* out, int32_t* waves, F value) {
  const int each = (E + 255) / 256, begin = threadIdx.x * each;
  int sum = 0;
  for (int j = 0; j < each; ++j) sum += begin + j < E ? value(begin + j) : 0;
  const int scan = wave_scan(sum), wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 63) waves[wave] = scan;
  __syncthreads();
  int at = scan - sum;
  for (int w = 0; w < wave; ++w) at += waves[w];
  for (int j = 0; j < each; ++j) {
    if (begin + j > E) break;
    out[begin + j] = at;
    at += begin + j < E ? value(begin + j) : 0;
  }
  if (begin + each == E) out[E] = at;
  __syncthreads();
}

// Lanes whose number equals this lane's, among those that are `there`.
__device__ __forceinline__ uint64_t equals(int v, bool there, int bits) {
  uint64_t same = __ballot(there);
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((v >> b) & 1);
    same &= (v >> b) & 1 ? set : ~set;
  }
  return same;
}

// The layout. Workgroup b places the choices of its piece and marks its share of the rows
// that hold none. LOCAL: the histograms are counted here, by every workgroup for itself.
template <bool LOCAL>
__global__ void __launch_bounds__(256) place_kernel(const LayoutParams p) {
  __shared__ int32_t total[kMaxExperts], start[kMaxExperts + 1], at[4][kMaxExperts], waves[4];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int first = blockIdx.x * kPiece;
  for (int e = threadIdx.x; e < p.E; e += 256) {
    int before = 0, sum = 0;
    if constexpr (!LOCAL) {
#pragma unroll 8
      for (int b = 0; b < p.pieces; ++b) {
        const int c = p.counted[(int64_t)b * p.E + e];
        before += b < (int)blockIdx.x ? c : 0;
        sum += c;
      }
    }
    total[e] = sum;
    at[0][e] = before;
    at[1][e] = at[2][e] = at[3][e] = 0;
  }
  __syncthreads();
  if constexpr (LOCAL) {
    for (int i = threadIdx.x; i < p.n; i += 256) {
      const int id = p.ids[i];
      if ((unsigned)id >= (unsigned)p.E) continue;
      atomicAdd(&total[id], 1);
      if (i < first) atomicAdd(&at[0][id], 1);
    }
    __syncthreads();
  }
  if (p.max_m == 0) {
    prefix(p.E, start, waves, [&](int e) { return (total[e] + kAlign - 1) / kAlign * kAlign; });
  } else {
    for (int e = threadIdx.x; e <= p.E; e += 256) start[e] = e * p.max_m;
    __syncthreads();
  }
  // A quarter of the piece for each wave: how many it has of each expert ..
  constexpr int kShare = kPiece / 4;
  const int begin = first + wave * kShare;
  int ids[kShare / 64];
#pragma unroll
  for (int i = 0; i < kShare / 64; ++i) {
    const int c = begin + i * 64 + lane;
    ids[i] = c < p.n ? p.ids[c] : -1;
    if ((unsigned)ids[i] >= (unsigned)p.E) ids[i] = -1;
    if (ids[i] >= 0 && wave < 3) atomicAdd(&at[wave + 1][ids[i]], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += 256) {
    int sum = at[0][e];
    for (int w = 1; w < 4; ++w) sum += at[w][e], at[w][e] = sum;
  }
  __syncthreads();
  // .. then their ranks in the expert's segment, 64 choices at a time.
#pragma unroll
  for (int i = 0; i < kShare / 64; ++i) {
    const int c = begin + i * 64 + lane, id = ids[i];
    const uint64_t same = equals(id, id >= 0, p.bits);
    if (id >= 0) {
      const int rank = at[wave][id] + __popcll(same & ((1ull << lane) - 1));
      const int64_t row = (int64_t)start[id] + rank;
      const bool fits = p.max_m ? rank < p.max_m : row < p.rows;
      p.positions[c] = fits ? (int)row : -1;
      if (fits) p.sources[row] = c;
    } else if (c < p.n) {
      p.positions[c] = -1;
    }
    __builtin_amdgcn_wave_barrier();  // every lane has read its count before it grows
    if (id >= 0 && (same >> lane) == 1) at[wave][id] += __popcll(same);
    __builtin_amdgcn_wave_barrier();
  }
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e < p.E; e += 256) {
      const int64_t room = p.max_m ? p.max_m : max((int64_t)0, p.rows - start[e]);
      p.counts[e] = (int)min((int64_t)total[e], room);
    }
  }
  // The rows' marks: 128 at a time, which lie in one segment of the contiguous layout.
  const int64_t blocks = (p.rows + 127) / 128;
  for (int64_t b = (int64_t)blockIdx.x * 4 + wave; b < blocks; b += (int64_t)gridDim.x * 4) {
    if (p.max_m) {
      for (int64_t r = b * 128 + lane; r < min(b * 128 + 128, p.rows); r += 64) {
        const int e = (int)(r / p.max_m);
        if ((int)(r - (int64_t)e * p.max_m) >= total[e]) p.sources[r] = -1;
      }
      continue;
    }
    // the last expert whose segment begins at or before the block; an empty one shares its place with the next
    int low = 0, high = p.E - 1;
    while (low < high) {
      const int mid = (low + high + 1) / 2;
      if (start[mid] <= b * 128) low = mid;
      else high = mid - 1;
    }
    const int64_t end = (int64_t)start[low] + total[low];
    for (int64_t r = b * 128 + lane; r < b * 128 + 128; r += 64) {
      p.m_indices[r] = r < end ? low : -1;
      if (r >= end) p.sources[r] = -1;
    }
  }
}

struct GatherParams {
  const uint8_t* Q;
  const float *sa, *weights;
  uint8_t* Qx;
  float* sax;
  const int32_t *positions, *sources;
  int64_t ldq, ld_sa, ldqx, ld_sax, rows;
  int max_m, T, top_k, E, K;
  int slices;        // of a row's codes, kSlice bytes each
  int64_t code_groups;  // workgroups that copy codes; the later ones copy scales
  int row_groups;    // runs of 64 rows: of the contiguous layout, or of each expert's rows
  int first_group;   // the launch's first workgroup of the call's
};

constexpr int kSlice = 64 * 16 * 4;   // bytes of a row that a wave holds
constexpr int kScaleBlocks = 8;       // K blocks of a wave's scales

// Rows and scales. A wave reads a slice of a token's codes once and writes it to each of the
// token's places. Scales, which lie across the rows, are copied the other way: a wave takes
// 64 neighbouring rows, whose scales it writes as whole lines.
__global__ void __launch_bounds__(256) gather_kernel(const GatherParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t group = (int64_t)p.first_group + blockIdx.x;
  if (group < p.code_groups) {
    const int64_t unit = group * 4 + (threadIdx.x >> 6);
    const int64_t token = unit / p.slices;
    if (token >= p.T) return;
    const int column = (int)(unit - token * p.slices) * kSlice + lane * 16;
    const uint8_t* from = p.Q + token * p.ldq + column;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (column + i * 1024 < p.K) v[i] = *reinterpret_cast<const uint4*>(from + i * 1024);
    for (int j = 0; j < p.top_k; ++j) {
      const int64_t row = p.positions[token * p.top_k + j];
      if (row < 0 || row >= p.rows) continue;
      uint8_t* to = p.Qx + row * p.ldqx + column;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (column + i * 1024 < p.K) *reinterpret_cast<uint4*>(to + i * 1024) = v[i];
    }
    return;
  }
  const int blocks = p.K >> 7, parts = (blocks + kScaleBlocks - 1) / kScaleBlocks;
  const int64_t unit = (group - p.code_groups) * 4 + (threadIdx.x >> 6);
  const int64_t run = unit / parts;
  const int first = (int)(unit - run * parts) * kScaleBlocks;
  int64_t row, column;
  float* to = p.sax;
  if (p.max_m) {
    const int64_t e = run / p.row_groups;
    if (e >= p.E) return;
    column = (run - e * p.row_groups) * 64 + lane;
    row = column < p.max_m ? e * p.max_m + column : p.rows;
    to += e * blocks * p.ld_sax;
  } else {
    if (run >= p.row_groups) return;
    row = column = run * 64 + lane;
  }
  const int source = row < p.rows ? p.sources[row] : -1;
  if (source < 0 || source >= (int64_t)p.T * p.top_k) return;
  const int token = source / p.top_k;
  const float w = p.weights ? p.weights[source] : 1.0f;
  const float* from = p.sa + token;
#pragma unroll
  for (int i = 0; i < kScaleBlocks; ++i)
    if (first + i < blocks) to[(first + i) * p.ld_sax + column] = from[(first + i) * p.ld_sa] * w;
}

}  // namespace fp8moe
