// Device code of the dispatch of tokens to experts: a stable counting sort of the choices by
// expert, and the copy of the tokens' 8-bit rows and scales to their places.
//
// Every place is the beginning of its expert's segment, plus the choices of that expert in
// the pieces before its own, plus those before it in the piece. Equal experts among 64
// choices are found by comparing the bits of their numbers across the wave, so a place
// depends on the order of choices alone, not on that of any atomics.
#pragma once

#include "common.hpp"

namespace fp8moe {

using namespace fp8layer;

constexpr int kMaxExperts = 1024;
constexpr int kPiece = 1024;     // choices of a counting or placing workgroup, a thread each
constexpr int kFewChoices = 64;  // of a workgroup that dispatches a few tokens at once
constexpr int kAlign = 128;      // rows that a segment of the contiguous layout begins at multiples of

struct LayoutParams {
  const int32_t* ids;
  int32_t* counted;  // [pieces + 1][E]: choices of each piece, then of those before it; last, all
  int32_t *positions, *sources, *m_indices, *counts;
  int64_t rows;
  int n, E, bits, max_m, pieces;
};

// Choices of each expert in a piece.
__global__ void __launch_bounds__(kPiece) count_kernel(const LayoutParams p) {
  __shared__ int32_t histogram[kMaxExperts];
  for (int e = threadIdx.x; e < p.E; e += kPiece) histogram[e] = 0;
  __syncthreads();
  const int c = blockIdx.x * kPiece + threadIdx.x;
  const int id = c < p.n ? p.ids[c] : -1;
  if ((unsigned)id < (unsigned)p.E) atomicAdd(&histogram[id], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kPiece) p.counted[(int64_t)blockIdx.x * p.E + e] = histogram[e];
}

// From the pieces' counts those of the pieces before each, and the sums. 64 experts a
// workgroup, a lane each; the pieces are cut among the waves, and read twice.
__global__ void __launch_bounds__(1024) scan_kernel(const LayoutParams p) {
  __shared__ int32_t sums[16][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, e = blockIdx.x * 64 + lane;
  const int share = (p.pieces + 15) / 16, first = wave * share, last = min(first + share, p.pieces);
  int32_t* column = p.counted + min(e, p.E - 1);
  int sum = 0;
#pragma unroll 8
  for (int b = first; b < last; ++b) sum += column[(int64_t)b * p.E];
  sums[wave][lane] = sum;
  __syncthreads();
  if (e >= p.E) return;
  int before = 0;
  for (int w = 0; w < wave; ++w) before += sums[w][lane];
  if (wave == 15) column[(int64_t)p.pieces * p.E] = before + sum;
#pragma unroll 8
  for (int b = first; b < last; ++b) {
    const int count = column[(int64_t)b * p.E];
    column[(int64_t)b * p.E] = before;
    before += count;
  }
}

// Counts the choices before `first` into `before`, the others into `rest` (both zeroed). Eight
// loads of a thread are in flight at once.
template <int THREADS>
__device__ __forceinline__ void count_all(const LayoutParams& p, int first, int32_t* before, int32_t* rest) {
  for (int begin = 0; begin < p.n; begin += 8 * THREADS) {
    int id[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = begin + j * THREADS + threadIdx.x;
      id[j] = i < p.n ? p.ids[i] : -1;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = begin + j * THREADS + threadIdx.x;
      if ((unsigned)id[j] < (unsigned)p.E) atomicAdd(i < first ? &before[id[j]] : &rest[id[j]], 1);
    }
  }
}

// Exclusive prefix sums of value(e), e < E, into out; by all threads, at most 4 experts each of
// the first 256. `waves`: scratch for four.
template <typename F>
__device__ __forceinline__ void prefix(int E, int32_t* out, int32_t* waves, F value) {
  const int each = (E + 255) / 256, begin = threadIdx.x * each, wave = threadIdx.x >> 6;
  int sum = 0, scan = 0;
  if (wave < 4) {
    for (int j = 0; j < each; ++j) sum += begin + j < E ? value(begin + j) : 0;
    scan = wave_scan(sum);
    if ((threadIdx.x & 63) == 63) waves[wave] = scan;
  }
  __syncthreads();
  if (wave < 4) {
    int at = scan - sum;
    for (int w = 0; w < wave; ++w) at += waves[w];
    for (int j = 0; j < each; ++j) {
      if (begin + j >= E) break;
      out[begin + j] = at;
      at += value(begin + j);
    }
  }
  __syncthreads();
}
// The beginning of each expert's segment.
__device__ __forceinline__ void segments(const LayoutParams& p, const int32_t* total, int32_t* start, int32_t* waves, int threads) {
  if (p.max_m == 0) {
    prefix(p.E, start, waves, [&](int e) { return (total[e] + kAlign - 1) / kAlign * kAlign; });
  } else {
    for (int e = threadIdx.x; e < p.E; e += threads) start[e] = e * p.max_m;
    __syncthreads();
  }
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
__device__ __forceinline__ int below(uint64_t lanes, int lane) { return __popcll(lanes & ((1ull << lane) - 1)); }

// Choice c of expert id goes to the rank-th row of its segment, if that is there.
__device__ __forceinline__ int place(const LayoutParams& p, int id, int rank, const int32_t* start) {
  const int64_t row = (int64_t)start[id] + rank;
  return (p.max_m ? rank < p.max_m : row < p.rows) ? (int)row : -1;
}

// Marks the rows that hold no choice, and the experts of the others; `unit` of `units` waves.
__device__ __forceinline__ void mark(const LayoutParams& p, const int32_t* total, const int32_t* start, int unit, int units) {
  const int lane = threadIdx.x & 63;
  if (p.max_m) {
    const int runs = (p.max_m + 63) / 64;
    for (int u = unit; u < p.E * runs; u += units) {
      const int e = u / runs, r = (u - e * runs) * 64 + lane;
      if (r < p.max_m && r >= total[e]) p.sources[(int64_t)e * p.max_m + r] = -1;
    }
    return;
  }
  const int blocks = (int)(p.rows / kAlign);
  for (int b = unit; b < blocks; b += units) {
    // the last expert whose segment begins at or before the block; an empty one shares its place with the next
    int low = 0, high = p.E - 1;
    while (low < high) {
      const int mid = (low + high + 1) / 2;
      if (start[mid] <= b * kAlign) low = mid;
      else high = mid - 1;
    }
    const int64_t end = (int64_t)start[low] + total[low];
#pragma unroll
    for (int i = 0; i < kAlign; i += 64) {
      const int64_t r = (int64_t)b * kAlign + i + lane;
      p.m_indices[r] = r < end ? low : -1;
      if (r >= end) p.sources[r] = -1;
    }
  }
}
__device__ __forceinline__ void write_counts(const LayoutParams& p, const int32_t* total, const int32_t* start, int threads) {
  for (int e = threadIdx.x; e < p.E; e += threads) {
    const int64_t room = p.max_m ? p.max_m : max((int64_t)0, p.rows - start[e]);
    p.counts[e] = (int)min((int64_t)total[e], room);
  }
}

// The layout, a piece a workgroup. LOCAL: every workgroup counts all choices for itself, which
// saves the two launches that count: 32768 choices 8.5 us, where counting by itself takes 4.8 and
// the rest 9.8.
template <bool LOCAL>
__global__ void __launch_bounds__(kPiece) place_kernel(const LayoutParams p) {
  constexpr int kWaves = kPiece / 64;
  __shared__ int32_t total[kMaxExperts], start[kMaxExperts], at[kWaves][kMaxExperts], waves[4];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int c = blockIdx.x * kPiece + threadIdx.x;
  int id = c < p.n ? p.ids[c] : -1;
  if ((unsigned)id >= (unsigned)p.E) id = -1;
  for (int e = threadIdx.x; e < p.E; e += kPiece) {
    total[e] = LOCAL ? 0 : p.counted[(int64_t)p.pieces * p.E + e];
    at[0][e] = LOCAL ? 0 : p.counted[(int64_t)blockIdx.x * p.E + e];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) at[w][e] = 0;
  }
  __syncthreads();
  if constexpr (LOCAL) {
    count_all<kPiece>(p, blockIdx.x * kPiece, at[0], total);
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kPiece) total[e] += at[0][e];
    __syncthreads();
  }
  // a wave's choices count for those after it
  const uint64_t same = equals(id, id >= 0, p.bits);
  if (id >= 0 && wave + 1 < kWaves && below(same, lane) == 0) at[wave + 1][id] = __popcll(same);
  segments(p, total, start, waves, kPiece);  // and its barriers
  for (int e = threadIdx.x; e < p.E; e += kPiece) {
    int sum = at[0][e];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += at[w][e], at[w][e] = sum;
  }
  __syncthreads();
  if (c < p.n) {
    const int row = id >= 0 ? place(p, id, at[wave][id] + below(same, lane), start) : -1;
    p.positions[c] = row;
    if (row >= 0) p.sources[row] = c;
  }
  if (blockIdx.x == 0) write_counts(p, total, start, kPiece);
  mark(p, total, start, blockIdx.x * kWaves + wave, gridDim.x * kWaves);
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

// Rows and scales. LANES lanes read a token's codes (a wave: a slice of them) once and write
// them to each of the token's places. Scales, which lie across the rows, are copied the other
// way: a wave takes 64 neighbouring rows, whose scales it writes as whole lines. Bound by memory,
// mostly by what is written: 4096 tokens of 7168 columns to 8 places each 58 us, 4.7 TB/s (a large
// copy reaches 4.8). Stores with the hint that the lines are not read again are 10% faster, and
// the product that reads them next is slower by more.
template <int LANES>
__global__ void __launch_bounds__(256) gather_kernel(const GatherParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t group = (int64_t)p.first_group + blockIdx.x;
  if (group < p.code_groups) {
    if constexpr (LANES < 64) {
      const int64_t token = group * (256 / LANES) + threadIdx.x / LANES;
      const int column = threadIdx.x % LANES * 16;
      if (token >= p.T || column >= p.K) return;
      const uint4 v = *reinterpret_cast<const uint4*>(p.Q + token * p.ldq + column);
      const int32_t* positions = p.positions + token * p.top_k;
      for (int first = 0; first < p.top_k; first += 4) {  // four choices' rows are looked up at once
        int row[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) row[j] = first + j < p.top_k ? positions[first + j] : -1;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (row[j] >= 0 && row[j] < p.rows) *reinterpret_cast<uint4*>(p.Qx + row[j] * p.ldqx + column) = v;
      }
    } else {
      const int64_t unit = group * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
      const int64_t token = p.slices == 1 ? unit : unit / p.slices;
      if (token >= p.T) return;
      const int column = (int)(unit - token * p.slices) * kSlice + lane * 16;
      const uint8_t* from = p.Q + token * p.ldq;
      v4u v[kSlice / 1024];  // past the row's end its last ones again: branches around the loads cost registers
#pragma unroll
      for (int i = 0; i < kSlice / 1024; ++i) v[i] = *reinterpret_cast<const v4u*>(from + min(column + i * 1024, p.K - 16));
      const int rows = lane < p.top_k ? p.positions[token * p.top_k + lane] : -1;
      for (int j = 0; j < p.top_k; ++j) {
        const int row = __builtin_amdgcn_readlane(rows, j);
        if (row < 0 || row >= p.rows) continue;
        uint8_t* to = p.Qx + row * p.ldqx + column;
#pragma unroll
        for (int i = 0; i < kSlice / 1024; ++i)
          if (column + i * 1024 < p.K) *reinterpret_cast<v4u*>(to + i * 1024) = v[i];
      }
    }
    return;
  }
  const int blocks = p.K >> 7, parts = (blocks + kScaleBlocks - 1) / kScaleBlocks;
  const int64_t unit = (group - p.code_groups) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
  float s[kScaleBlocks];
#pragma unroll
  for (int i = 0; i < kScaleBlocks; ++i)
    if (first + i < blocks) s[i] = from[(first + i) * p.ld_sa];
#pragma unroll
  for (int i = 0; i < kScaleBlocks; ++i)
    if (first + i < blocks) to[(first + i) * p.ld_sax + column] = s[i] * w;
}

// Layout and rows of a few tokens in one launch: a workgroup takes `tokens` of them, at most
// kFewChoices choices, counts all choices for itself, places its own and copies a slice of
// their rows. Here scales are written one by one; there are few. 64 tokens of 8 choices and 7168
// columns 5.4 us: a launch, and a chain of passes over LDS.
struct FewParams {
  LayoutParams layout;
  GatherParams copy;
  int tokens, slices, slice;  // slice: columns, a multiple of 128
};
__global__ void __launch_bounds__(256) dispatch_few_kernel(const FewParams f) {
  __shared__ int32_t total[kMaxExperts], start[kMaxExperts], before[kMaxExperts], waves[4], rows[kFewChoices];
  const LayoutParams& p = f.layout;
  const GatherParams& g = f.copy;
  const int part = blockIdx.x % f.slices, group = blockIdx.x / f.slices;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int first = group * f.tokens * g.top_k, mine = min(f.tokens * g.top_k, p.n - first);
  for (int e = threadIdx.x; e < p.E; e += 256) total[e] = 0, before[e] = 0;
  __syncthreads();
  count_all<256>(p, first, before, total);
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += 256) total[e] += before[e];
  __syncthreads();
  segments(p, total, start, waves, 256);
  if (wave == 0) {
    const int c = first + lane;
    int id = lane < mine ? p.ids[c] : -1;
    if ((unsigned)id >= (unsigned)p.E) id = -1;
    const uint64_t same = equals(id, id >= 0, p.bits);
    const int row = id >= 0 ? place(p, id, before[id] + below(same, lane), start) : -1;
    rows[lane] = row;
    if (part == 0 && lane < mine) {
      p.positions[c] = row;
      if (row >= 0) p.sources[row] = c;
    }
  }
  __syncthreads();
  const int begin = part * f.slice, end = min(begin + f.slice, g.K);
  for (int t = 0; t * g.top_k < mine; ++t) {
    const int64_t token = group * f.tokens + t;
    for (int column = begin + threadIdx.x * 16; column < end; column += 256 * 16) {
      const uint4 v = *reinterpret_cast<const uint4*>(g.Q + token * g.ldq + column);
      for (int j = 0; j < g.top_k; ++j) {
        const int row = rows[t * g.top_k + j];
        if (row >= 0) *reinterpret_cast<uint4*>(g.Qx + row * g.ldqx + column) = v;
      }
    }
    const int blocks = (end - begin) >> 7;
    for (int i = threadIdx.x; i < blocks * g.top_k; i += 256) {
      const int j = i / blocks, kb = (begin >> 7) + i - j * blocks;
      const int row = rows[t * g.top_k + j];
      if (row < 0) continue;
      float s = g.sa[kb * g.ld_sa + token];
      if (g.weights) s *= g.weights[token * g.top_k + j];
      int64_t line = kb, at = row;
      if (p.max_m) {
        const int e = row / p.max_m;
        line += (int64_t)e * (g.K >> 7), at = row - e * p.max_m;
      }
      g.sax[line * g.ld_sax + at] = s;
    }
  }
  if (blockIdx.x == 0) write_counts(p, total, start, 256);
  mark(p, total, start, blockIdx.x * 4 + wave, gridDim.x * 4);
}

}  // namespace fp8moe
