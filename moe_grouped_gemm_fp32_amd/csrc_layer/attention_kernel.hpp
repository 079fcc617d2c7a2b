// Device code of causal attention over the paged 8-bit cache.
//
// One pass over the keys with the running maximum and sum of a softmax, in base 2:
//     m' = max(m, max_j s_j),  l' = l 2^(m - m') + sum_j 2^(s_j - m'),
//     o' = o 2^(m - m') + sum_j 2^(s_j - m') v_j,   s_j = (q . k_j) softmax_scale log2(e)
//
// Rows. The query heads that share a key head, and the tokens of a call, are the rows of
// one product: row r of a sequence is token r / g, head r % g of the group of g. A tile is
// 16 of them, the N side of a 16x16x32 matrix instruction whose M side is keys (first
// product, S^T = K Q^T) or columns of V (second, O^T = V^T P^T). Taken this way round, a
// lane holds logits of one row only, the running statistics of that row live in the same
// lane, and the logits' layout is already the second product's operand: no transposition.
// The order in which the 32 summands of a product are fed is free, so it is chosen for the
// loads: a lane reads 16 consecutive bytes of a key, and D / 16 consecutive bytes of each
// of eight values.
//
// Numbers. e4m3 codes convert exactly to BF16 and FP16; queries stay BF16, so the first
// product's factors are exact. The second product is taken in FP16: probabilities are kept
// relative to a maximum that may lag by 2^kLag, times 2^(15 - kLag), which fills FP16's
// range from above and gives them 11 bits. The value scales (powers of two, one per page)
// enter the probabilities relative to the largest scale so far, which is carried like m.
//
// Work. A unit is a tile, a key head and a chunk of the tile's keys; four waves share it,
// each with its own run of keys. The chunk length follows from the call's total work, found
// on the device, so that ragged batches and single long sequences both fill the GPU. The
// last unit of a tile to arrive joins the parts in their order.
#pragma once

#include "common.hpp"

namespace fp8layer {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kLag = 8;                 // how far (base 2) logits may exceed m before m moves
constexpr float kNone = -1e30f;         // m of a row that has seen no key
constexpr int kCounters = 16384;        // arrival counters at the workspace's start
constexpr int kRowTile = 16;            // rows of a tile
constexpr int kMinChunk = 128;          // least keys of a unit: one step for each wave

struct AttentionParams {
  const uint16_t* q;
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int32_t *block_table, *seq_lens, *cu_q;
  uint16_t* O;
  float* lse;
  int32_t* counters;
  float* parts;
  int64_t ldq, ldo, ld_bt;
  float scale_log2;
  int window, B, T, Hq, Hkv, group, num_pages, log_p, max_pages;
  int units_wanted;  // units that the chunk length aims at; 0: no splitting
};

// What a sequence asks for: its row tiles, and the most keys that one of them reads.
struct Demand {
  int tiles, keys;
};
template <int TILE, int STEP>
__device__ __forceinline__ Demand demand(const Sequence& s, const AttentionParams& p) {
  const int tiles = (s.rows * p.group + TILE - 1) / TILE;
  // a window's start is rounded down to a step
  const int64_t most = p.window ? min((int64_t)s.len, (int64_t)p.window + s.rows + STEP - 2) : (int64_t)s.len;
  return {tiles, (int)most};
}

// A unit of work, found by scanning the sequences' unit counts (every wave does it for
// itself). Everything is wave-uniform.
struct Unit {
  Sequence seq;
  int b, h, tile, tiles;
  int slot;          // number of the unit: its place among the parts
  int tile_id;       // number of the tile and head: its counter
  int chunk;         // this unit's chunk
  int chunks;        // chunks of the tile
  int row0, rows;    // the tile's rows within the sequence
  int pos0, pos1;    // positions of the tile's first and last token
  int lo, hi;        // keys that some row of the tile sees, lo rounded down to a step
  int k0, k1;        // this unit's keys
};
template <int TILE, int STEP>
__device__ __forceinline__ bool find_unit(const AttentionParams& p, int number, int min_chunk, Unit& u) {
  const int lane = threadIdx.x & 63;
  const int max_len = p.max_pages << p.log_p;
  int chunk_len = INT32_MAX;
  if (p.units_wanted > 0) {
    int64_t work = 0;  // keys over all tiles and heads
    for (int base = 0; base < p.B; base += 64) {
      int64_t mine = 0;
      if (base + lane < p.B) {
        const Demand d = demand<TILE, STEP>(sequence(p.cu_q, p.seq_lens, base + lane, p.T, max_len), p);
        mine = (int64_t)d.tiles * d.keys;
      }
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) mine += __shfl_xor((long long)mine, o, 64);
      work += mine;
    }
    const int64_t each = (work * p.Hkv + p.units_wanted - 1) / p.units_wanted;
    chunk_len = (int)min((int64_t)(1 << 30), max((int64_t)min_chunk, (each + 127) / 128 * 128));
  }
  u.slot = number;
  u.h = number % p.Hkv;
  const int want = number / p.Hkv;
  int before = 0, tiles_before = 0;
  for (int base = 0; base < p.B; base += 64) {
    Sequence s{};
    Demand d{};
    int count = 0;
    if (base + lane < p.B) {
      s = sequence(p.cu_q, p.seq_lens, base + lane, p.T, max_len);
      d = demand<TILE, STEP>(s, p);
      count = d.tiles * max(1, (int)(((int64_t)d.keys + chunk_len - 1) / chunk_len));
    }
    const int incl = wave_scan(count, lane);
    const int tiles_incl = wave_scan(d.tiles, lane);
    const uint64_t hit = __ballot(want < before + incl);
    if (hit) {
      const int src = __ffsll((unsigned long long)hit) - 1;
      auto pick = [&](int v) { return __builtin_amdgcn_readlane(v, src); };
      u.b = base + src;
      u.seq = {pick(s.row0), pick(s.rows), pick(s.len)};
      u.tiles = pick(d.tiles);
      const int within = want - (before + pick(incl - count));
      u.chunk = within / u.tiles;
      u.tile = u.tiles - 1 - within % u.tiles;  // the tiles with the most keys first
      u.tile_id = (tiles_before + pick(tiles_incl - d.tiles) + u.tile) * p.Hkv + u.h;
      const int total = u.seq.rows * p.group;
      u.row0 = u.tile * TILE;
      u.rows = min(TILE, total - u.row0);
      const int first = u.seq.len - u.seq.rows;
      u.pos0 = first + u.row0 / p.group;
      u.pos1 = first + (u.row0 + u.rows - 1) / p.group;
      u.lo = p.window ? max(0, u.pos0 - p.window + 1) / STEP * STEP : 0;
      u.hi = max(u.lo, min(u.seq.len, u.pos1 + 1));
      u.chunks = max(1, (int)(((int64_t)(u.hi - u.lo) + chunk_len - 1) / chunk_len));
      if (u.chunk >= u.chunks) return false;  // a tile that sees fewer keys than the sequence's last
      u.k0 = (int)min((int64_t)u.hi, u.lo + (int64_t)u.chunk * chunk_len);
      u.k1 = (int)min((int64_t)u.hi, u.k0 + (int64_t)chunk_len);
      return true;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
    tiles_before += __builtin_amdgcn_readlane(tiles_incl, 63);
  }
  return false;  // the grid covers the most units that there can be
}

// The raw bytes of 32 keys and values that a lane feeds: keys kg of the 16-key groups'
// rows `lane & 15`, and eight values (kg = lane >> 4).
template <int D>
struct Raw {
  uint4 k[2][D / 64];
  uint32_t v[8][D / 64];
};

template <int D>
__device__ __forceinline__ void load_value(uint32_t (&dst)[D / 64], const uint8_t* src) {
  if constexpr (D == 64) {
    dst[0] = *reinterpret_cast<const uint32_t*>(src);
  } else if constexpr (D == 128) {
    const uint2 x = *reinterpret_cast<const uint2*>(src);
    dst[0] = x.x, dst[1] = x.y;
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(src);
    dst[0] = x.x, dst[1] = x.y, dst[2] = x.z, dst[3] = x.w;
  }
}

// base0, base1: token slots (over pages and heads) of the two 16-key groups.
template <int D>
__device__ __forceinline__ void load_raw(Raw<D>& r, const AttentionParams& p, int64_t base0, int64_t base1, int lane) {
  const int n = lane & 15, kg = lane >> 4;
  const uint8_t* k0 = p.k_cache + base0 * D + n * D + kg * 16;
  const uint8_t* k1 = p.k_cache + base1 * D + n * D + kg * 16;
  const uint8_t* v0 = p.v_cache + base0 * D + kg * 4 * D + n * (D / 16);
  const uint8_t* v1 = p.v_cache + base1 * D + kg * 4 * D + n * (D / 16);
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    r.k[0][i] = *reinterpret_cast<const uint4*>(k0 + i * 64);
    r.k[1][i] = *reinterpret_cast<const uint4*>(k1 + i * 64);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    load_value<D>(r.v[j], v0 + j * D);
    load_value<D>(r.v[4 + j], v1 + j * D);
  }
}

// Eight codes to BF16, exactly.
__device__ __forceinline__ v8bf codes_bf16(uint32_t a, uint32_t b) {
  const v2bf x0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
  const v2bf x1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
  const v2bf x2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
  const v2bf x3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
  return v8bf{x0.x, x0.y, x1.x, x1.y, x2.x, x2.y, x3.x, x3.y};
}

// Byte e (0 .. 3) of eight words to FP16, exactly, for e and e + 1 (e even).
__device__ __forceinline__ void columns_f16(const uint32_t (&w)[8], bool upper, v8h& even, v8h& odd) {
  const uint32_t sel = upper ? 0x07030602u : 0x05010400u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t x = __builtin_amdgcn_perm(w[2 * j + 1], w[2 * j], sel);
    const v2h lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, 1.0f, false);
    const v2h hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, 1.0f, true);
    even[2 * j] = lo.x, even[2 * j + 1] = lo.y;
    odd[2 * j] = hi.x, odd[2 * j + 1] = hi.y;
  }
}

// Exponent field of a power of two.
__device__ __forceinline__ int exponent(float x) { return (int)((__float_as_uint(x) >> 23) & 0xFF); }
// 2^e; 0 where that is below the normal range, infinity above.
__device__ __forceinline__ float pow2(int e) {
  return e < -126 ? 0.f : e > 127 ? INFINITY : __uint_as_float((uint32_t)(e + 127) << 23);
}
// 2^x for a difference of two maxima: 0 for minus infinity.
__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ bool any_nan_code(uint32_t w) { return (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0; }

// Partial results travel between workgroups (of any XCD) as device-coherent accesses.
constexpr int kDeviceScope = 16;        // buffer cache policy sc1
constexpr int kRawDword3 = 0x00020000;  // buffer descriptor: 32-bit untyped

template <int D>
__global__ void __launch_bounds__(256) attention_kernel(const AttentionParams p) {
  constexpr int kWords = D / 64;       // 32-bit words of one value a lane feeds
  constexpr int kTiles = D / 16;       // 16-column tiles of V
  constexpr int kStride = D + 4;       // of a row of O in LDS
  constexpr int kSlotFloats = kRowTile * (D + 1);
  __shared__ float o_sh[4][kRowTile][kStride];
  __shared__ float m_sh[4][kRowTile], l_sh[4][kRowTile];
  __shared__ int e_sh[4], last_sh;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, kg = lane >> 4;
  Unit u;
  if (!find_unit<kRowTile, 32>(p, blockIdx.x, kMinChunk, u)) return;

  // this lane's row: query fragments, and the keys that it sees, [key_lo, key_hi)
  const bool live = n < u.rows;
  const int row = u.row0 + (live ? n : 0);
  const int token = row / p.group, head = u.h * p.group + row % p.group;
  const int pos = u.seq.len - u.seq.rows + token;
  const int key_hi = min(u.seq.len, pos + 1);
  const int key_lo = p.window ? max(0, pos - p.window + 1) : 0;
  v8bf qf[D / 32];
  {
    const uint16_t* src = p.q + (int64_t)(u.seq.row0 + token) * p.ldq + head * D;
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (live) x = *reinterpret_cast<const uint4*>(src + (s >> 1) * 64 + kg * 16 + (s & 1) * 8);
      qf[s] = __builtin_bit_cast(v8bf, x);
    }
  }
  // keys that every row of the tile sees
  const int all_hi = min(u.seq.len, u.pos0 + 1), all_lo = p.window ? u.pos1 - p.window + 1 : 0;

  v4f o[kTiles];
#pragma unroll
  for (int t = 0; t < kTiles; ++t) o[t] = v4f{0.f, 0.f, 0.f, 0.f};
  float m = kNone, l = 0.f;
  int ev = 0;  // exponent field of the largest value scale so far

  const int steps = (u.k1 - u.k0 + 31) >> 5, share = (steps + 3) >> 2;
  const int step0 = min(steps, wave * share), step1 = min(steps, step0 + share);
  for (int seg = step0; seg < step1; seg += 32) {
    // lane i holds what group i (16 keys) of the next 64 needs: its page and scales
    int page = -1;
    float ks = 0.f, vs = 0.f;
    {
      const int key = u.k0 + seg * 32 + lane * 16;
      if (key < u.k1) {
        page = p.block_table[u.b * p.ld_bt + (key >> p.log_p)];
        if (page >= 0 && page < p.num_pages) {
          ks = p.k_scale[(int64_t)page * p.Hkv + u.h] * p.scale_log2;
          vs = p.v_scale[(int64_t)page * p.Hkv + u.h];
        } else {
          page = -1;
        }
      }
    }
    const int count = min(32, step1 - seg);
    auto fetch = [&](int s, Raw<D>& r) {
      const int key = u.k0 + (seg + s) * 32;
      const int p0 = __builtin_amdgcn_readlane(page, 2 * s), p1 = __builtin_amdgcn_readlane(page, 2 * s + 1);
      const int mask = (1 << p.log_p) - 1;
      const int64_t b0 = (((int64_t)max(p0, 0) * p.Hkv + u.h) << p.log_p) + (key & mask);
      const int64_t b1 = (((int64_t)max(p1, 0) * p.Hkv + u.h) << p.log_p) + ((key + 16) & mask);
      load_raw<D>(r, p, b0, b1, lane);
    };
    Raw<D> next;
    fetch(0, next);
    for (int s = 0; s < count; ++s) {
      Raw<D> r = next;
      if (s + 1 < count) fetch(s + 1, next);
      const int key = u.k0 + (seg + s) * 32;
      const int pg0 = __builtin_amdgcn_readlane(page, 2 * s), pg1 = __builtin_amdgcn_readlane(page, 2 * s + 1);
      const float c0 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ks), 2 * s));
      const float c1 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ks), 2 * s + 1));
      const int e0 = exponent(__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(vs), 2 * s)));
      const int e1 = exponent(__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(vs), 2 * s + 1)));

      v4f s0{0.f, 0.f, 0.f, 0.f}, s1{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        s0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16(r.k[0][i].x, r.k[0][i].y), qf[2 * i], s0, 0, 0, 0);
        s1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16(r.k[1][i].x, r.k[1][i].y), qf[2 * i], s1, 0, 0, 0);
        s0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16(r.k[0][i].z, r.k[0][i].w), qf[2 * i + 1], s0, 0, 0, 0);
        s1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16(r.k[1][i].z, r.k[1][i].w), qf[2 * i + 1], s1, 0, 0, 0);
      }
      float x[8];  // this lane's keys: key + 4 kg + j, and 16 further for j >= 4
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = s0[j] * c0, x[4 + j] = s1[j] * c1;
      uint32_t nan_keys = 0;
      if (key < all_lo || key + 32 > all_hi || pg0 < 0 || pg1 < 0) {  // some row does not see all of the step
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int at = key + (j >> 2) * 16 + kg * 4 + (j & 3);
          const bool there = (j < 4 ? pg0 : pg1) >= 0;
          if (!there || at < key_lo || at >= key_hi) x[j] = -INFINITY;
          // values that no row sees may be anything: they count as 0. Where a row sees a
          // NaN code and another does not, the product gets 0 and the rows that see it NaN
          // by their probability.
          if (!there || at < u.lo || at >= u.hi) {
#pragma unroll
            for (int w = 0; w < kWords; ++w) r.v[j][w] = 0;
          } else {
            bool bad = false;
#pragma unroll
            for (int w = 0; w < kWords; ++w) bad |= any_nan_code(r.v[j][w]);
            if (bad) {
              nan_keys |= 1u << j;
#pragma unroll
              for (int w = 0; w < kWords; ++w) r.v[j][w] = 0;
            }
          }
        }
        if (__any(nan_keys != 0)) {  // over the 16 lanes that feed the same keys
#pragma unroll
          for (int off = 1; off < 16; off <<= 1) nan_keys |= __shfl_xor((int)nan_keys, off, 64);
        }
      }
      float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
      if (__any(top > m + kLag) || max(e0, e1) > ev) {  // rare after a row's first steps
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float now = fmaxf(m, top);
        const int e_now = max(ev, max(e0, e1));
        const float a = exp2_of(m - now), b = a * pow2(ev - e_now);
        m = now, ev = e_now;
        l *= a;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) o[t] *= b;
      }
      const float f0 = pow2(15 - kLag + e0 - ev), f1 = pow2(15 - kLag + e1 - ev);
      v8h pf;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float pr = exp2_of(x[j] - m);
        l += pr;
        float w = pr * (j < 4 ? f0 : f1);
        if ((nan_keys >> j & 1) && x[j] > -INFINITY) w = __builtin_nanf("");
        pf[j] = (_Float16)w;
      }
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        uint32_t words[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) words[j] = r.v[j][w];
        v8h a, b;
        columns_f16(words, false, a, b);
        o[4 * w] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pf, o[4 * w], 0, 0, 0);
        o[4 * w + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, pf, o[4 * w + 1], 0, 0, 0);
        columns_f16(words, true, a, b);
        o[4 * w + 2] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pf, o[4 * w + 2], 0, 0, 0);
        o[4 * w + 3] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, pf, o[4 * w + 3], 0, 0, 0);
      }
    }
  }

  // join the four waves: row n's column (4 kg + i) (D / 16) + t is o[t][i]
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int t = 0; t < kTiles; t += 4)
      *reinterpret_cast<float4*>(&o_sh[wave][n][(4 * kg + i) * kTiles + t]) =
          make_float4(o[t][i], o[t + 1][i], o[t + 2][i], o[t + 3][i]);
  if (kg == 0) m_sh[wave][n] = m, l_sh[wave][n] = l;
  if (lane == 0) e_sh[wave] = ev;
  __syncthreads();

  // thread (r, x): row r, columns x D / 16 .. + D / 16
  const int r = threadIdx.x >> 4, x = threadIdx.x & 15;
  float top = kNone, sum = 0.f, out[kTiles];
#pragma unroll
  for (int w = 0; w < 4; ++w) top = fmaxf(top, m_sh[w][r]);
#pragma unroll
  for (int t = 0; t < kTiles; ++t) out[t] = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float a = exp2_of(m_sh[w][r] - top);
    sum += a * l_sh[w][r];
    // a wave's sums stand for themselves times 2^(its value exponent) / 2^(15 - kLag)
    const int e = e_sh[w] - 127 - (15 - kLag);
    const float b = a * pow2(e / 2), c = pow2(e - e / 2);  // in two steps: each in range
#pragma unroll
    for (int t = 0; t < kTiles; t += 4) {
      const float4 y = *reinterpret_cast<const float4*>(&o_sh[w][r][x * kTiles + t]);
      out[t] += y.x * b * c, out[t + 1] += y.y * b * c, out[t + 2] += y.z * b * c, out[t + 3] += y.w * b * c;
    }
  }
  // a row that saw no key: 0, and minus infinity
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
  for (int t = 0; t < kTiles; ++t) out[t] *= inv;
  float lse2 = sum == 0.f ? -INFINITY : top + __log2f(sum);

  if (u.chunks > 1) {
    const int slot_bytes = kSlotFloats * 4;
    const int stride = u.tiles * p.Hkv;  // slots between chunks of a tile
    const int first = u.slot - u.chunk * stride;
    float* base = p.parts + (int64_t)first * kSlotFloats;
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc(base, 0, ((u.chunks - 1) * stride + 1) * slot_bytes, kRawDword3);
    const int at = r * D * 4 + x * kTiles * 4, lse_at = (kRowTile * D + r) * 4;
    if (r < u.rows) {
#pragma unroll
      for (int t = 0; t < kTiles; t += 4)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, v4f{out[t], out[t + 1], out[t + 2], out[t + 3]}),
                                               rs, u.chunk * stride * slot_bytes + at + t * 4, 0, kDeviceScope);
      if (x == 0)
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(lse2), rs, u.chunk * stride * slot_bytes + lse_at, 0,
                                              kDeviceScope);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the part has reached the device-coherent level
    __syncthreads();
    if (threadIdx.x == 0)
      last_sh = __hip_atomic_fetch_add(&p.counters[u.tile_id], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                u.chunks - 1;
    __syncthreads();
    if (!last_sh) return;
    if (threadIdx.x == 0) __hip_atomic_store(&p.counters[u.tile_id], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (r < u.rows) {
      float most = -INFINITY;
      for (int c = 0; c < u.chunks; ++c)
        most = fmaxf(most, __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, c * stride * slot_bytes + lse_at, 0,
                                                                                kDeviceScope)));
      if (!(most > -INFINITY)) most = 0.f;
      sum = 0.f;
#pragma unroll
      for (int t = 0; t < kTiles; ++t) out[t] = 0.f;
      for (int c = 0; c < u.chunks; ++c) {
        const int off = c * stride * slot_bytes;
        const float part = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, off + lse_at, 0, kDeviceScope));
        const float a = exp2_of(part - most);
        sum += a;
#pragma unroll
        for (int t = 0; t < kTiles; t += 4) {
          const v4f y = __builtin_bit_cast(
              v4f, __builtin_amdgcn_raw_buffer_load_b128(rs, off + at + t * 4, 0, kDeviceScope));
          out[t] += a * y.x, out[t + 1] += a * y.y, out[t + 2] += a * y.z, out[t + 3] += a * y.w;
        }
      }
      const float scale = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
      for (int t = 0; t < kTiles; ++t) out[t] *= scale;
      lse2 = sum == 0.f ? -INFINITY : most + __log2f(sum);
    }
  }
  if (r < u.rows) {
    const int rr = u.row0 + r;
    const int64_t tok = u.seq.row0 + rr / p.group;
    const int hd = u.h * p.group + rr % p.group;
    uint16_t* dst = p.O + tok * p.ldo + hd * D + x * kTiles;
#pragma unroll
    for (int t = 0; t < kTiles; t += 4)
      *reinterpret_cast<uint2*>(dst + t) = make_uint2(pack_bf16(out[t], out[t + 1]), pack_bf16(out[t + 2], out[t + 3]));
    if (p.lse && x == 0) p.lse[tok * p.Hq + hd] = lse2 * 0.6931471805599453f;
  }
}

}  // namespace fp8layer
