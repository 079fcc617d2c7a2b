// Device code of the append to the paged 8-bit cache, with the rotation on the way.
//
// Work is divided by what shares a scale: one unit is one page, one head, keys or values,
// shared by WAVES waves. The largest magnitude of its new tokens settles the page's scale,
// then they are encoded: a thread holds its first kHeld groups of columns in between (a
// whole page up to 8192 columns over four waves, or 2048 over one) and reads further ones
// again. So a page's scale and codes have one writer, and the result does not depend on
// any order. The queries' rotation, which no unit waits for, fills further workgroups of
// the same launch.
//
// Bound by memory where tokens are many (8636 tokens of 6 prompts, 32 + 2 x 8 heads of 128,
// pages of 16: 45.1 us, 4.4 TB/s), by the chain of sequences, page, tokens, maximum and codes
// where they are few (64 users, one token each: 4.5 us). Fewer registers a wave, for more
// waves on a CU, spilled: 54 to 75 us instead of 48.
//
// A thread handles two groups of eight columns at a time: of a rotated head, the first
// and second members of eight pairs; of other columns, 16 in a row.
#pragma once

#include "common.hpp"

namespace fp8layer {

struct AppendParams {
  const uint16_t *q, *k, *v;
  const float* cos_sin;
  const int32_t *positions, *block_table, *seq_lens, *cu_q;
  uint16_t* q_out;
  uint8_t *k_cache, *v_cache;
  float *k_scale, *v_scale;
  int64_t ldq, ldk, ldv, ld_cs, ld_bt, ldqo;
  int max_pos, rot_dim, interleaved, max_pages, num_pages, log_p;
  int B, T, Hq, Hkv;
  int unit_groups;   // workgroups that hold units; the later ones rotate queries,
  int group_tokens;  // of so many tokens each
  int first_group;   // the launch's first workgroup of the call's
};

constexpr int kHeld = 2;

// Bits of the smallest power of two, 2^-126 at least, by which amax fits 448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t fit_scale_bits(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(e, 1) << 23;
}

// The two column groups of item i of a head: their first columns, and whether they turn.
struct Item {
  int lo, hi;
  bool turns;
};
__device__ __forceinline__ Item item_of(int i, int rot_dim, int interleaved) {
  const bool turns = 16 * i < rot_dim;
  const bool halves = turns && !interleaved;
  return {halves ? 8 * i : 16 * i, halves ? (rot_dim >> 1) + 8 * i : 16 * i + 8, turns};
}

// Turns the item's 16 columns by cos/sin of pairs 8 i .. 8 i + 7 of the row `cs`. Every
// product and sum is rounded by itself.
__device__ __forceinline__ void turn_item(const Eight<uint16_t>& lo, const Eight<uint16_t>& hi, const float* cs, const Item& it, int i,
                                          int rot_dim, int interleaved, float (&a)[8], float (&b)[8]) {
#pragma clang fp contract(off)
  lo.get(a);
  hi.get(b);
  if (it.turns) {
    float c[8], s[8];
    load8(cs + 8 * i, c);
    load8(cs + (rot_dim >> 1) + 8 * i, s);
    if (interleaved) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a1 = a[2 * j], a2 = a[2 * j + 1], b1 = b[2 * j], b2 = b[2 * j + 1];
        a[2 * j] = a1 * c[j] - a2 * s[j];
        a[2 * j + 1] = a2 * c[j] + a1 * s[j];
        b[2 * j] = b1 * c[4 + j] - b2 * s[4 + j];
        b[2 * j + 1] = b2 * c[4 + j] + b1 * s[4 + j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x1 = a[j], x2 = b[j];
        a[j] = x1 * c[j] - x2 * s[j];
        b[j] = x2 * c[j] + x1 * s[j];
      }
    }
  }
}

__device__ __forceinline__ void encode(float (&x)[8], float inv) {
  // infinities become NaN here, so that both are stored as the NaN code
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = fabsf(x[j]) < INFINITY ? x[j] * inv : __builtin_nanf("");
}

template <int D, int WAVES, bool STREAM>
__global__ void __launch_bounds__(256) rope_append_kernel(const AppendParams p) {
  constexpr int kItems = D / 16;               // items of one head
  constexpr int kThreads = WAVES * 64;         // threads of a unit
  constexpr int kTokens = kThreads / kItems;   // tokens handled at a time
  __shared__ float part[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int P = 1 << p.log_p;
  const int max_len = p.max_pages << p.log_p;
  const int group = p.first_group + (int)blockIdx.x;

  if (group >= p.unit_groups) {  // queries: a thread has item n % kItems of every so many heads
    const int t0 = (group - p.unit_groups) * p.group_tokens, t1 = min(p.T, t0 + p.group_tokens);
    for (int n0 = 0; n0 < p.Hq * kItems; n0 += 256) {
      const int n = n0 + threadIdx.x, i = n % kItems, h = n / kItems;
      const bool live = n < p.Hq * kItems;
      const Item it = item_of(i, p.rot_dim, p.interleaved);
      Eight<uint16_t> lo, hi;  // of the next token
      auto fetch = [&](int t) {
        if (live && t < t1) {
          const uint16_t* src = p.q + t * p.ldq + h * D;
          lo.template load<STREAM>(src + it.lo), hi.template load<STREAM>(src + it.hi);
        }
      };
      fetch(t0);
      Sequence sq{};
      for (int t = t0; t < t1; ++t) {
        if (t == t0 || t >= sq.row0 + sq.rows) {  // the token's sequence: the last with cu_q[b] <= t
          int b = -1;
          for (int base = 0; base < p.B; base += 64) {
            const int before = __popcll(__ballot(base + lane < p.B && p.cu_q[min(base + lane, p.B - 1)] <= t));
            b += before;
            if (before < 64) break;
          }
          sq = sequence(p.cu_q, p.seq_lens, max(b, 0), p.T, max_len);
          if (t >= sq.row0 + sq.rows) break;  // past the last sequence
        }
        const int at = p.positions ? p.positions[t] : sq.start + (t - sq.row0);
        const float* cs = p.cos_sin + min(max(at, 0), p.max_pos - 1) * p.ld_cs;
        const Eight<uint16_t> lo0 = lo, hi0 = hi;
        fetch(t + 1);
        if (live) {
          float a[8], c[8];
          turn_item(lo0, hi0, cs, it, i, p.rot_dim, p.interleaved, a, c);
          uint16_t* dst = p.q_out + t * p.ldqo + h * D;
          store8(dst + it.lo, a);
          store8(dst + it.hi, c);
        }
      }
    }
    return;
  }

  // the unit: a page of a sequence (found by scanning the sequences' page counts), a head,
  // keys or values
  const int unit = WAVES == 4 ? group : group * 4 + wave;
  const bool keys = (unit & 1) == 0;
  const int h = (unit >> 1) % p.Hkv;
  const int want = (unit >> 1) / p.Hkv;
  Sequence sq{};
  int first_page = 0, done = 0;
  bool found = false;
  for (int base = 0; base < p.B && !found; base += 64) {
    Sequence mine{};
    int count = 0, page0 = 0;
    if (base + lane < p.B) {
      mine = sequence(p.cu_q, p.seq_lens, base + lane, p.T, max_len);
      page0 = max(mine.start, 0) >> p.log_p;
      if (mine.rows > 0 && mine.start < mine.len) count = ((mine.len - 1) >> p.log_p) - page0 + 1;
    }
    const int incl = wave_scan(count);
    const uint64_t hit = __ballot(want < done + incl);
    if (hit) {
      const int src = __ffsll((unsigned long long)hit) - 1;
      auto pick = [&](int v) { return __builtin_amdgcn_readlane(v, src); };
      sq = {pick(mine.row0), pick(mine.rows), pick(mine.start), pick(mine.len)};
      const int within = want - (done + pick(incl - count));
      if ((uint32_t)within >= (uint32_t)pick(count)) return;  // only where overlapping rows overflow the sums
      first_page = pick(page0) + within;
      done = base + src;  // the sequence, from here on
      found = true;
    } else {
      done += last_lane(incl);
    }
  }
  if (!found) return;  // the grid covers the most units that there can be (all waves of a shared unit agree)
  const int page = p.block_table[done * p.ld_bt + first_page];
  if (page < 0 || page >= p.num_pages) return;
  const int slot0 = first_page << p.log_p;
  const int from = max(sq.start - slot0, 0);        // earlier tokens of this page: [0, from)
  const int to = min(sq.len - slot0, P);            // new ones: [from, to)
  const int row_at = sq.row0 - sq.start + slot0;       // row of slot 0 of the page
  const uint16_t* src = keys ? p.k : p.v;
  const int64_t ld = keys ? p.ldk : p.ldv;
  const int64_t head = (int64_t)page * p.Hkv + h;
  uint8_t* codes = (keys ? p.k_cache : p.v_cache) + (head << p.log_p) * D;
  float* scale = (keys ? p.k_scale : p.v_scale) + head;
  const int rot = keys ? p.rot_dim : 0;
  const int t = WAVES == 4 ? threadIdx.x : lane;
  const int i = t % kItems;
  const Item it = item_of(i, rot, p.interleaved);
  const uint32_t before = from > 0 ? __float_as_uint(*scale) & 0x7F800000u : 0u;

  auto fetch = [&](int s, float(&a)[8], float(&b)[8]) {
    const int row = row_at + s;
    const int at = p.positions ? p.positions[row] : slot0 + s;
    const int pos = min(max(at, 0), p.max_pos - 1);
    Eight<uint16_t> lo, hi;
    lo.template load<STREAM>(src + row * ld + h * D + it.lo), hi.template load<STREAM>(src + row * ld + h * D + it.hi);
    turn_item(lo, hi, p.cos_sin + pos * p.ld_cs, it, i, rot, p.interleaved, a, b);
  };

  float held_a[kHeld][8], held_b[kHeld][8];
  float amax = 0.f;
  auto measure = [&](const float(&a)[8], const float(&b)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = fabsf(a[j]), y = fabsf(b[j]);
      amax = fmaxf(amax, x < INFINITY ? x : 0.f);
      amax = fmaxf(amax, y < INFINITY ? y : 0.f);
    }
  };
  const int s0 = from + t / kItems;
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (s0 + k * kTokens < to) {
      fetch(s0 + k * kTokens, held_a[k], held_b[k]);
      measure(held_a[k], held_b[k]);
    }
  for (int s = s0 + kHeld * kTokens; s < to; s += kTokens) {
    float a[8], b[8];
    fetch(s, a, b);
    measure(a, b);
  }
  amax = wave_max(amax);
  if constexpr (WAVES == 4) {
    if (lane == 0) part[wave] = amax;
    __syncthreads();  // also: every thread has read the old scale
    amax = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  }
  const uint32_t now = max(fit_scale_bits(amax), before);
  if (t == 0) *scale = __uint_as_float(now);
  // 1 / scale: exponents mirrored around 127; 2^127 (a scale that no append makes) has the
  // subnormal 2^-127
  const float inv = now == 0x7F000000u ? 0x1p-127f : __uint_as_float(0x7F000000u - now);

  if (from > 0 && now > before) {  // the earlier codes, at the larger scale
    const float ratio = __uint_as_float(before) * inv;
    for (int s = t / kItems; s < from; s += kTokens) {
      uint4* at = reinterpret_cast<uint4*>(codes + s * D + 16 * i);
      const uint4 old = *at;
      const uint32_t w[4] = {old.x, old.y, old.z, old.w};
      float a[8], b[8];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const v2f a0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], false), a1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], true);
        const v2f b0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[2 + j], false),
                  b1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[2 + j], true);
        a[4 * j] = a0.x * ratio, a[4 * j + 1] = a0.y * ratio, a[4 * j + 2] = a1.x * ratio, a[4 * j + 3] = a1.y * ratio;
        b[4 * j] = b0.x * ratio, b[4 * j + 1] = b0.y * ratio, b[4 * j + 2] = b1.x * ratio, b[4 * j + 3] = b1.y * ratio;
      }
      const uint2 lo = pack_e4m3(a), hi = pack_e4m3(b);
      *at = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
  }
  auto put = [&](int s, float(&a)[8], float(&b)[8]) {
    encode(a, inv);
    encode(b, inv);
    *reinterpret_cast<uint2*>(codes + s * D + it.lo) = pack_e4m3(a);
    *reinterpret_cast<uint2*>(codes + s * D + it.hi) = pack_e4m3(b);
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (s0 + k * kTokens < to) put(s0 + k * kTokens, held_a[k], held_b[k]);
  for (int s = s0 + kHeld * kTokens; s < to; s += kTokens) {
    float a[8], b[8];
    fetch(s, a, b);
    put(s, a, b);
  }
}

}  // namespace fp8layer
