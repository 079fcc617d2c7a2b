// Device code of causal attention over the paged 8-bit cache.
//
// One pass over the keys with the running maximum and sum of a softmax, in base 2:
//     m' = max(m, max_j s_j),  l' = l 2^(m - m') + sum_j 2^(s_j - m'),
//     o' = o 2^(m - m') + sum_j 2^(s_j - m') v_j,   s_j = (q . k_j) softmax_scale log2(e)
//
// Rows. The query heads that share a key head, and the tokens of a call, are the rows of
// one product: row r of a sequence is token r / g, head r % g of the group of g. 16 of them
// are the N side of a 16x16x32 matrix instruction whose M side is keys (first product,
// S^T = K Q^T) or columns of V (second, O^T = V^T P^T). Taken this way round, a lane holds
// logits of one row only, the running statistics of that row live in the same lane, and
// the logits' layout is already the second product's operand: no transposition. A tile is
// R times 16 rows, which share each key and value that is read and converted.
// The order in which the 32 summands of a product are fed is free, so it is chosen for the
// loads: a lane feeds 16 consecutive bytes of a key, and D / 16 consecutive bytes of each
// of eight values.
//
// Loads. Each wave streams its own keys and values into a ring of two 32-key stages in LDS,
// by loads that go there without passing registers, and refills the key half and the value
// half of a stage as soon as it has read them: three quarters of the ring are in flight at
// any time, without a barrier.
//
// Numbers. e4m3 codes convert exactly to BF16 and FP16; queries stay BF16, so the first
// product's factors are exact. The second product is taken in FP16, whose 11 bits a
// probability needs more than range. The value scales (powers of two, one per page) enter
// by the exponent, w_j = 2^(s_j + log2 vscale_j - mo + 15 - kLag), relative to a maximum mo
// of their own, so that whatever contributes most to o lies at the top of FP16's range;
// l is summed from the same w, each 16-key group by its factor 2^(.. - m). Both maxima may
// lag behind by 2^kLag before o and l are rescaled, which is rare after the first steps.
//
// Work. A unit is a tile, a key head and a chunk of the tile's keys; four waves share it,
// each with its own run of keys. The chunk length follows from the call's total work,
// found on the device (Plan), so that ragged batches and single long sequences both fill
// the GPU. The parts of a tile are joined in their order by whoever arrives last: first in
// groups of kJoin neighbours, then the groups' results.
//
// What bounds it. Many rows: vector instructions (64 codes converted a lane and step, eight
// exponentials a row block: 195 of them and 48 matrix instructions a step of 48 rows) that
// hardly overlap with the matrix unit: it works in 37 % of the cycles and they issue in 60 %,
// as a wave's steps depend on each other and registers allow two waves a SIMD (2 x 2048 prompt
// tokens over 8192 keys 524 us, 918 TFLOP/s of the 1280 that a large BF16 product reaches). Few rows, many keys: memory (64 x 8192 keys 165 us, 6.5 TB/s;
// 64 users of 500 to 8192 keys 112 us, 5.4 TB/s). Little work: latencies, in us for one user
// of 777 keys 1.4 to find the unit, 1.2 to the first keys, 0.8 a step, 0.9 to join the waves,
// 1.1 to hand over to the last arriver, 0.4 and 1.0 to join the parts and write: 8.1 in all.
#pragma once

#include "common.hpp"

namespace fp8layer {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr float kLag = 8.f;             // how far (base 2) logits may exceed m before m moves
constexpr float kNone = -1e30f;         // m of a row that has seen no key
constexpr int kTileCounters = 8192;     // arrival counters at the workspace's start: of tiles,
constexpr int kPartCounters = 8192;     // and of groups of parts
constexpr int kCounters = kTileCounters + kPartCounters;
constexpr int kMinChunk = 128;          // least keys of a unit: one step for each wave
constexpr int kMostKeys = 1 << 30;      // most keys of a sequence: key numbers a segment further fit 32 bits,
constexpr int kWhole = kMostKeys;       // and a chunk of so many leaves every tile whole
constexpr int kJoin = 8;                // parts joined at a time, all loads in flight together
// Where a page's values are so small that even the likeliest key adds less than 2^-60 of
// what o holds, w keeps this much below the likeliest key's 2^0 instead, for l's sake.
constexpr float kFar = -60.f;

// Division of numbers below 2^31 by a divisor known on the host: n m / 2^s with m the
// quotient 2^s / d rounded up, s = 31 + ceil(log2 d), so that n times m's error is below 2^s.
struct Divisor {
  uint32_t m, s;
  __device__ __forceinline__ int of(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> s); }
};

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
  float scale_log2;  // |softmax_scale| log2(e)
  uint32_t q_sign;   // the scale's sign, as the sign bits of two BF16 values
  int window, B, T, Hq, Hkv, group, num_pages, log_p, max_pages;
  Divisor by_group, by_heads;  // group, Hkv
  int cus;         // compute units
  int most_units;  // units that splitting may add; 0: no splitting
  int first_unit;  // the launch's first unit (0 with splitting)

  // The first key that a row at position `pos` sees. (A window may be 2^31 - 1 wide, and rows
  // below position 0, which see none, far below it.)
  __device__ __forceinline__ int first_key(int pos) const { return window ? max(0, max(pos, -1) - window + 1) : 0; }
};

// Chunks of `len` keys that `keys` keys make, and keys rounded up to whole steps of four waves.
// A tile that may not be cut is one chunk at every length that a call can have.
constexpr __host__ __device__ int pieces(int keys, int len) { return (int)(((uint32_t)keys + (uint32_t)len - 1) / (uint32_t)len); }
constexpr __host__ __device__ int up128(int keys) { return (int)(((uint32_t)keys + 127) / 128 * 128); }
static_assert(pieces(kMostKeys, kWhole) == 1 && pieces(kMostKeys, up128((int)(float)kWhole)) == 1 && up128(kMostKeys) == kMostKeys);
static_assert((int64_t)kMostKeys + 64 * 32 <= INT32_MAX);

// What a sequence asks for: its row tiles, and the most keys that one of them reads. With a
// window that is an upper bound, as if a tile held all new tokens: with the tile's own tokens
// alone 4 x 300 tokens in a window of 1024 take 45 us in place of 48, but 2048 tokens of eight
// heads on one key head 42 in place of 29.
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

// How the call's work is cut, by an estimate of the time in keys that a CU reads in it (a CU
// reads about 100 keys of 128 columns a microsecond). `even` keys are a CU's share.
//   One unit for each CU, nothing but a start and an end that do not overlap: needs chunks of
//     `even` keys or a little more, so that the tiles' last chunks fit as well.
//   Tiles whole: the longest as often as there are rounds, or, of ragged lengths, the share
//     and a part of the longest.
//   Several rounds of chunks of c keys: the share, that part of c, and what each unit's start
//     and end cost; least at c = sqrt(kUnitCost / kTail even).
// Measured, heads of 128, 8 key heads, one unit for each CU, whole tiles, rounds of 1024 and
// of 2048: 4 x 65536 keys 86, -, 104, 99 us; 64 x 8192 -, 166, 181, 181; 64 users of 500 to
// 8192 keys -, 133, 115, 114; 16 x 16000 88, 106, 106, 95.
constexpr float kUnitCost = 200.f;
constexpr float kTail = 0.4f;
template <int TILE, int STEP>
struct Plan {
  Sequence seq;   // the lane's sequence and demand, of the 64 looked at last
  Demand want;
  int chunk_len;

  __device__ __forceinline__ int chunks_of(int keys) const { return pieces(keys, chunk_len); }
  __device__ __forceinline__ void look(const AttentionParams& p, int base) {
    const int b = base + (threadIdx.x & 63);
    seq = {}, want = {};
    if (b < p.B) {
      seq = sequence(p.cu_q, p.seq_lens, b, p.T, p.max_pages << p.log_p);
      want = demand<TILE, STEP>(seq, p);
    }
  }
  __device__ __forceinline__ int rounded(float chunk) const {
    return max(kMinChunk, up128((int)fminf(chunk, (float)kWhole)));
  }
  // unit_cost: kUnitCost for the call's head size.
  __device__ __forceinline__ void make(const AttentionParams& p, float unit_cost) {
    chunk_len = kWhole;
    if (p.most_units == 0) return;
    // in FP32: every wave of the call gets the same sums
    float keys = 0.f, tiles = 0.f, most = 0.f;
    for (int base = 0; base < p.B; base += 64) {
      look(p, base);
      keys += wave_sum((float)want.tiles * (float)want.keys);
      tiles += wave_sum((float)want.tiles);
      most = fmaxf(most, wave_max((float)want.keys));
    }
    keys *= (float)p.Hkv, tiles *= (float)p.Hkv;
    const float cus = (float)p.cus, even = keys * __builtin_amdgcn_rcpf(cus);
    // one each, where half of every tile's last chunk is empty
    float chunk = keys * __builtin_amdgcn_rcpf(fmaxf(cus - 0.5f * tiles, 0.5f * cus));
    if (chunk > kMinChunk) {
      if (tiles < cus && p.B <= 64) {  // or exactly, if so many units are no more than the CUs: two counts in one sum
        const int n = last_lane(wave_scan(units(even) + (units(1.125f * even) << 16))) * p.Hkv;
        if ((n >> 16) <= p.cus) chunk = (n & 0xFFFF) <= p.cus ? even : 1.125f * even;
      }
      const float rounds = ceilf(tiles * __builtin_amdgcn_rcpf(cus));
      const float whole = fminf(rounds * most, even + kTail * most) + rounds * unit_cost;
      const float several = __builtin_amdgcn_sqrtf(unit_cost * (1.f / kTail) * even);
      float cost = tiles < cus ? chunk + unit_cost : INFINITY;
      if (whole < cost) chunk = most, cost = whole;
      if (even + 2.f * kTail * several < cost) chunk = several;
    }
    // one level of joining where that takes chunks of two steps for each wave at most (1500
    // keys of one user: 10.3 us by two levels, 9.1 by one; 2500 keys: 10.5 and 10.7)
    if (most <= 2.f * kMinChunk * kJoin) chunk = fmaxf(chunk, most * (1.f / kJoin));
    // a ten-thousandth more than the sums can be off: no more units than there are slots
    chunk_len = rounded(fmaxf(chunk, keys * __builtin_amdgcn_rcpf((float)p.most_units) * 1.0001f));
  }
  // The lane's sequence in about so many keys each (tiles times chunks).
  __device__ __forceinline__ int units(float chunk) const {
    return want.tiles * (int)ceilf((float)want.keys * __builtin_amdgcn_rcpf((float)rounded(chunk)) - 1e-3f);
  }
};

// A unit of work. Everything is wave-uniform.
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
// Unit `number`, found by scanning the sequences' unit counts (every wave does it for
// itself); false if there is none.
template <int TILE, int STEP>
__device__ __forceinline__ bool find_unit(const AttentionParams& p, Plan<TILE, STEP>& plan, int number, Unit& u) {
  u.slot = number;
  const int want = p.by_heads.of(number);
  u.h = number - want * p.Hkv;
  int before = 0, tiles_before = 0;
  for (int base = 0; base < p.B; base += 64) {
    if (p.B > 64 || p.most_units == 0) plan.look(p, base);
    const Demand d = plan.want;
    const int count = d.tiles * max(1, plan.chunks_of(d.keys));
    const int incl = wave_scan(count);
    const uint64_t hit = __ballot(want < before + incl);
    if (hit) {
      const int src = __ffsll((unsigned long long)hit) - 1;
      auto pick = [&](int v) { return __builtin_amdgcn_readlane(v, src); };
      const int tiles_incl = wave_scan(d.tiles);
      u.b = base + src;
      u.seq = {pick(plan.seq.row0), pick(plan.seq.rows), pick(plan.seq.start), pick(plan.seq.len)};
      u.tiles = pick(d.tiles);
      const int within = want - (before + pick(incl - count));
      if ((uint32_t)within >= (uint32_t)pick(count)) return false;  // only where overlapping rows overflow the sums
      u.chunk = (uint32_t)within / (uint32_t)u.tiles;
      u.tile = u.tiles - 1 - (within - u.chunk * u.tiles);  // the tiles with the most keys first
      u.tile_id = (tiles_before + pick(tiles_incl - d.tiles) + u.tile) * p.Hkv + u.h;
      const int total = u.seq.rows * p.group;
      u.row0 = u.tile * TILE;
      u.rows = min(TILE, total - u.row0);
      u.pos0 = u.seq.start + p.by_group.of(u.row0);
      u.pos1 = u.seq.start + p.by_group.of(u.row0 + u.rows - 1);
      u.lo = min(p.first_key(u.pos0), u.seq.len) / STEP * STEP;
      u.hi = max(u.lo, min(u.seq.len, u.pos1 + 1));
      // as many chunks as the length asks for, of equal length
      const int keys = u.hi - u.lo;
      const int len = max(kMinChunk, up128(pieces(keys, max(1, plan.chunks_of(keys)))));
      u.chunks = max(1, pieces(keys, len));
      // Where rows overlap (cu_q is not trusted), more units can be asked for than there are: a
      // tile whose chunks do not all have a workgroup and a slot, or whose counter would not be
      // a tile's, stays whole, so that everyone whom a counter waits for arrives.
      const int64_t last_slot = number + (int64_t)(u.chunks - 1 - u.chunk) * u.tiles * p.Hkv;
      const bool whole = u.chunks > 1 && (last_slot >= (int64_t)gridDim.x || u.tile_id >= kTileCounters);
      if (whole) u.chunks = 1;
      if (u.chunk >= u.chunks) return false;  // also a tile that sees fewer keys than the sequence's last
      u.k0 = min(u.hi, u.lo + u.chunk * len);
      u.k1 = whole ? u.hi : (int)min((uint32_t)u.hi, (uint32_t)u.k0 + len);
      return true;
    }
    before += last_lane(incl);
    tiles_before += last_lane(wave_scan(d.tiles));
  }
  return false;  // the grid covers the most units that there can be
}

// Waits and loads into LDS. The compiler does not track these loads; each wait stands
// between scheduling barriers, so that nothing written after it is done before it.
__device__ __forceinline__ void fence_schedule() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
template <int N>
__device__ __forceinline__ void wait_loads() {  // until at most N are outstanding
  static_assert(N >= 0 && N < 64, "vmcnt range");
  fence_schedule();
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
  fence_schedule();
}
__device__ __forceinline__ void wait_lds_reads() {
  fence_schedule();
  __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));
  fence_schedule();
}
// Every lane's 16 bytes at base + off, to LDS at lds + 16 * lane. base and lds are
// wave-uniform. STREAM: with the hint that the lines are read once.
template <bool STREAM>
__device__ __forceinline__ void load_to_lds(const uint8_t* base, uint32_t off, uint32_t lds) {
  if constexpr (STREAM)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt" ::"v"(off), "s"(base), "s"(lds) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}
// One stage of a wave's ring: 32 keys in the order their lanes feed them ([16-key group]
// [64-byte piece][lane][16 bytes]), then 32 values, row after row, each row's 16-byte pieces
// permuted by an exclusive or with a number of the row, so that the rows which are read
// together lie in different banks.
template <int D, bool STREAM>
struct Stage {
  static constexpr int kPieces = D / 64;            // 64-byte pieces of a row
  static constexpr int kLoads = 2 * kPieces;        // load instructions of a half
  static constexpr int kHalf = 32 * D, kBytes = 2 * kHalf;
  static constexpr int kShared = D == 64 ? 2 : D == 128 ? 1 : 0;  // log2 of the rows in one line of the 64 banks
  static constexpr int kLane16 = D / 16;            // 16-byte pieces of a row
  // row 0 .. 31 of a stage; the 16 rows r & 8 apart from each other share no bank
  static __device__ __forceinline__ constexpr uint32_t turn(int row) { return ((row & 7) >> kShared | (row >> 4) << (3 - kShared)) * 16; }
  // base0, base1: first rows of the two 16-key groups
  static __device__ __forceinline__ void load_keys(const uint8_t* base0, const uint8_t* base1, uint32_t lds, int lane) {
    const uint32_t off = (lane & 15) * D + (lane >> 4) * 16;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      load_to_lds<STREAM>((i < kPieces ? base0 : base1) + (i % kPieces) * 64, off, lds + i * 1024);
  }
  static __device__ __forceinline__ void load_values(const uint8_t* base0, const uint8_t* base1, uint32_t lds, int lane) {
    constexpr int kRows = 1024 / D;  // of an instruction
    const uint32_t off = lane * 16 ^ turn(lane / kLane16 & 7);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      load_to_lds<STREAM>((i < kPieces ? base0 : base1) + (i % kPieces) * 1024, off ^ turn(i * kRows), lds + kHalf + i * 1024);
  }
  // Where the lane reads for the transposing load of value columns 16 t .. 16 t + 15, but
  // for an exclusive or with 16 t: of 16 lanes, two hold a row's halves.
  static __device__ __forceinline__ uint32_t value_at(int lane) {
    const int j = (lane & 15) >> 1, row = (j >> 2) * 16 + (lane >> 4) * 4 + (j & 3);
    return row * D + turn(row) + (lane & 1) * 8;
  }
};

// Eight values of one column each: 16 lanes read 8 rows of 16 bytes, and lane n gets the rows'
// bytes n in their order.
typedef int v2i __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint2 load_columns(uint32_t lds) {
  const v2i x = __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) v2i*)(uintptr_t)lds);
  return make_uint2((uint32_t)x.x, (uint32_t)x.y);
}

// Eight codes to BF16, exactly.
__device__ __forceinline__ v8bf codes_bf16(uint32_t a, uint32_t b) {
  const v2bf x0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
  const v2bf x1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
  const v2bf x2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
  const v2bf x3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
  return v8bf{x0.x, x0.y, x1.x, x1.y, x2.x, x2.y, x3.x, x3.y};
}

// Eight codes to FP16, exactly.
__device__ __forceinline__ v8h codes_f16(uint2 w) {
  const v2h x0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w.x, 1.0f, false);
  const v2h x1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w.x, 1.0f, true);
  const v2h x2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w.y, 1.0f, false);
  const v2h x3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w.y, 1.0f, true);
  return v8h{x0.x, x0.y, x1.x, x1.y, x2.x, x2.y, x3.x, x3.y};
}

// Exponent field of a power of two.
__device__ __forceinline__ int exponent(uint32_t bits) { return (int)((bits >> 23) & 0xFF); }
__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// Bit 7 of each of the four codes that is NaN.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Partial results travel between workgroups (of any XCD) as device-coherent accesses.
constexpr int kDeviceScope = 16;        // buffer cache policy sc1
constexpr int kRawDword3 = 0x00020000;  // buffer descriptor: 32-bit untyped

// Arrives at a counter; true for the last of `expected`, who leaves it zero. Called by the
// whole workgroup, after stores that the others' results must be seen through.
__device__ __forceinline__ bool arrive_last(int32_t* counter, int expected, int* flag) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the stores have reached the device-coherent level
  __syncthreads();
  if (threadIdx.x == 0) {
    const bool last = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == expected - 1;
    if (last) __hip_atomic_store(counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *flag = last;
  }
  __syncthreads();
  return *flag != 0;
}

// C columns of one row of a result, normalised, with its log sum exp in base 2.
template <int C>
struct RowPart {
  float out[C];
  float lse2;
};

// Joins n parts of R rows, `stride` bytes apart from at[i] (columns) and lse_at[i] (log
// sum): the loads of as many parts as registers hold are in flight together.
template <int R, int C>
__device__ __forceinline__ void join_parts(RowPart<C> (&r)[R], __amdgpu_buffer_rsrc_t rs, const int (&at)[R], const int (&lse_at)[R],
                                           int stride, int n) {
  constexpr int kBatch = R * C <= 16 ? kJoin : kJoin / 2;
  float top[R], sum[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    top[i] = -INFINITY, sum[i] = 0.f;
#pragma unroll
    for (int t = 0; t < C; ++t) r[i].out[t] = 0.f;
  }
  for (int base = 0; base < n; base += kBatch) {
    float w[R][kBatch];
    v4f y[R][kBatch][C / 4];
#pragma unroll
    for (int c = 0; c < kBatch; ++c) {
      const int off = min(base + c, n - 1) * stride;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        w[i][c] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, off + lse_at[i], 0, kDeviceScope));
#pragma unroll
        for (int t = 0; t < C / 4; ++t)
          y[i][c][t] = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rs, off + at[i] + t * 16, 0, kDeviceScope));
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float most = top[i];
#pragma unroll
      for (int c = 0; c < kBatch; ++c) {
        if (base + c >= n) w[i][c] = -INFINITY;
        most = fmaxf(most, w[i][c]);
      }
      const float ref = most > -INFINITY ? most : 0.f;  // rows that have seen nothing stay at weight 0
      const float a = exp2_of(top[i] - ref);
      sum[i] *= a;
#pragma unroll
      for (int t = 0; t < C; ++t) r[i].out[t] *= a;
#pragma unroll
      for (int c = 0; c < kBatch; ++c) {
        const float b = base + c < n ? exp2_of(w[i][c] - ref) : 0.f;
        sum[i] += b;
#pragma unroll
        for (int t = 0; t < C; ++t) r[i].out[t] += base + c < n ? b * y[i][c][t / 4][t % 4] : 0.f;
      }
      top[i] = most;
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const float inv = sum[i] == 0.f ? 0.f : __builtin_amdgcn_rcpf(sum[i]);
#pragma unroll
    for (int t = 0; t < C; ++t) r[i].out[t] *= inv;
    r[i].lse2 = sum[i] == 0.f ? -INFINITY : top[i] + __log2f(sum[i]);
  }
}

// Publishes a unit's rows, joins the tile's parts if it is the last to arrive, and writes
// the rows out. Thread (r, x) holds rows r + 16 i, columns x C .. x C + C - 1.
template <int D, int R, int C>
__device__ __forceinline__ void finish_unit(const AttentionParams& p, const Unit& u, RowPart<C> (&part)[R], int* flag) {
  const int r = threadIdx.x >> 4, x = threadIdx.x & 15;
  if (u.chunks > 1) {
    constexpr int kSlotFloats = 16 * R * (D + 1);
    const int step = u.tiles * p.Hkv;  // slots between neighbouring chunks of a tile
    const int first = u.slot - u.chunk * step;
    const int stride = step * kSlotFloats * 4;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        p.parts + (int64_t)first * kSlotFloats, 0, (u.chunks - 1) * stride + kSlotFloats * 4, kRawDword3);
    auto publish = [&](int off) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int row = r + 16 * i;
        if (row < u.rows) {
#pragma unroll
          for (int t = 0; t < C; t += 4)
            __builtin_amdgcn_raw_buffer_store_b128(
                __builtin_bit_cast(v4u, v4f{part[i].out[t], part[i].out[t + 1], part[i].out[t + 2], part[i].out[t + 3]}), rs,
                off + (row * D + x * C + t) * 4, 0, kDeviceScope);
          if (x == 0)
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(part[i].lse2), rs, off + (16 * R * D + row) * 4, 0, kDeviceScope);
        }
      }
    };
    auto join = [&](int off, int gap, int n) {
      int at[R], lse_at[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int row = min(r + 16 * i, u.rows - 1);  // rows past the tile: as its last, and not written
        at[i] = off + (row * D + x * C) * 4, lse_at[i] = off + (16 * R * D + row) * 4;
      }
      join_parts<R, C>(part, rs, at, lse_at, gap, n);
    };
    // first the group of kJoin neighbours that this unit is one of, then the groups, whose
    // results stand in their first member's place
    const int group = u.chunk / kJoin, groups = (u.chunks + kJoin - 1) / kJoin;
    const int in_group = min(kJoin, u.chunks - group * kJoin);
    const int group_off = group * kJoin * stride;
    if (in_group > 1) {
      publish(u.chunk * stride);
      if (!arrive_last(&p.counters[kTileCounters + first + group * kJoin * step], in_group, flag)) return;
      join(group_off, stride, in_group);
    }
    if (groups > 1) {
      __syncthreads();  // the flag is used again
      publish(group_off);
      if (!arrive_last(&p.counters[u.tile_id], groups, flag)) return;
      join(0, kJoin * stride, groups);
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = r + 16 * i;
    if (row < u.rows) {
      const int rr = u.row0 + row;
      const int in_seq = p.by_group.of(rr);
      const int64_t token = u.seq.row0 + in_seq;
      const int head = u.h * p.group + rr - in_seq * p.group;
      uint16_t* dst = p.O + token * p.ldo + head * D + x * C;
#pragma unroll
      for (int t = 0; t < C; t += 4)
        *reinterpret_cast<uint2*>(dst + t) =
            make_uint2(pack_bf16(part[i].out[t], part[i].out[t + 1]), pack_bf16(part[i].out[t + 2], part[i].out[t + 3]));
      if (p.lse && x == 0) p.lse[token * p.Hq + head] = part[i].lse2 * 0.6931471805599453f;
    }
  }
}

// Eight weights of a row from a lane's logits s (times c), by exponent offsets a0 and a1 of
// the two 16-key groups, as FP16; k0 and k1 turn their sums into l's terms.
__device__ __forceinline__ v8h weights(const v4f& s0, const v4f& s1, float c0, float c1, float a0, float a1, float k0, float k1,
                                       float& l) {
  float w[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w[j] = exp2_of(__builtin_fmaf(s0[j], c0, a0));
    w[4 + j] = exp2_of(__builtin_fmaf(s1[j], c1, a1));
  }
  l = __builtin_fmaf((w[0] + w[1]) + (w[2] + w[3]), k0, l);
  l = __builtin_fmaf((w[4] + w[5]) + (w[6] + w[7]), k1, l);
  v8h out;
#pragma unroll
  for (int j = 0; j < 8; ++j) out[j] = (_Float16)w[j];
  return out;
}
__device__ __forceinline__ v8h weights(const v4f& s0, const v4f& s1, float c, float a, float k, float& l) {
  float w[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w[j] = exp2_of(__builtin_fmaf(s0[j], c, a));
    w[4 + j] = exp2_of(__builtin_fmaf(s1[j], c, a));
  }
  l = __builtin_fmaf(((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7])), k, l);
  v8h out;
#pragma unroll
  for (int j = 0; j < 8; ++j) out[j] = (_Float16)w[j];
  return out;
}
// A maximum as a chain from a constant: the compiler makes it of maxima of three, and of a
// chain only its first operands, if they could be signalling NaN, cost an instruction to
// quiet. (Not as inline assembly: the waits between a matrix instruction and a reader of
// its result are the compiler's to insert, and it does not for assembly.)
__device__ __forceinline__ float max4(float from, const v4f& s) { return fmaxf(fmaxf(fmaxf(fmaxf(from, s[0]), s[1]), s[2]), s[3]); }
__device__ __forceinline__ bool rarely(bool x) { return __builtin_expect(x, 0); }

// Workgroups that registers leave room for on a CU.
constexpr int attention_residents(int D, int R) { return D == 64 ? (R == 1 ? 4 : R == 2 ? 3 : 2) : D == 128 ? 2 : 1; }

// STREAM: no other unit reads this one's keys and values. The hint is worth 10% then (64
// users of 8192 keys: 183 us without, 165 with, 6.5 TB/s) and costs 4% where many tiles
// share them (2048 prompt tokens in 32-row tiles: 488 and 506 us).
// WIDE: pages hold 32 keys and more, so that a step has one scale of each kind. Worth 4%
// where vector instructions set the pace (2 x 2048 prompt tokens over 8192 keys: 544 us without,
// 524 with, 918 TFLOP/s), nothing where memory does, so only shared tiles have it.
template <int D, int R, bool STREAM, bool WIDE>
__global__ void __launch_bounds__(256, attention_residents(D, R)) attention_kernel(const AttentionParams p) {
  using Ring = Stage<D, STREAM>;
  constexpr int kTiles = D / 16;       // 16-column tiles of V
  constexpr int kStride = D + 4;       // of a row of O in LDS
  // the ring, and after the loop the waves' results, 16 rows at a time
  constexpr int kRingBytes = 4 * 2 * Ring::kBytes, kResultBytes = 4 * 16 * kStride * 4;
  __shared__ __align__(256) uint8_t shared[kRingBytes > kResultBytes ? kRingBytes : kResultBytes];
  __shared__ float m_sh[4][16], mo_sh[4][16], l_sh[4][16];
  __shared__ int flag;
  auto o_sh = reinterpret_cast<float(*)[16][kStride]>(shared);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, kg = lane >> 4;
  Plan<16 * R, 32> plan;
  plan.make(p, kUnitCost * 128 / D);
  Unit u;
  if (!find_unit(p, plan, p.first_unit + (int)blockIdx.x, u)) return;

  const int steps = (u.k1 - u.k0 + 31) >> 5, share = (steps + 3) >> 2;
  const int step0 = min(steps, wave * share), step1 = min(steps, step0 + share);

  // A segment is up to 32 steps, of whose 64 groups of 16 keys lane i holds what group i
  // needs: where its rows start in the caches, the factor of its logits, and the base 2
  // logarithm of its value scale. The loads of a unit's start depend on each other in
  // three rounds: the sequences, the pages, and then at once the scales, the queries and
  // the first two stages.
  auto page_of_lane = [&](int seg) {
    const int key = u.k0 + seg * 32 + lane * 16;
    return seg < step1 && key < u.k1 ? p.block_table[u.b * p.ld_bt + (key >> p.log_p)] : -1;
  };
  struct Segment {
    uint32_t at_lo, at_hi;
    float c, v;
    uint64_t holes, changes;  // groups without a page; with another value scale than two groups before
    int count;
  };
  const uint8_t* ring = shared + wave * 2 * Ring::kBytes;
  const uint32_t ring_lds = __builtin_amdgcn_readfirstlane(lds_address(ring));
  const uint32_t value_at = lds_address(ring) + Ring::kHalf + Ring::value_at(lane);
  Segment g;
  auto rows_of = [&](const uint8_t* cache, int i) {
    const uint32_t lo = __builtin_amdgcn_readlane(g.at_lo, i), hi = __builtin_amdgcn_readlane(g.at_hi, i);
    return cache + ((uint64_t)hi << 32 | lo);
  };
  auto fetch_keys = [&](int s) {
    Ring::load_keys(rows_of(p.k_cache, 2 * s), rows_of(p.k_cache, 2 * s + 1), ring_lds + (s & 1) * Ring::kBytes, lane);
  };
  auto fetch_values = [&](int s) {
    Ring::load_values(rows_of(p.v_cache, 2 * s), rows_of(p.v_cache, 2 * s + 1), ring_lds + (s & 1) * Ring::kBytes, lane);
  };
  float ks = 0.f, vs = 0.f;
  auto open = [&](int seg, int page) {  // starts a segment's loads
    const int key = u.k0 + seg * 32 + lane * 16;
    const bool there = page >= 0 && page < p.num_pages;
    const int64_t head = (int64_t)page * p.Hkv + u.h;
    const uint64_t at = there ? (uint64_t)((head << p.log_p) + (key & ((1 << p.log_p) - 1))) * D : 0;  // page 0 stands in for none
    g.at_lo = (uint32_t)at, g.at_hi = (uint32_t)(at >> 32);
    g.holes = ~__ballot(there);
    g.count = min(32, step1 - seg);
    ks = vs = 0.f;
    if (there) ks = p.k_scale[head], vs = p.v_scale[head];
    if (g.count > 0) {
      fetch_keys(0);
      fetch_values(0);
      if (g.count > 1) {
        fetch_keys(1);
        fetch_values(1);
      }
    }
    fence_schedule();
  };
  auto settle = [&]() {  // once the scales are there
    g.c = __uint_as_float(__float_as_uint(ks) & 0x7F800000u) * p.scale_log2;
    g.v = (float)(exponent(__float_as_uint(vs)) - 127);
    const float before = __shfl(g.v, max(lane - 2, 0), 64);
    g.changes = __ballot(lane < 2 || g.v != before);
  };
  auto of_lane = [&](float v, int i) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), i)); };
  const int first_page = page_of_lane(step0);

  // this lane's rows: query fragments, and the keys that each sees, [key_lo, key_hi)
  int key_lo[R], key_hi[R];
  uint4 q_raw[R][D / 32];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const bool live = n + 16 * i < u.rows;
    const int row = u.row0 + (live ? n + 16 * i : 0);
    const int token = p.by_group.of(row), head = u.h * p.group + row - token * p.group;
    const int pos = u.seq.start + token;
    key_hi[i] = min(u.seq.len, pos + 1);
    key_lo[i] = p.first_key(pos);
    const uint16_t* src = p.q + (int64_t)(u.seq.row0 + token) * p.ldq + head * D;
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
      q_raw[i][s] = make_uint4(0, 0, 0, 0);
      if (live) q_raw[i][s] = *reinterpret_cast<const uint4*>(src + (s >> 1) * 64 + kg * 16 + (s & 1) * 8);
    }
  }
  fence_schedule();
  open(step0, first_page);
  v8bf qf[R][D / 32];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {  // the scale's sign is taken here, so that the factors of logits are not negative
      const uint4 x = q_raw[i][s];
      qf[i][s] = __builtin_bit_cast(v8bf, make_uint4(x.x ^ p.q_sign, x.y ^ p.q_sign, x.z ^ p.q_sign, x.w ^ p.q_sign));
    }
  // keys that every row of the tile sees
  const int all_hi = min(u.seq.len, u.pos0 + 1), all_lo = p.first_key(u.pos1);

  v4f o[R][kTiles];
  float m[R], mo[R], l[R];
  float a0[R], a1[R], k0[R], k1[R];  // offsets and factors of the step's two 16-key groups
#pragma unroll
  for (int i = 0; i < R; ++i) {
    m[i] = mo[i] = kNone, l[i] = 0.f;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) o[i][t] = v4f{0.f, 0.f, 0.f, 0.f};
  }

  for (int seg = step0; seg < step1; seg += 32) {
    if (seg > step0) open(seg, page_of_lane(seg));
    settle();
    const int count = g.count;
    for (int s = 0; s < count; ++s) {
      const int left = count - 1 - s;  // steps after this one
      const uint8_t* stage = ring + (s & 1) * Ring::kBytes;
      const int key = u.k0 + (seg + s) * 32;
      float c0 = of_lane(g.c, 2 * s), c1 = of_lane(g.c, 2 * s + 1);
      const float v0 = of_lane(g.v, 2 * s), v1 = of_lane(g.v, 2 * s + 1);
      const uint32_t hole = (uint32_t)(g.holes >> (2 * s)) & 3;

      v4f s0[R], s1[R];
#pragma unroll
      for (int i = 0; i < R; ++i) s0[i] = s1[i] = v4f{0.f, 0.f, 0.f, 0.f};
      if (left >= 1) wait_loads<3 * Ring::kLoads>();
      else wait_loads<Ring::kLoads>();
      uint4 kx[2][D / 64];
#pragma unroll
      for (int i = 0; i < Ring::kLoads; ++i)
        kx[i / Ring::kPieces][i % Ring::kPieces] = *reinterpret_cast<const uint4*>(stage + i * 1024 + lane * 16);
      if (left >= 2) {
        wait_lds_reads();
        fetch_keys(s + 2);
      }
#pragma unroll
      for (int d = 0; d < D / 32; ++d) {
        const uint4 x = kx[0][d >> 1], y = kx[1][d >> 1];
        const v8bf a = (d & 1) ? codes_bf16(x.z, x.w) : codes_bf16(x.x, x.y);
        const v8bf b = (d & 1) ? codes_bf16(y.z, y.w) : codes_bf16(y.x, y.y);
#pragma unroll
        for (int i = 0; i < R; ++i) {
          s0[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, qf[i][d], s0[i], 0, 0, 0);
          s1[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, qf[i][d], s1[i], 0, 0, 0);
        }
      }
      // some row does not see all of the step
      auto seen = [&](int i, int j) {
        const int at = key + (j >> 2) * 16 + kg * 4 + (j & 3);
        return (hole >> (j >> 2) & 1) == 0 && at >= key_lo[i] && at < key_hi[i];
      };
      const bool partly = key < all_lo || key + 32 > all_hi || hole != 0;
      if (rarely(partly)) {
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (j < 4) s0[i][j] = seen(i, j) ? s0[i][j] * c0 : -INFINITY;  // factors may be 0: they come before the mask
            else s1[i][j - 4] = seen(i, j) ? s1[i][j - 4] * c1 : -INFINITY;
          }
        c0 = c1 = 1.f;
      }
      float top[R], top_o[R];
      bool move = false;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if constexpr (WIDE) {
          top[i] = max4(max4(kNone, s0[i]), s1[i]) * c0, top_o[i] = top[i] + v0;
        } else {
          const float t0 = max4(kNone, s0[i]) * c0, t1 = max4(kNone, s1[i]) * c1;
          top[i] = fmaxf(t0, t1), top_o[i] = fmaxf(t0 + v0, t1 + v1);
        }
        move |= fmaxf(top[i] - m[i], top_o[i] - mo[i]) > kLag;
      }
      const bool moved = __any(move);
      if (rarely(moved)) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          float t = fmaxf(top[i], __shfl_xor(top[i], 16, 64)), to = fmaxf(top_o[i], __shfl_xor(top_o[i], 16, 64));
          t = fmaxf(m[i], fmaxf(t, __shfl_xor(t, 32, 64))), to = fmaxf(mo[i], fmaxf(to, __shfl_xor(to, 32, 64)));
          l[i] *= exp2_of(m[i] - t);
          const float b = exp2_of(mo[i] - to);
          m[i] = t, mo[i] = to;
#pragma unroll
          for (int t2 = 0; t2 < kTiles; ++t2) o[i][t2] *= b;
        }
      }
      if (rarely(moved || (g.changes >> (2 * s) & 3) != 0)) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          a0[i] = fmaxf(v0 + (15 - kLag) - mo[i], kFar - m[i]), k0[i] = exp2_of(-(a0[i] + m[i]));
          if constexpr (!WIDE) a1[i] = fmaxf(v1 + (15 - kLag) - mo[i], kFar - m[i]), k1[i] = exp2_of(-(a1[i] + m[i]));
        }
      }
      v8h pf[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if constexpr (WIDE) pf[i] = weights(s0[i], s1[i], c0, a0[i], k0[i], l[i]);
        else pf[i] = weights(s0[i], s1[i], c0, c1, a0[i], a1[i], k0[i], k1[i], l[i]);
      }
      if (left >= 2) wait_loads<3 * Ring::kLoads>();
      else if (left == 1) wait_loads<2 * Ring::kLoads>();
      else wait_loads<0>();
      uint2 v[kTiles];  // this lane's values: keys 4 kg + j, and 16 further for j >= 4, of column 16 t + n
      const uint32_t at_values = value_at + (s & 1) * Ring::kBytes;
#pragma unroll
      for (int t = 0; t < kTiles; ++t) v[t] = load_columns(at_values ^ t * 16);
      if (left >= 2) {
        wait_lds_reads();
        fetch_values(s + 2);
      }
      if (rarely(partly)) {
        // values that no row sees may be anything: they count as 0. Where a row sees a NaN
        // code and another does not, the product gets 0, and o of the rows that see it
        // becomes NaN here.
        uint32_t see[2] = {0, 0}, nan[2] = {0, 0};  // a byte for each key
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int at = key + (j >> 2) * 16 + kg * 4 + (j & 3);
          see[j >> 2] |= (hole >> (j >> 2) & 1) == 0 && at >= u.lo && at < u.hi ? 0xFFu << (j & 3) * 8 : 0u;
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          v[t].x &= see[0], v[t].y &= see[1];
          const uint32_t x = nan_codes(v[t].x), y = nan_codes(v[t].y);
          nan[0] |= x, nan[1] |= y;
          v[t].x &= ~((x >> 7) * 0xFF), v[t].y &= ~((y >> 7) * 0xFF);
        }
        if (rarely(__any((nan[0] | nan[1]) != 0))) {
#pragma unroll
          for (int off = 1; off < 16; off <<= 1)  // over the lanes that feed the same keys
            nan[0] |= __shfl_xor((int)nan[0], off, 64), nan[1] |= __shfl_xor((int)nan[1], off, 64);
#pragma unroll
          for (int i = 0; i < R; ++i) {
            int bad = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) bad |= (nan[j >> 2] >> (8 * (j & 3) + 7) & 1) && seen(i, j);
            bad |= __shfl_xor(bad, 16, 64);
            bad |= __shfl_xor(bad, 32, 64);
            if (bad) {
#pragma unroll
              for (int t = 0; t < kTiles; ++t) o[i][t] = v4f{__builtin_nanf(""), __builtin_nanf(""), __builtin_nanf(""), __builtin_nanf("")};
            }
          }
        }
      }
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        const v8h a = codes_f16(v[t]);
#pragma unroll
        for (int i = 0; i < R; ++i) o[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pf[i], o[i][t], 0, 0, 0);
      }
    }
  }

  // join the four waves: row n + 16 i's column 16 t + 4 kg + j is o[i][t][j]; then
  // thread (r, x) has rows r + 16 i, columns x D / 16 .. + D / 16
  RowPart<kTiles> part[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    l[i] += __shfl_xor(l[i], 16, 64);
    l[i] += __shfl_xor(l[i], 32, 64);
    __syncthreads();  // the ring, or the rows before, have been read
#pragma unroll
    for (int t = 0; t < kTiles; ++t) *reinterpret_cast<v4f*>(&o_sh[wave][n][16 * t + 4 * kg]) = o[i][t];
    if (kg == 0) m_sh[wave][n] = m[i], mo_sh[wave][n] = mo[i], l_sh[wave][n] = l[i];
    __syncthreads();
    const int r = threadIdx.x >> 4, x = threadIdx.x & 15;
    float top = kNone, top_o = kNone, sum = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) top = fmaxf(top, m_sh[w][r]), top_o = fmaxf(top_o, mo_sh[w][r]);
#pragma unroll
    for (int t = 0; t < kTiles; ++t) part[i].out[t] = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      sum += exp2_of(m_sh[w][r] - top) * l_sh[w][r];
      const float b = exp2_of(mo_sh[w][r] - top_o);
#pragma unroll
      for (int t = 0; t < kTiles; t += 4) {
        const float4 y = *reinterpret_cast<const float4*>(&o_sh[w][r][x * kTiles + t]);
        part[i].out[t] += y.x * b, part[i].out[t + 1] += y.y * b, part[i].out[t + 2] += y.z * b, part[i].out[t + 3] += y.w * b;
      }
    }
    // o stands for itself times 2^(mo - m - (15 - kLag)), in two factors so that each is in
    // range; a row that saw no key gives 0, and minus infinity
    const float inv = sum == 0.f ? 0.f : __builtin_amdgcn_rcpf(sum);
    const float shift = fminf(fmaxf(0.5f * (top_o - top - (15 - kLag)), -126.f), 126.f), half = exp2_of(shift);
#pragma unroll
    for (int t = 0; t < kTiles; ++t) part[i].out[t] = part[i].out[t] * inv * half * half;
    part[i].lse2 = sum == 0.f ? -INFINITY : top + __log2f(sum);
  }
  finish_unit<D, R, kTiles>(p, u, part, &flag);
}

}  // namespace fp8layer
