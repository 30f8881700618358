// cache_attention_kernel.h -- the attention kernel over the 4-bit cache, one
// template for all head widths, group sizes and tile heights; each
// cache_attention_*.hip instantiates one width.
//
// Mathematics. For a query row q and a cached token j with key codes c_jd,
// scales s_jg and value codes and scales c'_jd, s'_jg (g the channel's group):
//   a_j = scale * sum_g s_jg * (sum_{d in g} q_d c_jd)
//   out_d = sum_j p_j s'_jg c'_jd / sum_j p_j,   p_j = exp(a_j - m).
// Both products run on the matrix cores with the codes as one operand, exact
// binary16 integers c (u - 8 for affine codes, whose sums then get (z - 8) sum q
// and (z - 8) sum w taken off). Taking a word of 8 codes apart is 9 VALU
// operations. 5 would do with the masked nibbles used as binary16 subnormals
// u * 2^-24, but the matrix instructions align a subnormal as if it were 2^-14:
// measured, the products then lose their bits below 2^-14 of a code, always
// downward. As integers they are truncated below 2^-24 of the largest.
//   scores: the scale multiplies the finished dot product of its group.
//   values: w_j = p_j s'_jg is rounded to binary16 (nearest: 2^-11 of w_j, or 2^-25,
//     half a step of a subnormal, which the reference m below keeps under 2^-33 of the
//     largest p times the largest s'; include/int4dq_cache.h states the bound), since
//     the matrix instructions take no wider operand beside binary16 codes, and a second
//     product for the remainder would double the values' matrix work;
//     affine sums take off (z - 8) times the rounded w, so the offset cancels.
// Queries are brought to [2^13, 2^14) by a power of two per row, which is exact
// for bfloat16 and binary16 down to 2^-27 of the row's largest entry.
//
// The reference m of the running softmax is not the plain maximum: it is kept
// within 6 of max_j a_j + log2 max_j s'_j - 9 (log2 units), which keeps every
// w_j below 2^15 and the large ones far above binary16's subnormals whatever
// the values' magnitude; and it moves only when exceeded by 6, so that the
// accumulators are rescaled a few times a sequence, not every step. Far from zero
// (2^22) a sum of the two cannot be held: its rounding, 2^6 and more from scores of
// 2^30 on, would end up in the exponent. There m is the largest score alone, without
// the 6, and w_j at most a scale. For that the product of score and factor has to be
// exact: the factor is a power of two, and the rest of scale * log2 e goes into the
// keys' scales. (The largest score taken off every score instead: prompts 5% slower;
// in a branch for far scores: 1 to 2%.)
//
// Work. A wavefront takes 64 tokens a step for 16 QT query rows; the four
// wavefronts of a block take turns on a chunk of the tokens and are joined
// through LDS at the end. Scores are computed as (keys x queries), so that a
// lane holds the scores of 16 tokens of one query: these are, in place, the
// operand that the product with the values needs, so probabilities never move
// between lanes. For that, row m = 4a + i of score tile n is token
// 16 a + 4 n + {0, 2, 1, 3}[i] of the step, the order in which a word of four
// tokens' value codes comes apart. The codes come from memory straight
// into the operand's lanes (see the layouts in include/int4dq_cache.h), 16
// bytes a lane for 128 channels, with the next step's loads in flight while
// this one's are used; no LDS in the loop. For prompts the codes are taken apart
// once a block instead, and shared through LDS (see the second kernel).
//
// What bounds it (8 key/value heads of 128 channels, 32 query heads). Token
// generation, 64 sequences of 130 to 8190 tokens, groups of 64, bfloat16: memory, 295
// MB in 67 us. One sequence of 131071 tokens, groups of 32 with zero points: the
// VALU, which takes codes apart and applies scales; 159 MB in 50 us. A prompt of
// 4096 tokens: 137 GFLOP in 192 us, the VALU busy for 56% of it and the matrix pipes
// for 28%, with little overlap at two wavefronts a SIMD.
#pragma once

#include <type_traits>
#include <utility>

#include "cache.h"
#include "cache_schedule.h"
#include "device_common.h"
#include "lanes.h"

namespace int4dq {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------- wavefront sums

// Over the four rows of 16 lanes, lane by lane.
__device__ __forceinline__ float rows_max(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  v = __builtin_fmaxf(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
  const uint32_t w = __builtin_bit_cast(uint32_t, v);
  const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  return __builtin_fmaxf(__builtin_bit_cast(float, (uint32_t)b[0]), __builtin_bit_cast(float, (uint32_t)b[1]));
}
__device__ __forceinline__ float rows_sum(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  v = __builtin_bit_cast(float, (uint32_t)a[0]) + __builtin_bit_cast(float, (uint32_t)a[1]);
  const uint32_t w = __builtin_bit_cast(uint32_t, v);
  const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  return __builtin_bit_cast(float, (uint32_t)b[0]) + __builtin_bit_cast(float, (uint32_t)b[1]);
}

// ---------------------------------------------------------------- the block's share

struct BlockWork {
  int b, tile, chunk, chunks, slot;      // slot: of its partial result, where chunks > 1
  SequenceWork w;
};

// The share of block `unit` of its head; every lane of the wavefront takes part.
// False if it has none. `used`: the slots of partial results in all, where this
// counts them (0 otherwise).
__device__ __forceinline__ bool find_block(const AttentionArgs& a, const Schedule& s, const Workspace& ws, int unit,
                                           BlockWork* out, int* used) {
  const int lane = threadIdx.x & (kWave - 1);
  int i;                                 // the block, counted from the sequence's first
  *used = 0;
  if (s.target > 0 && !s.planned) {      // all sequences at once
    const SequenceWork w = lane < a.r.batch ? sequence_work(a, s.tile_rows, lane) : SequenceWork{};
    const float work = lane_value(lane_scan((float)w.tiles * (float)w.steps), kWave - 1);
    const float tiles = lane_value(lane_scan((float)w.tiles), kWave - 1);
    const int per = steps_per_block(s, work, tiles, lane_max(w.tiles > 0 ? w.steps : 0), [&](int x) {
      return lane_value(lane_scan(w.tiles > 0 ? (chunks_of(w.steps, x) - 1) * w.tiles : 0), kWave - 1);
    });
    const int chunks = w.tiles > 0 ? chunks_of(w.steps, per) : 0;
    const int mine = chunks * w.tiles, mine_slots = chunks > 1 ? mine : 0;
    const int upto = lane_scan(mine), slots_upto = lane_scan(mine_slots);
    *used = lane_value(slots_upto, kWave - 1);
    const uint64_t hit = __ballot(unit >= upto - mine && unit < upto);
    if (hit == 0) return false;
    const int at = __builtin_ctzll(hit);
    out->b = at;
    out->w = SequenceWork{lane_value(w.first, at), lane_value(w.end, at), lane_value(w.rows, at),
                          lane_value(w.length, at), lane_value(w.keys, at), lane_value(w.tiles, at), 0};
    out->chunks = lane_value(chunks, at);
    i = unit - lane_value(upto - mine, at);
    out->slot = lane_value(slots_upto - mine_slots, at) + i;
  } else if (s.target > 0) {
    out->b = lane_search(a.r.batch, unit, [&](int b) { return (int64_t)ws.plan[b].blocks; });
    const PlanEntry from = ws.plan[out->b], to = ws.plan[out->b + 1];
    i = unit - from.blocks;
    if (i < 0 || i >= to.blocks - from.blocks) return false;
    out->w = sequence_work(a, s.tile_rows, out->b);
    out->chunks = (to.blocks - from.blocks) / out->w.tiles;
    out->slot = from.slots + i;
  } else {
    if (a.r.starts) {
      out->b = lane_search(a.r.batch, unit, [&](int b) { return tiles_before(a, s, b); });
      i = unit - (int)tiles_before(a, s, out->b);
    } else {
      const int tiles = (a.ratio + s.tile_rows - 1) / s.tile_rows;
      out->b = unit / tiles;
      if (out->b >= a.r.batch) return false;
      i = unit % tiles;
    }
    out->w = sequence_work(a, s.tile_rows, out->b);
    if (i < 0 || i >= out->w.tiles) return false;
    out->chunks = 1;
    out->slot = 0;
  }
  out->chunk = i % out->chunks;
  out->tile = out->w.tiles - 1 - i / out->chunks;            // tiles that see most first
  return true;
}

// ---------------------------------------------------------------- operands

template <int N>
struct Words {
  uint32_t w[N];
};

// N words from a 4-byte aligned address (16-byte aligned for multiples of 4
// words), in the widest loads that takes.
template <int N>
__device__ __forceinline__ Words<N> load_words(const uint8_t* p) {
  Words<N> r;
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4_t v = reinterpret_cast<const u32x4_t*>(p)[i];
      r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const u32x2_t v = reinterpret_cast<const u32x2_t*>(p)[i];
      r.w[2 * i] = v.x; r.w[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) r.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
  return r;
}

// A word of 8 codes as exact binary16 integers: c for symmetric codes, u - 8 for
// affine ones, (c0, c4), (c1, c5), (c2, c6), (c3, c7).
template <bool AFF>
__device__ __forceinline__ void code_pairs(uint32_t d, half2_t out[4]) {
  if constexpr (AFF) codes_to_half_spread_zp(d, out, zp_bias_lo(8), zp_bias_hi(8));
  else codes_to_half_spread(d, out);
}

// A lane's row of 16 lanes holds one value a token of its 16-token unit: that of
// token `n`, in every lane of the row (folded into the instruction that uses it).
template <int n>
__device__ __forceinline__ float of_token(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x150 + n, 0xF, 0xF, true));
}

// Token (of a 16-token unit) of score i = 4 n + r in a lane.
constexpr int token_of(int i) { return (i & ~3) | ((i & 1) << 1) | ((i >> 1) & 1); }

// Calls f(integral_constant<int, 0>) .. f(integral_constant<int, N - 1>).
template <int N, typename F, int... I>
__device__ __forceinline__ void each_of(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F f) {
  each_of<N>(f, std::make_integer_sequence<int, N>{});
}

// The largest over the lanes of a row of 16.
__device__ __forceinline__ uint32_t row_umax(uint32_t v) {
  auto step = [&](auto ctrl) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, 0xF, 0xF, true);
    v = v > o ? v : o;
  };
  step(std::integral_constant<int, 0xB1>{});    // lanes 0 1 | 2 3 exchanged
  step(std::integral_constant<int, 0x4E>{});    // pairs exchanged
  step(std::integral_constant<int, 0x141>{});   // halves of 8 mirrored
  step(std::integral_constant<int, 0x140>{});   // row mirrored
  return v;
}

// Element e of 8 binary16 or bfloat16 patterns.
__device__ __forceinline__ float query_value(const Words<4>& r, int e, int bf16) {
  const uint32_t h = e & 1 ? r.w[e / 2] >> 16 : r.w[e / 2] & 0xFFFFu;
  return bf16 ? __builtin_bit_cast(float, h << 16) : half_bits_to_float((uint16_t)h);
}

// Two outputs as binary16 or bfloat16 patterns, rounded to nearest even.
__device__ __forceinline__ uint32_t output_pair(float x, float y, int bf16) {
  if (bf16) {
    const bf16x2_t v = {(__bf16)x, (__bf16)y};
    return __builtin_bit_cast(uint32_t, v);
  }
  const half2_t v = {(_Float16)x, (_Float16)y};
  return __builtin_bit_cast(uint32_t, v);
}

// Channels d0 .. d0 + N - 1 of one output row (N 4 or 8), those below D.
template <int N>
__device__ __forceinline__ void store_output(const AttentionArgs& a, int64_t row, int d0, const float* v) {
  uint16_t* const p = static_cast<uint16_t*>(a.out) + row * a.c.D + d0;
  Words<N / 2> w;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) w.w[i] = output_pair(v[2 * i], v[2 * i + 1], a.bf16);
  if (a.c.D % 8 == 0 && ((uintptr_t)a.out & 15) == 0) {
    if (d0 >= a.c.D) return;
    if constexpr (N == 4) *reinterpret_cast<u32x2_t*>(p) = u32x2_t{w.w[0], w.w[1]};
    else *reinterpret_cast<u32x4_t*>(p) = u32x4_t{w.w[0], w.w[1], w.w[2], w.w[3]};
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (d0 + i < a.c.D) p[i] = (uint16_t)(w.w[i / 2] >> (16 * (i & 1)));
  }
}

__device__ __forceinline__ float lse_of(float m, float sum) {
  return sum == 0.0f ? -__builtin_inff() : 0.69314718055994530942f * (m + __builtin_amdgcn_logf(sum));
}

// ---------------------------------------------------------------- where a step's codes lie

// The 16-token units of the cache that hold the four of a step (0 where there is
// no page; bit u of `found` tells).
struct Units {
  int at[4];
  uint32_t found;
};
struct Pages {
  int p[4];
};

// Page numbers come through scalar loads, ahead of their use: as vector loads they
// would make the wait for them a wait for every load before them.
struct PageTable {
  typedef const int32_t __attribute__((address_space(4))) * ScalarPtr;
  ScalarPtr table;
  int shift, last, slots, page_units, head_unit, pages;

  __device__ __forceinline__ PageTable(const AttentionArgs& a, int b, int kh)
      : table((ScalarPtr)(uintptr_t)(a.r.table + (int64_t)b * a.r.table_stride)), shift(a.c.page_shift),
        last((int)a.r.max_pages - 1), slots((1 << a.c.page_shift) - 1), page_units(a.c.heads << (a.c.page_shift - 4)),
        head_unit(kh << (a.c.page_shift - 4)), pages((int)a.c.pages) {}

  __device__ __forceinline__ Pages pages_of(int step) const {
    Pages r;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int index = (int)(unit_token(step, u) >> shift);
      r.p[u] = table[index < last ? index : last];
    }
    return r;
  }
  __device__ __forceinline__ Units units_of(int step, const Pages& x) const {
    Units r;
    r.found = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool ok = (uint32_t)x.p[u] < (uint32_t)pages;
      r.at[u] = ok ? x.p[u] * page_units + head_unit + (int)((unit_token(step, u) & (uint32_t)slots) >> 4) : 0;
      r.found |= ok ? 1u << u : 0u;
    }
    return r;
  }
};

__device__ __forceinline__ int pick(const Units& x, int u) {
  const int a0 = x.at[0], a1 = x.at[1], a2 = x.at[2], a3 = x.at[3];      // values: no address is selected
  const int low = u & 1 ? a1 : a0, high = u & 1 ? a3 : a2;
  return u & 2 ? high : low;
}

// Token of its unit, within 4, whose key row a lane of `row` takes.
__device__ __forceinline__ int key_token(int row) { return (row & 3) == 1 ? 2 : (row & 3) == 2 ? 1 : (row & 3); }

// Scales and zero points of a step as a lane holds them: of token `row` of the
// unit `quarter`, and for the values' zero points of all its tokens.
template <int NG, bool AFF>
struct StepScales {
  // 32-bit registers, as the loads leave them: a narrower type would be masked as
  // soon as it arrives, and that be a wait for the load where it was issued.
  uint32_t k[NG], v[NG];
  uint32_t kz[AFF ? NG : 1];
  Words<4> vz[AFF ? NG : 1];
};

// ---------------------------------------------------------------- a wavefront's rows

// 16 QT query rows of one key/value head: lane (row, quarter) holds query row `row`
// of each tile of 16, and of a step the scores of the tokens of unit `quarter`.
template <int C, int GC, int QT, bool AFF>
struct Rows {
  static constexpr int NG = C / GC;
  int row, quarter;
  int flat0, flats;                      // the first flat row, and the sequence's number of them
  int lo[QT], hi[QT];                    // visible keys
  half8_t q[QT][C];
  float factor[QT], qsum[QT][AFF ? NG : 1];          // factor: a power of two
  static constexpr float kFar = 0x1p22f;
  float4_t acc[QT][2 * C];               // [.][2 j]: channels of the low nibbles of byte rows 16 j .., [2 j + 1]: high
  float m[QT], l[QT], zsum[QT][AFF ? NG : 1];
  float s[QT][16];                       // scores, then probabilities: tokens token_of(0) .. token_of(15)
  int group_of[NG];

  // Query loads only; a row that the tile does not have reads the sequence's last.
  __device__ __forceinline__ void load(const AttentionArgs& a, const SequenceWork& w, int kh, Words<4> raw[QT][C]) {
    const uint32_t ratio = (uint32_t)a.ratio;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int x = NG == 1 ? 0 : g * GC * 32 / a.c.group;
      group_of[g] = x < a.c.G ? x : a.c.G - 1;
    }
    const uint16_t* at[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      const int flat = flat0 + 16 * t + row;
      const uint32_t f = flat < flats ? flat : flats - 1, token = f / ratio;
      visible(a, w, token, &lo[t], &hi[t]);
      if (flat >= flats) lo[t] = hi[t] = 0;
      at[t] = static_cast<const uint16_t*>(a.q) + (int64_t)(w.first + token) * a.q_row_stride +
              (int64_t)(kh * ratio + f % ratio) * a.q_head_stride;
    }
    if (a.q_wide) {
#pragma unroll
      for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int i = 0; i < C; ++i) {
          const int d = 32 * i + 8 * quarter;
          raw[t][i] = load_words<4>(reinterpret_cast<const uint8_t*>(at[t] + (d < a.c.D ? d : 0)));
        }
    } else {
#pragma unroll
      for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int d = 32 * i + 8 * quarter + 2 * e, last = a.c.D - 1;
            raw[t][i].w[e] = at[t][d < last ? d : last] | (uint32_t)at[t][d + 1 < last ? d + 1 : last] << 16;
          }
    }
  }

  // The operand, the factor of the scores and the sums for affine codes.
  __device__ __forceinline__ void start(const AttentionArgs& a, Words<4> raw[QT][C]) {
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      // the largest magnitude: its pattern orders like an unsigned number
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // channels from head_dim on, and rows that the tile does not have, are 0
          const int have = flat0 + 16 * t + row < flats ? a.c.D - 32 * i - 8 * quarter - 2 * e : 0;
          const uint32_t x = raw[t][i].w[e] & (have >= 2 ? 0xFFFFFFFFu : have == 1 ? 0xFFFFu : 0u);
          raw[t][i].w[e] = x;
          const uint32_t low = x & 0x7FFFu, high = (x >> 16) & 0x7FFFu;
          top = low > top ? low : top;
          top = high > top ? high : top;
        }
      const Words<4> one = {{top, 0, 0, 0}};
      const float most = rows_max(query_value(one, 0, a.bf16));
      // most * 2^up in [2^13, 2^14)
      const int e = (int)(__builtin_bit_cast(uint32_t, most) >> 23) - 127;
      const int up = most > 0.0f ? (e > 110 ? -97 : 13 - e) : 0;
      // neither 0 nor infinite, which a hidden score or a score of 0 would turn to NaN: at
      // 2^-126 and below scores, less than 2^43 here, are 0 to the last bit of their softmax
      const int x = a.scale_exp - up;
      factor[t] = __builtin_ldexpf(1.0f, x < -126 ? -126 : x > 127 ? 127 : x);
#pragma unroll
      for (int g = 0; g < (AFF ? NG : 1); ++g) qsum[t][g] = 0.0f;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        _Float16 h[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          h[n] = (_Float16)__builtin_ldexpf(query_value(raw[t][i], n, a.bf16), up);
          if constexpr (AFF) qsum[t][i / GC] += (float)h[n];
        }
        q[t][i] = half8_t{h[0], h[4], h[1], h[5], h[2], h[6], h[3], h[7]};
      }
#pragma unroll
      for (int g = 0; g < (AFF ? NG : 0); ++g) qsum[t][g] = rows_sum(qsum[t][g]);
      m[t] = -1e30f;
      l[t] = 0.0f;
#pragma unroll
      for (int g = 0; g < (AFF ? NG : 1); ++g) zsum[t][g] = 0.0f;
#pragma unroll
      for (int j = 0; j < 2 * C; ++j) acc[t][j] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
  }

  // Scores of key tile n from its operand (a block of 32 channels each).
  template <int n>
  __device__ __forceinline__ void score(const half8_t k[C], const StepScales<NG, AFF>& x, float part) {
#pragma unroll
    for (int t = 0; t < QT; ++t) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float ks = half_bits_to_float((uint16_t)x.k[g]) * part;
        float4_t dot = {0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (AFF) {               // (8 - z) sum q
          const float z = 8.0f - (float)x.kz[g];
          each<4>([&](auto ii) {
            constexpr int i = decltype(ii)::value;
            dot[i] = qsum[t][g] * of_token<token_of(4 * n + i)>(z);
          });
        }
#pragma unroll
        for (int i = g * GC; i < (g + 1) * GC; ++i)
          dot = __builtin_amdgcn_mfma_f32_16x16x32_f16(k[i], q[t][i], dot, 0, 0, 0);
        each<4>([&](auto ii) {
          constexpr int i = decltype(ii)::value;
          const float y = dot[i] * of_token<token_of(4 * n + i)>(ks);
          s[t][4 * n + i] = g == 0 ? y : s[t][4 * n + i] + y;
        });
      }
    }
  }

  // Hides the step's tokens that a row does not see. Scales of tokens that the
  // sequence does not have (their memory may hold anything) become 0.
  __device__ __forceinline__ void hide(int step, uint32_t found, int keys, uint32_t vs[NG]) {
    const int token0 = step * kStep + 16 * quarter;
    const bool there = (found >> quarter) & 1u;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      const int from = lo[t] - token0, to = there ? hi[t] - token0 : -1;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (token_of(i) < from || token_of(i) >= to) s[t][i] = -__builtin_inff();
    }
    const int have = there ? keys - token0 : 0;
#pragma unroll
    for (int g = 0; g < NG; ++g)
      if (row >= have) vs[g] = 0;
  }

  // The exponent of the largest scale of a lane's token, of either sign, for reach.
  static __device__ __forceinline__ uint32_t scale_binade(const uint32_t vs[NG]) {
    uint32_t big = vs[0] & 0x7FFFu;
#pragma unroll
    for (int g = 1; g < NG; ++g) big = (vs[g] & 0x7FFFu) > big ? vs[g] & 0x7FFFu : big;
    return big >> 10;
  }
  static __device__ __forceinline__ float binades(uint32_t e) { return (float)((int)e - 14 - 9 - 6); }

  // What the reference has to reach for a lane's tokens, less 6: the largest score
  // plus the exponent of the largest scale, an upper bound of log2 of every weight,
  // less 9; or far from zero the largest score, an upper bound of log2 of every
  // probability. Where tokens are hidden (each_token) each score goes with its own
  // token's scale: one that a row does not see must not take bits from what it sees.
  template <bool each_token>
  __device__ __forceinline__ void reach(const uint32_t vs[NG], float cand[QT]) const {
    const uint32_t e = scale_binade(vs);
    const float own = binades(e), spread = binades(row_umax(e));
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      float top = s[t][0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = __builtin_fmaxf(top, s[t][i]);
      top *= factor[t];
      float near = top + spread;
      if constexpr (each_token) {
        near = -__builtin_inff();
        each<16>([&](auto ii) {
          constexpr int i = decltype(ii)::value;
          near = __builtin_fmaxf(near, s[t][i] * factor[t] + of_token<token_of(i)>(own));
        });
      }
      cand[t] = __builtin_fabsf(top) > kFar ? top : near;
    }
  }

  // Moves the running reference where it has to and turns the scores into
  // probabilities; cand: of reach.
  __device__ __forceinline__ void settle(float cand[QT]) {
    bool move = false;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      cand[t] = rows_max(cand[t]);
      move |= cand[t] > m[t];
    }
    if (__ballot(move) != 0) {
#pragma unroll
      for (int t = 0; t < QT; ++t) {
        const float to = __builtin_fmaxf(m[t], __builtin_fabsf(cand[t]) > kFar ? cand[t] : cand[t] + 6.0f);
        const float shrink = __builtin_amdgcn_exp2f(m[t] - to);
        m[t] = to;
        l[t] *= shrink;
#pragma unroll
        for (int g = 0; g < (AFF ? NG : 0); ++g) zsum[t][g] *= shrink;
#pragma unroll
        for (int j = 0; j < 2 * C; ++j) acc[t][j] *= shrink;
      }
    }
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[t][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][i], factor[t], -m[t]));
        l[t] += s[t][i];
      }
  }

  // The weights of group g, probability times scale in binary16, as the operand of
  // the product with the values: tokens 0 .. 7 of the unit, then 8 .. 15.
  __device__ __forceinline__ void weights(int g, bool masked, uint32_t scale, const StepScales<NG, AFF>& x, half8_t w[QT][2]) {
    const float vs = half_bits_to_float((uint16_t)scale);
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      half2_t pair[8];
      if (!masked) {
        each<8>([&](auto ii) {
          constexpr int i = 2 * decltype(ii)::value;
          pair[i / 2] = half2_t{(_Float16)(s[t][i] * of_token<token_of(i)>(vs)),
                                (_Float16)(s[t][i + 1] * of_token<token_of(i + 1)>(vs))};
        });
      } else {                             // a hidden token's scale may be infinite or NaN
        each<8>([&](auto ii) {
          constexpr int i = 2 * decltype(ii)::value;
          const float y0 = s[t][i] * of_token<token_of(i)>(vs), y1 = s[t][i + 1] * of_token<token_of(i + 1)>(vs);
          pair[i / 2] = half2_t{(_Float16)(s[t][i] == 0.0f ? 0.0f : y0), (_Float16)(s[t][i + 1] == 0.0f ? 0.0f : y1)};
        });
      }
      if constexpr (AFF) {
        const half2_t off = {(_Float16)-1032.0f, (_Float16)-1032.0f};
#pragma unroll
        for (int i = 0; i < 8; ++i) {      // 1024 + z, then z - 8
          const uint32_t zw = x.vz[g].w[i / 2];
          const uint32_t z = ((i & 1 ? zw >> 8 : zw) & 0x00FF00FFu) | 0x64006400u;
          zsum[t][g] = __builtin_amdgcn_fdot2(pair[i], __builtin_bit_cast(half2_t, z) + off, zsum[t][g], false);
        }
      }
      w[t][0] = as_half8(pair);
      w[t][1] = as_half8(pair + 4);
    }
  }

  // Adds the products of byte rows 16 j .. of the values, tokens 8 u .. of each unit.
  __device__ __forceinline__ void add(int j, half8_t even, half8_t odd, const half8_t w[QT][2], int u) {
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      acc[t][2 * j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(even, w[t][u], acc[t][2 * j], 0, 0, 0);
      acc[t][2 * j + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(odd, w[t][u], acc[t][2 * j + 1], 0, 0, 0);
    }
  }

  // The lane's sums over its row's four lanes; then result() gives the channels
  // 32 j + 8 quarter .. + 7 of its row.
  __device__ __forceinline__ void finish(int t) {
    l[t] = rows_sum(l[t]);
#pragma unroll
    for (int g = 0; g < (AFF ? NG : 0); ++g) zsum[t][g] = rows_sum(zsum[t][g]);
  }
  __device__ __forceinline__ void result(int t, int j, float factor_, float v[8]) const {
    const float z = AFF ? zsum[t][AFF ? j / GC : 0] : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = (acc[t][2 * j][i] - z) * factor_;
      v[2 * i + 1] = (acc[t][2 * j + 1][i] - z) * factor_;
    }
  }
};

// Value operands of two words (two channels of eight tokens) each.
template <bool AFF>
__device__ __forceinline__ void value_operands(uint32_t w0, uint32_t w1, half8_t* even, half8_t* odd) {
  half2_t c[8];
  code_pairs<AFF>(w0, c);
  code_pairs<AFF>(w1, c + 4);
  const half2_t lows[4] = {c[0], c[2], c[4], c[6]}, highs[4] = {c[1], c[3], c[5], c[7]};
  *even = as_half8(lows);
  *odd = as_half8(highs);
}

template <int C, bool AFF>
__device__ __forceinline__ void key_operands(const Words<C>& w, half8_t k[C]) {
#pragma unroll
  for (int i = 0; i < C; ++i) {
    half2_t c[4];
    code_pairs<AFF>(w.w[i], c);
    k[i] = as_half8(c);
  }
}

template <int NG, bool AFF>
__device__ __forceinline__ void load_key_scales(const CacheView& c, int unit, int row, const int group_of[NG],
                                                StepScales<NG, AFF>* x) {
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int64_t at = ((int64_t)unit * c.G + group_of[g]) * 16;
    x->k[g] = c.k_scales[at + row];
    if constexpr (AFF) x->kz[g] = c.k_zeros[at + row];
  }
}
template <int NG, bool AFF>
__device__ __forceinline__ void load_value_scales(const CacheView& c, int unit, int row, const int group_of[NG],
                                                  StepScales<NG, AFF>* x) {
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int64_t at = ((int64_t)unit * c.G + group_of[g]) * 16;
    x->v[g] = c.v_scales[at + row];
    if constexpr (AFF) x->vz[g] = load_words<4>(c.v_zeros + at);
  }
}

// What a block does first: its share, the record of a partial result, the number
// of them. False if it has no share.
__device__ __forceinline__ bool begin_block(const AttentionArgs& a, const Schedule& sched, const Workspace& ws,
                                            BlockWork* work) {
  const int heads = a.c.heads;
  int used;
  const bool found = find_block(a, sched, ws, blockIdx.x / heads, work, &used);
  if (sched.target > 0 && !sched.planned && blockIdx.x == 0 && threadIdx.x == 0) *ws.used = used;
  if (!found) return false;
  if (work->chunks > 1 && blockIdx.x % heads == 0 && threadIdx.x == 0)
    ws.record[work->slot] = PartRecord{work->w.first, work->tile * sched.tile_rows, work->w.rows * a.ratio, work->chunk,
                                       work->chunks, {}};
  return true;
}

// Visible keys of flat rows [flat0, flat0 + n) that the sequence has: of the first
// row and of the last.
struct Span {
  int lo_first, hi_first, lo_last, hi_last;
  __device__ __forceinline__ Span(const AttentionArgs& a, const SequenceWork& w, int flat0, int n) {
    const int flats = w.rows * a.ratio;
    visible(a, w, (uint32_t)flat0 / (uint32_t)a.ratio, &lo_first, &hi_first);
    visible(a, w, (uint32_t)((flat0 + n < flats ? flat0 + n : flats) - 1) / (uint32_t)a.ratio, &lo_last, &hi_last);
  }
  __device__ __forceinline__ bool masks(int step) const { return step_masked(step, lo_last, hi_first); }
};

// ---------------------------------------------------------------- few rows

// C blocks of 32 channels, GC of them to a scale (scale_blocks), QT tiles of 16
// query rows. The block's four wavefronts take turns on the steps; their results
// are joined through LDS.
template <int C, int GC, int QT, bool AFF>
__global__ __launch_bounds__(256, resident_blocks(C, C / GC, AFF, 16 * QT)) void cache_attention_kernel(
    AttentionArgs a, Schedule sched, Workspace ws) {
  constexpr int NG = C / GC, DB = 16 * C, TR = 16 * QT;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);     // known to be uniform
  const int heads = a.c.heads, kh = blockIdx.x % heads;
  BlockWork work;
  if (!begin_block(a, sched, ws, &work)) return;
  Rows<C, GC, QT, AFF> r;
  r.row = lane & 15;
  r.quarter = lane >> 4;
  r.flat0 = work.tile * TR;
  r.flats = work.w.rows * a.ratio;
  const Span span(a, work.w, r.flat0, TR);
  int begin, end;
  chunk_steps(span.lo_first, span.hi_last, work.chunk, work.chunks, &begin, &end);
  Words<4> raw[QT][C];
  r.load(a, work.w, kh, raw);

  // A lane's key rows lie in the 16-token unit row / 4 of the step, its values and
  // scales in unit `quarter`.
  const PageTable table(a, work.b, kh);
  const int key_off = key_token(r.row) * DB + r.quarter * 4 * C;
  Words<C> kw[4];
  Words<4> vw[C];
  StepScales<NG, AFF> sc;
  auto load_keys = [&](const Units& x) {
    const uint8_t* const p = a.c.k_packed + (int64_t)pick(x, r.row >> 2) * (16 * DB) + key_off;
#pragma unroll
    for (int n = 0; n < 4; ++n) kw[n] = load_words<C>(p + n * 4 * DB);
    load_key_scales(a.c, pick(x, r.quarter), r.row, r.group_of, &sc);
  };
  auto load_values = [&](const Units& x) {
    const int vu = pick(x, r.quarter);
    const uint8_t* const p = a.c.v_packed + (int64_t)vu * (16 * DB) + r.row * 16;
#pragma unroll
    for (int j = 0; j < C; ++j) vw[j] = load_words<4>(p + j * 256);
    load_value_scales(a.c, vu, r.row, r.group_of, &sc);
  };
  int step = begin + wave;
  Units units{};
  Pages pages{};
  if (step < end) {
    units = table.units_of(step, table.pages_of(step));
    pages = table.pages_of(step + 4);
    load_keys(units);
    load_values(units);
  }
  r.start(a, raw);

  for (; step < end; step += 4) {
    // The loads for the next step are always issued, after the last one for this step
    // again (out of the L2): behind a branch, every wait would have to assume the
    // fewest loads in flight, and wait for the newest.
    const int next = step + 4 < end ? step + 4 : step;
    const uint32_t found = units.found;
    if (next > step) units = table.units_of(next, pages);
    pages = table.pages_of(next + 4);
    each<4>([&](auto nn) {
      constexpr int n = decltype(nn)::value;
      half8_t k[C];
      key_operands<C, AFF>(kw[n], k);
      r.template score<n>(k, sc, a.scale_part);
      // no instruction, but an order: this tile's scores are finished before the
      // next one's codes are taken apart, which keeps the live registers few
#pragma unroll
      for (int t = 0; t < QT; ++t)
        asm volatile("" : "+v"(r.s[t][4 * n]), "+v"(r.s[t][4 * n + 1]), "+v"(r.s[t][4 * n + 2]), "+v"(r.s[t][4 * n + 3]));
      if constexpr (n < 3) {
#pragma unroll
        for (int i = 0; i < C; ++i) asm volatile("" : "+v"(kw[n + 1].w[i]));
      }
    });
    load_keys(units);
    const bool masked = span.masks(step) || found != 15u;
    // a copy: changed in place, the scales would have to be moved where they arrive
    uint32_t vs[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) vs[g] = sc.v[g];
    float cand[QT];
    if (masked) {
      r.hide(step, found, work.w.keys, vs);
      r.template reach<true>(vs, cand);
    } else {
      r.template reach<false>(vs, cand);
    }
    r.settle(cand);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      half8_t w[QT][2];
      r.weights(g, masked, vs[g], sc, w);
#pragma unroll
      for (int j = g * GC; j < (g + 1) * GC; ++j) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          half8_t even, odd;
          value_operands<AFF>(vw[j].w[2 * u], vw[j].w[2 * u + 1], &even, &odd);
          r.add(j, even, odd, w, u);
        }
        if (j + 1 < C) {
#pragma unroll
          for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(vw[j + 1].w[i]) : "v"(r.acc[QT - 1][2 * j + 1]));
        }
      }
    }
    load_values(units);
  }

  // --- join the wavefronts, 16 rows at a time
  __shared__ float ml[2][4][16];
  __shared__ __attribute__((aligned(16))) float rows_out[4][16][32 * C + 4];
  const int tid = threadIdx.x, orow = tid >> 4;
  const uint32_t ratio = (uint32_t)a.ratio;
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    r.finish(t);
    if (r.quarter == 0) {
      ml[0][wave][r.row] = r.m[t];
      ml[1][wave][r.row] = r.l[t];
    }
    __syncthreads();
    const float top = __builtin_fmaxf(__builtin_fmaxf(ml[0][0][r.row], ml[0][1][r.row]),
                                      __builtin_fmaxf(ml[0][2][r.row], ml[0][3][r.row]));
    const float shrink = __builtin_amdgcn_exp2f(r.m[t] - top);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      float v[8];
      r.result(t, j, shrink, v);
      float4_t* const to = reinterpret_cast<float4_t*>(&rows_out[wave][r.row][32 * j + 8 * r.quarter]);
      to[0] = float4_t{v[0], v[1], v[2], v[3]};
      to[1] = float4_t{v[4], v[5], v[6], v[7]};
    }
    __syncthreads();
    const int flat = r.flat0 + 16 * t + orow;
    if (flat < r.flats) {
      float mm = ml[0][0][orow];
#pragma unroll
      for (int i = 1; i < 4; ++i) mm = __builtin_fmaxf(mm, ml[0][i][orow]);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += ml[1][i][orow] * __builtin_amdgcn_exp2f(ml[0][i][orow] - mm);
      const bool whole = work.chunks == 1;
      const float inv = whole ? (sum == 0.0f ? 0.0f : 1.0f / sum) : 1.0f;
      const int64_t at = (int64_t)(work.w.first + (uint32_t)flat / ratio) * heads * ratio + kh * ratio + (uint32_t)flat % ratio;
      float* const slot = ws.part + ((int64_t)work.slot * heads + kh) * partial_floats(TR, C);
      for (int d = (tid & 15) * 4; d < 32 * C; d += 64) {
        float4_t v = *reinterpret_cast<const float4_t*>(&rows_out[0][orow][d]);
#pragma unroll
        for (int i = 1; i < 4; ++i) v += *reinterpret_cast<const float4_t*>(&rows_out[i][orow][d]);
        v *= inv;
        const float o[4] = {v.x, v.y, v.z, v.w};
        if (whole) store_output<4>(a, at, d, o);
        else *reinterpret_cast<float4_t*>(slot + (16 * t + orow) * (32 * C) + d) = v;
      }
      if ((tid & 15) == 0) {
        if (!whole) {
          slot[TR * 32 * C + 2 * (16 * t + orow)] = mm;
          slot[TR * 32 * C + 2 * (16 * t + orow) + 1] = sum;
        } else if (a.lse) {
          a.lse[at] = lse_of(mm, sum);
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- many rows

// The form for prompts: each of the block's wavefronts has 16 QT rows of its own
// (128 in all: four wavefronts of 32 rows, or eight of 16 where the registers do
// not hold more) and all take the same steps. The codes of a step are taken apart
// once a block: each wavefront turns its share of them into operands and leaves
// those in LDS, in the lanes' order, for all, one step ahead of their use (two
// buffers, one barrier a step).
template <int C, int GC, int QT, bool AFF>
__global__ __launch_bounds__(512 / QT) void cache_attention_wide_kernel(AttentionArgs a, Schedule sched, Workspace ws) {
  constexpr int NG = C / GC, DB = 16 * C, TR = kWideRows;
  constexpr int VJ = (C + 3) / 4;        // byte rows (of 16) of the values that a wavefront prepares
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);     // known to be uniform
  const int heads = a.c.heads, kh = blockIdx.x % heads;
  BlockWork work;
  if (!begin_block(a, sched, ws, &work)) return;
  Rows<C, GC, QT, AFF> r;
  r.row = lane & 15;
  r.quarter = lane >> 4;
  r.flat0 = work.tile * TR + wave * 16 * QT;
  r.flats = work.w.rows * a.ratio;
  const bool rows_here = r.flat0 < r.flats;
  const Span all(a, work.w, work.tile * TR, TR);
  const Span span(a, work.w, rows_here ? r.flat0 : work.tile * TR, 16 * QT);
  int begin, end;
  chunk_steps(all.lo_first, all.hi_last, work.chunk, work.chunks, &begin, &end);
  // the steps of which this wavefront's rows see something
  const int first = span.lo_first / kStep, last = rows_here && span.hi_last > span.lo_first ? (span.hi_last - 1) / kStep : -1;
  Words<4> raw[QT][C];
  r.load(a, work.w, kh, raw);

  const PageTable table(a, work.b, kh);
  // The shares: one key tile and one in four of the values' byte rows for each of
  // four wavefronts, or either for each of eight.
  const bool does_keys = QT == 2 || wave < 4, does_values = QT == 2 || wave >= 4;
  const int share = wave & 3;
  const int key_off = key_token(r.row) * DB + share * 4 * DB + r.quarter * 4 * C;
  __shared__ __attribute__((aligned(16))) u32x4_t keys[2][4 * C][kWave];            // [4 tiles][C]
  __shared__ __attribute__((aligned(16))) u32x4_t values[2][4 * C][kWave];          // [C][2 halves][even, odd]
  Words<C> kw;
  Words<4> vw[VJ];
  StepScales<NG, AFF> sc, sc_next;
  auto load = [&](const Units& x) {
    const int vu = pick(x, r.quarter);
    if (does_keys) kw = load_words<C>(a.c.k_packed + (int64_t)pick(x, r.row >> 2) * (16 * DB) + key_off);
    if (does_values) {
      const uint8_t* const p = a.c.v_packed + (int64_t)vu * (16 * DB) + r.row * 16;
#pragma unroll
      for (int i = 0; i < VJ; ++i) {
        const int j = share + 4 * i;
        vw[i] = load_words<4>(p + (j < C ? j : C - 1) * 256);
      }
    }
    load_key_scales(a.c, vu, r.row, r.group_of, &sc_next);
    load_value_scales(a.c, vu, r.row, r.group_of, &sc_next);
  };
  auto prepare = [&](int buffer) {
    if (does_keys) {
      half8_t k[C];
      key_operands<C, AFF>(kw, k);
#pragma unroll
      for (int i = 0; i < C; ++i) keys[buffer][share * C + i][lane] = __builtin_bit_cast(u32x4_t, k[i]);
    }
#pragma unroll
    for (int i = 0; i < VJ; ++i) {
      const int j = share + 4 * i;
      if (does_values && j < C) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          half8_t even, odd;
          value_operands<AFF>(vw[i].w[2 * u], vw[i].w[2 * u + 1], &even, &odd);
          values[buffer][4 * j + 2 * u][lane] = __builtin_bit_cast(u32x4_t, even);
          values[buffer][4 * j + 2 * u + 1][lane] = __builtin_bit_cast(u32x4_t, odd);
        }
      }
    }
  };

  int step = begin;
  Units units{};
  Pages pages{};
  uint32_t found = 0, found_next = 0;
  if (step < end) {
    units = table.units_of(step, table.pages_of(step));
    pages = table.pages_of(step + 1);
    found = units.found;
    load(units);
  }
  r.start(a, raw);
  if (step < end) {
    prepare(0);
    sc = sc_next;
    if (step + 1 < end) units = table.units_of(step + 1, pages);
    pages = table.pages_of(step + 2);
    found_next = units.found;
    load(units);
    lds_barrier();
  }
#pragma unroll 1
  for (int buffer = 0; step < end; ++step, buffer ^= 1) {
    if (step >= first && step <= last) {
      // Operands are read from LDS one tile of keys, or one byte row of values, ahead
      // of the products that take them; the empty statements keep that order.
      half8_t k[2][C], v[2][4];
      auto read_keys = [&](int n, half8_t* to) {
#pragma unroll
        for (int i = 0; i < C; ++i) to[i] = __builtin_bit_cast(half8_t, keys[buffer][n * C + i][lane]);
        asm volatile("" ::: "memory");
      };
      auto read_values = [&](int j, half8_t* to) {
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = __builtin_bit_cast(half8_t, values[buffer][4 * j + i][lane]);
        asm volatile("" ::: "memory");
      };
      read_keys(0, k[0]);
      __builtin_amdgcn_s_setprio(1);
      each<4>([&](auto nn) {
        constexpr int n = decltype(nn)::value;
        if constexpr (n < 3) read_keys(n + 1, k[(n + 1) & 1]);
        r.template score<n>(k[n & 1], sc, a.scale_part);
      });
      __builtin_amdgcn_s_setprio(0);
      read_values(0, v[0]);
      const bool masked = span.masks(step) || found != 15u;
      uint32_t vs[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) vs[g] = sc.v[g];
      float cand[QT];
      if (masked) {
        r.hide(step, found, work.w.keys, vs);
        r.template reach<true>(vs, cand);
      } else {
        r.template reach<false>(vs, cand);
      }
      r.settle(cand);
      each<NG>([&](auto gg) {
        constexpr int g = decltype(gg)::value;
        half8_t w[QT][2];
        r.weights(g, masked, vs[g], sc, w);
        each<GC>([&](auto jj) {
          constexpr int j = g * GC + decltype(jj)::value;
          if constexpr (j + 1 < C) read_values(j + 1, v[(j + 1) & 1]);
          __builtin_amdgcn_s_setprio(1);
          r.add(j, v[j & 1][0], v[j & 1][1], w, 0);
          r.add(j, v[j & 1][2], v[j & 1][3], w, 1);
          __builtin_amdgcn_s_setprio(0);
        });
      });
    }
    // (at the end the last step's loads and operands once more, for no one: see the
    // loads of the form for few rows)
    prepare(buffer ^ 1);                 // last read in the step before, which all have left
    sc = sc_next;
    found = found_next;
    if (step + 2 < end) units = table.units_of(step + 2, pages);
    pages = table.pages_of(step + 3);
    found_next = units.found;
    load(units);
    lds_barrier();
  }

  if (!rows_here) return;
  const uint32_t ratio = (uint32_t)a.ratio;
  const bool whole = work.chunks == 1;
  float* const slot = ws.part + ((int64_t)work.slot * heads + kh) * partial_floats(TR, C);
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    r.finish(t);
    const int flat = r.flat0 + 16 * t + r.row;
    if (flat >= r.flats) continue;
    const int64_t at = (int64_t)(work.w.first + (uint32_t)flat / ratio) * heads * ratio + kh * ratio + (uint32_t)flat % ratio;
    const float inv = whole ? (r.l[t] == 0.0f ? 0.0f : 1.0f / r.l[t]) : 1.0f;
    const int in_tile = wave * 16 * QT + 16 * t + r.row;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      float v[8];
      r.result(t, j, inv, v);
      const int d = 32 * j + 8 * r.quarter;
      if (whole) {
        store_output<8>(a, at, d, v);
      } else {
        float4_t* const to = reinterpret_cast<float4_t*>(slot + (int64_t)in_tile * (32 * C) + d);
        to[0] = float4_t{v[0], v[1], v[2], v[3]};
        to[1] = float4_t{v[4], v[5], v[6], v[7]};
      }
    }
    if (r.quarter == 0) {
      if (!whole) {
        slot[TR * 32 * C + 2 * in_tile] = r.m[t];
        slot[TR * 32 * C + 2 * in_tile + 1] = r.l[t];
      } else if (a.lse) {
        a.lse[at] = lse_of(r.m[t], r.l[t]);
      }
    }
  }
}

// Defined for each width in a file of its own: launches the form for the cache's
// groups and the schedule's tile height.
template <int C>
hipError_t launch_attention_width(const AttentionArgs& a, const Schedule& s, const Workspace& ws, hipStream_t stream);

}  // namespace int4dq
