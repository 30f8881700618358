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
//   values: w_j = p_j s'_jg is rounded to binary16 (nearest, <= 2^-11 relative);
//     affine sums take off (z - 8) times the rounded w, so the offset cancels.
// Queries are brought to [2^13, 2^14) by a power of two per row, which is exact
// for bfloat16 and binary16 down to 2^-27 of the row's largest entry.
//
// The reference m of the running softmax is not the plain maximum: it is kept
// within 6 of max_j a_j + log2 max_j s'_j - 9 (log2 units), which keeps every
// w_j below 2^15 and the large ones far above binary16's subnormals whatever
// the values' magnitude; and it moves only when exceeded by 6, so that the
// accumulators are rescaled a few times a sequence, not every step.
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
// this one's are used; no LDS in the loop.
#pragma once

#include <type_traits>
#include <utility>

#include "cache.h"
#include "cache_schedule.h"
#include "device_common.h"

namespace int4dq {

// ---------------------------------------------------------------- wavefront sums

// Inclusive sums over the lanes: within rows of 16 by shifts, then across rows.
template <typename T>
__device__ __forceinline__ T lane_scan(T v) {
  auto add = [&](auto ctrl, auto mask) {
    const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value,
                                              decltype(mask)::value, 0xF, false);
    v += __builtin_bit_cast(T, o);
  };
  using std::integral_constant;
  add(integral_constant<int, 0x111>{}, integral_constant<int, 0xF>{});
  add(integral_constant<int, 0x112>{}, integral_constant<int, 0xF>{});
  add(integral_constant<int, 0x114>{}, integral_constant<int, 0xF>{});
  add(integral_constant<int, 0x118>{}, integral_constant<int, 0xF>{});
  add(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});
  add(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});
  return v;
}

template <typename T>
__device__ __forceinline__ T lane_value(T v, int lane) {
  return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

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

// Slots of partial results that the call uses in all.
__device__ __forceinline__ int slots_used(const AttentionArgs& a, const Schedule& s) {
  const int lane = threadIdx.x & (kWave - 1);
  float all = 0.0f;
  for (int b = lane; b < a.r.batch; b += kWave) {
    const SequenceWork x = sequence_work(a, s.tile_rows, b);
    all += (float)x.tiles * (float)x.steps;
  }
  const float each_step = blocks_per_step(s, lane_value(lane_scan(all), kWave - 1));
  int slots = 0;
  for (int b = lane; b < a.r.batch; b += kWave) {
    const SequenceWork x = sequence_work(a, s.tile_rows, b);
    const int chunks = chunks_of(x.steps, each_step);
    if (chunks > 1) slots += chunks * x.tiles;
  }
  return lane_value(lane_scan(slots), kWave - 1);
}

// The share of block `unit` of its head; every lane of the wavefront takes part.
// False if it has none.
__device__ __forceinline__ bool find_block(const AttentionArgs& a, const Schedule& s, int unit, BlockWork* out) {
  const int lane = threadIdx.x & (kWave - 1);
  float all = 0.0f;
  SequenceWork w{};
  for (int b = lane; b < a.r.batch; b += kWave) {
    const SequenceWork x = sequence_work(a, s.tile_rows, b);
    all += (float)x.tiles * (float)x.steps;
    if (b < kWave) w = x;
  }
  const float each_step = blocks_per_step(s, lane_value(lane_scan(all), kWave - 1));
  int blocks = 0, slots = 0;
  for (int b0 = 0; b0 < a.r.batch; b0 += kWave) {
    const int b = b0 + lane;
    int chunks = 0;
    if (b < a.r.batch) {
      if (b0 > 0) w = sequence_work(a, s.tile_rows, b);
      chunks = chunks_of(w.steps, each_step);
    }
    const int mine = b < a.r.batch ? chunks * w.tiles : 0, mine_slots = chunks > 1 ? mine : 0;
    const int upto = blocks + lane_scan(mine), slots_upto = slots + lane_scan(mine_slots);
    const uint64_t hit = __ballot(unit >= upto - mine && unit < upto);
    if (hit) {
      const int at = __builtin_ctzll(hit);
      out->b = b0 + at;
      out->w = SequenceWork{lane_value(w.first, at), lane_value(w.end, at), lane_value(w.rows, at),
                            lane_value(w.length, at), lane_value(w.keys, at), lane_value(w.tiles, at), 0};
      out->chunks = lane_value(chunks, at);
      const int i = unit - lane_value(upto - mine, at);
      out->chunk = i % out->chunks;
      out->tile = out->w.tiles - 1 - i / out->chunks;      // tiles that see most first
      out->slot = lane_value(slots_upto - mine_slots, at) + i;
      return true;
    }
    blocks = lane_value(upto, kWave - 1);
    slots = lane_value(slots_upto, kWave - 1);
  }
  return false;
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

__device__ __forceinline__ uint16_t output_bits(float v, int bf16) {
  if (!bf16) return __builtin_bit_cast(uint16_t, (_Float16)v);
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40u);   // NaN stays NaN
  return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

// Channels d0 .. d0+3 of one output row (those below D).
__device__ __forceinline__ void store_output(const AttentionArgs& a, int64_t row, int d0, float4_t v) {
  uint16_t* const p = static_cast<uint16_t*>(a.out) + row * a.c.D + d0;
  const uint16_t h[4] = {output_bits(v.x, a.bf16), output_bits(v.y, a.bf16), output_bits(v.z, a.bf16),
                         output_bits(v.w, a.bf16)};
  if (a.c.D % 4 == 0 && ((uintptr_t)a.out & 7) == 0) {
    if (d0 < a.c.D)
      *reinterpret_cast<u32x2_t*>(p) = u32x2_t{h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (d0 + i < a.c.D) p[i] = h[i];
  }
}

// ---------------------------------------------------------------- the kernel

// C blocks of 32 channels, GC of them to a scale (scale_blocks), QT tiles of 16
// query rows.
template <int C, int GC, int QT, bool AFF>
__global__ __launch_bounds__(256) void cache_attention_kernel(AttentionArgs a, Schedule sched, Workspace ws) {
  constexpr int NG = C / GC, DB = 16 * C, TR = 16 * QT;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);     // known to be uniform
  const int row = lane & 15, quarter = lane >> 4;
  const int heads = a.c.heads, kh = blockIdx.x % heads;
  BlockWork work;
  if (sched.target > 0 && blockIdx.x == gridDim.x - 1 && wave == 0) {
    const int used = slots_used(a, sched);
    if (lane == 0) *ws.used = used;
  }
  if (!find_block(a, sched, blockIdx.x / heads, &work)) return;
  const int flat0 = work.tile * TR, flats = work.w.rows * a.ratio;
  if (work.chunks > 1 && kh == 0 && threadIdx.x == 0)
    ws.record[work.slot] = PartRecord{work.w.first, flat0, flats, work.chunk, work.chunks, {}};

  // --- the tile's visible keys
  const uint32_t ratio = (uint32_t)a.ratio;
  int lo_first, hi_first, lo_last, hi_last;
  visible(a, work.w, (uint32_t)flat0 / ratio, &lo_first, &hi_first);
  visible(a, work.w, ((flat0 + TR < flats ? flat0 + TR : flats) - 1) / ratio, &lo_last, &hi_last);
  int begin, end;
  chunk_steps(lo_first, hi_last, work.chunk, work.chunks, &begin, &end);

  // --- queries: loads only; a row that the tile does not have reads the last one
  Words<4> raw[QT][C];
  int lo[QT], hi[QT];
  int64_t q_at[QT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const int flat = flat0 + 16 * t + row;
    const uint32_t f = flat < flats ? flat : flats - 1, token = f / ratio;
    visible(a, work.w, token, &lo[t], &hi[t]);
    if (flat >= flats) lo[t] = hi[t] = 0;
    q_at[t] = (int64_t)(work.w.first + token) * a.q_row_stride + (int64_t)(kh * ratio + f % ratio) * a.q_head_stride;
  }
  if (a.q_wide) {
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int d = 32 * i + 8 * quarter;
        raw[t][i] = load_words<4>(reinterpret_cast<const uint8_t*>(static_cast<const uint16_t*>(a.q) + q_at[t] +
                                                                   (d < a.c.D ? d : 0)));
      }
  } else {
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int d = 32 * i + 8 * quarter + 2 * e, last = a.c.D - 1;
          const uint16_t* const p = static_cast<const uint16_t*>(a.q) + q_at[t];
          raw[t][i].w[e] = p[d < last ? d : last] | (uint32_t)p[d + 1 < last ? d + 1 : last] << 16;
        }
  }

  // --- loads of a step: the lane's key rows lie in the 16-token unit row / 4 of
  // the step, its values and scales in unit `quarter`
  typedef const int32_t __attribute__((address_space(4))) * ScalarPtr;         // read by scalar loads
  const ScalarPtr table = (ScalarPtr)(uintptr_t)(a.r.table + (int64_t)work.b * a.r.table_stride);
  const int key_off = ((row & 3) == 1 ? 2 : (row & 3) == 2 ? 1 : (row & 3)) * DB + quarter * 4 * C;
  int group_of[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int x = NG == 1 ? 0 : g * GC * 32 / a.c.group;
    group_of[g] = x < a.c.G ? x : a.c.G - 1;
  }
  // The 16-token units of the cache that hold the four of a step (0 where there is
  // no page; bit u of `found` tells). Page numbers come through scalar loads, two
  // steps ahead: as vector loads they would make the wait for them a wait for
  // every load before them.
  struct Units {
    int at[4];
    uint32_t found;
  };
  struct Pages {
    int p[4];
  };
  const int page_units = heads << (a.c.page_shift - 4), head_unit = kh << (a.c.page_shift - 4);
  const int last_index = (int)a.r.max_pages - 1, slots = (1 << a.c.page_shift) - 1;
  auto pages_of = [&](int step) {
    Pages r;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int index = (step * kStep + 16 * u) >> a.c.page_shift;
      r.p[u] = table[index < last_index ? index : last_index];
    }
    return r;
  };
  auto units_of = [&](int step, const Pages& pages) {
    Units r;
    r.found = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool ok = (uint32_t)pages.p[u] < (uint32_t)a.c.pages;
      r.at[u] = ok ? pages.p[u] * page_units + head_unit + (((step * kStep + 16 * u) & slots) >> 4) : 0;
      r.found |= ok ? 1u << u : 0u;
    }
    return r;
  };
  auto pick = [&](const Units& x, int u) {
    const int a0 = x.at[0], a1 = x.at[1], a2 = x.at[2], a3 = x.at[3];      // values: no address is selected
    const int low = u & 1 ? a1 : a0, high = u & 1 ? a3 : a2;
    return u & 2 ? high : low;
  };
  Words<C> kw[4];
  Words<4> vw[C];
  uint16_t ksc[NG], vsc[NG];             // of token `row` of the quarter's unit
  uint8_t kz[AFF ? NG : 1];
  Words<4> vz[AFF ? NG : 1];             // of the unit's 16 tokens
  auto load_keys = [&](const Units& x) {
    const int ku = pick(x, row >> 2), vu = pick(x, quarter);
    const uint8_t* const p = a.c.k_packed + (int64_t)ku * (16 * DB) + key_off;
#pragma unroll
    for (int n = 0; n < 4; ++n) kw[n] = load_words<C>(p + n * 4 * DB);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int64_t at = ((int64_t)vu * a.c.G + group_of[g]) * 16;
      ksc[g] = a.c.k_scales[at + row];
      if constexpr (AFF) kz[g] = a.c.k_zeros[at + row];
    }
  };
  auto load_values = [&](const Units& x) {
    const int vu = pick(x, quarter);
    const uint8_t* const p = a.c.v_packed + (int64_t)vu * (16 * DB) + row * 16;
#pragma unroll
    for (int j = 0; j < C; ++j) vw[j] = load_words<4>(p + j * 256);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int64_t at = ((int64_t)vu * a.c.G + group_of[g]) * 16;
      vsc[g] = a.c.v_scales[at + row];
      if constexpr (AFF) vz[g] = load_words<4>(a.c.v_zeros + at);
    }
  };

  int step = begin + wave;
  Units units{};
  Pages pages{};
  if (step < end) {
    units = units_of(step, pages_of(step));
    pages = pages_of(step + 4);
    load_keys(units);
    load_values(units);
  }

  // --- queries: operand, factor of the scores, sums for affine codes
  half8_t q[QT][C];
  float factor[QT], qsum[QT][AFF ? NG : 1];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // channels from head_dim on, and rows that the tile does not have, are 0
        const int have = flat0 + 16 * t + row < flats ? a.c.D - 32 * i - 8 * quarter - 2 * e : 0;
        raw[t][i].w[e] &= have >= 2 ? 0xFFFFFFFFu : have == 1 ? 0xFFFFu : 0u;
        top = __builtin_fmaxf(top, __builtin_fabsf(query_value(raw[t][i], 2 * e, a.bf16)));
        top = __builtin_fmaxf(top, __builtin_fabsf(query_value(raw[t][i], 2 * e + 1, a.bf16)));
      }
    top = rows_max(top);
    // top * 2^up in [2^13, 2^14)
    const int e = (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127;
    const int up = top > 0.0f ? (e > 110 ? -97 : 13 - e) : 0;
    factor[t] = __builtin_ldexpf(a.scale * 1.44269504088896340736f, -up);
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
  }

  float4_t acc[QT][2 * C];               // [.][2 j]: channels of the low nibbles of byte rows 16 j .., [2 j + 1]: high
  float m[QT], l[QT], zsum[QT][AFF ? NG : 1];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    m[t] = -1e30f;
    l[t] = 0.0f;
#pragma unroll
    for (int g = 0; g < (AFF ? NG : 1); ++g) zsum[t][g] = 0.0f;
#pragma unroll
    for (int j = 0; j < 2 * C; ++j) acc[t][j] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }

  for (; step < end; step += 4) {
    const int next = step + 4;
    const uint32_t found = units.found;
    units = units_of(next, pages);
    pages = pages_of(next + 4);

    // --- scores
    float s[QT][16], ks[NG], zk[AFF ? NG : 1];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      ks[g] = half_bits_to_float(ksc[g]);
      if constexpr (AFF) zk[g] = 8.0f - (float)kz[g];
    }
    each<4>([&](auto nn) {
      constexpr int n = decltype(nn)::value;
      half8_t k[C];
#pragma unroll
      for (int i = 0; i < C; ++i) {
        half2_t c[4];
        code_pairs<AFF>(kw[n].w[i], c);
        k[i] = as_half8(c);
      }
#pragma unroll
      for (int t = 0; t < QT; ++t) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float4_t dot = {0.0f, 0.0f, 0.0f, 0.0f};
          if constexpr (AFF)               // (8 - z) sum q
            each<4>([&](auto ii) {
              constexpr int i = decltype(ii)::value;
              dot[i] = qsum[t][g] * of_token<token_of(4 * n + i)>(zk[g]);
            });
#pragma unroll
          for (int i = g * GC; i < (g + 1) * GC; ++i)
            dot = __builtin_amdgcn_mfma_f32_16x16x32_f16(k[i], q[t][i], dot, 0, 0, 0);
          each<4>([&](auto ii) {
            constexpr int i = decltype(ii)::value, tok = token_of(4 * n + i);
            const float x = dot[i] * of_token<tok>(ks[g]);
            s[t][4 * n + i] = g == 0 ? x : s[t][4 * n + i] + x;
          });
        }
      }
      // no instruction, but an order: this tile's scores are finished before the
      // next one's codes are taken apart, which keeps the live registers few
#pragma unroll
      for (int t = 0; t < QT; ++t)
        asm volatile("" : "+v"(s[t][4 * n]), "+v"(s[t][4 * n + 1]), "+v"(s[t][4 * n + 2]), "+v"(s[t][4 * n + 3]));
      if constexpr (n < 3) {
#pragma unroll
        for (int i = 0; i < C; ++i) asm volatile("" : "+v"(kw[n + 1].w[i]));
      }
    });
    if (next < end) load_keys(units);

    // --- masks: only where a row does not see the whole step
    const int token0 = step * kStep + 16 * quarter;
    const bool masked = step * kStep < lo_last || (step + 1) * kStep > hi_first || found != 15u;
    if (masked) {
      const bool there = (found >> quarter) & 1u;
#pragma unroll
      for (int t = 0; t < QT; ++t) {
        const int from = lo[t] - token0, to = there ? hi[t] - token0 : -1;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (token_of(i) < from || token_of(i) >= to) s[t][i] = -__builtin_inff();
      }
      // scales of tokens that the sequence does not have (their memory may hold
      // anything) take no part in the largest scale
      const int have = there ? work.w.keys - token0 : 0;
#pragma unroll
      for (int g = 0; g < NG; ++g)
        if (row >= have) vsc[g] = 0;
    }

    // --- the running reference: largest score plus the exponent of the largest
    // scale, an upper bound of log2 of every weight
    uint32_t big = vsc[0];
#pragma unroll
    for (int g = 1; g < NG; ++g) big = vsc[g] > big ? vsc[g] : big;
    const float spread = (float)((int)(row_umax(big) >> 10) - 14 - 9);
    bool move = false;
    float cand[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      float top = s[t][0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = __builtin_fmaxf(top, s[t][i]);
      cand[t] = rows_max(__builtin_fmaf(top, factor[t], spread));
      move |= cand[t] > m[t] + 6.0f;
    }
    if (__ballot(move) != 0) {
#pragma unroll
      for (int t = 0; t < QT; ++t) {
        const float to = __builtin_fmaxf(m[t], cand[t]);
        const float shrink = __builtin_amdgcn_exp2f(m[t] - to);
        m[t] = to;
        l[t] *= shrink;
#pragma unroll
        for (int g = 0; g < (AFF ? NG : 0); ++g) zsum[t][g] *= shrink;
#pragma unroll
        for (int j = 0; j < 2 * C; ++j) acc[t][j] *= shrink;
      }
    }

    // --- probabilities
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[t][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][i], factor[t], -m[t]));
        l[t] += s[t][i];
      }

    // --- values, a group of channels at a time
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      half8_t w[QT][2];
      const float vs = half_bits_to_float(vsc[g]);
#pragma unroll
      for (int t = 0; t < QT; ++t) {
        half2_t pair[8];
        if (!masked) {
          each<8>([&](auto ii) {
            constexpr int i = 2 * decltype(ii)::value;
            pair[i / 2] = half2_t{(_Float16)(s[t][i] * of_token<token_of(i)>(vs)),
                                  (_Float16)(s[t][i + 1] * of_token<token_of(i + 1)>(vs))};
          });
        } else {                         // a hidden token's scale may be infinite or NaN
          each<8>([&](auto ii) {
            constexpr int i = 2 * decltype(ii)::value;
            const float x = s[t][i] * of_token<token_of(i)>(vs), y = s[t][i + 1] * of_token<token_of(i + 1)>(vs);
            pair[i / 2] = half2_t{(_Float16)(s[t][i] == 0.0f ? 0.0f : x), (_Float16)(s[t][i + 1] == 0.0f ? 0.0f : y)};
          });
        }
        if constexpr (AFF) {
          const half2_t off = {(_Float16)-1032.0f, (_Float16)-1032.0f};
#pragma unroll
          for (int i = 0; i < 8; ++i) {     // 1024 + z, then z - 8
            const uint32_t z = ((i & 1 ? vz[g].w[i / 2] >> 8 : vz[g].w[i / 2]) & 0x00FF00FFu) | 0x64006400u;
            zsum[t][g] = __builtin_amdgcn_fdot2(pair[i], __builtin_bit_cast(half2_t, z) + off, zsum[t][g], false);
          }
        }
        w[t][0] = as_half8(pair);
        w[t][1] = as_half8(pair + 4);
      }
#pragma unroll
      for (int j = g * GC; j < (g + 1) * GC; ++j) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          // a word: two channels of four tokens
          half2_t c[8];
          code_pairs<AFF>(vw[j].w[2 * u], c);
          code_pairs<AFF>(vw[j].w[2 * u + 1], c + 4);
          const half2_t lows[4] = {c[0], c[2], c[4], c[6]}, highs[4] = {c[1], c[3], c[5], c[7]};
          const half8_t even = as_half8(lows), odd = as_half8(highs);
#pragma unroll
          for (int t = 0; t < QT; ++t) {
            acc[t][2 * j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(even, w[t][u], acc[t][2 * j], 0, 0, 0);
            acc[t][2 * j + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(odd, w[t][u], acc[t][2 * j + 1], 0, 0, 0);
          }
        }
        if (j + 1 < C) {
#pragma unroll
          for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(vw[j + 1].w[i]) : "v"(acc[QT - 1][2 * j + 1]));
        }
      }
    }
    if (next < end) load_values(units);
  }

  // --- join the block's wavefronts, 16 rows at a time. Lane (row, quarter) holds
  // channels 32 j + 8 quarter .. + 7 of query row `row`.
  __shared__ float ml[2][4][16];
  __shared__ __attribute__((aligned(16))) float rows_out[4][16][32 * C + 4];
  const int tid = threadIdx.x, orow = tid >> 4;
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const float lt = rows_sum(l[t]);
    float zt[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) zt[g] = AFF ? rows_sum(zsum[t][AFF ? g : 0]) : 0.0f;
    if (quarter == 0) {
      ml[0][wave][row] = m[t];
      ml[1][wave][row] = lt;
    }
    __syncthreads();
    const float top = __builtin_fmaxf(__builtin_fmaxf(ml[0][0][row], ml[0][1][row]),
                                      __builtin_fmaxf(ml[0][2][row], ml[0][3][row]));
    const float shrink = __builtin_amdgcn_exp2f(m[t] - top);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = (acc[t][2 * j][i] - zt[j / GC]) * shrink;
        v[2 * i + 1] = (acc[t][2 * j + 1][i] - zt[j / GC]) * shrink;
      }
      float4_t* const to = reinterpret_cast<float4_t*>(&rows_out[wave][row][32 * j + 8 * quarter]);
      to[0] = float4_t{v[0], v[1], v[2], v[3]};
      to[1] = float4_t{v[4], v[5], v[6], v[7]};
    }
    __syncthreads();
    const int flat = flat0 + 16 * t + orow;
    if (flat < flats) {
      float mm = ml[0][0][orow];
#pragma unroll
      for (int i = 1; i < 4; ++i) mm = __builtin_fmaxf(mm, ml[0][i][orow]);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += ml[1][i][orow] * __builtin_amdgcn_exp2f(ml[0][i][orow] - mm);
      const bool whole = work.chunks == 1;
      const float inv = whole ? (sum == 0.0f ? 0.0f : 1.0f / sum) : 1.0f;
      const int64_t orow_at = (work.w.first + (uint32_t)flat / ratio) * ((int64_t)heads * ratio) + kh * ratio +
                              (uint32_t)flat % ratio;
      float* const slot = ws.part + ((int64_t)work.slot * heads + kh) * partial_floats(TR, C);
      for (int d = (tid & 15) * 4; d < 32 * C; d += 64) {
        float4_t v = *reinterpret_cast<const float4_t*>(&rows_out[0][orow][d]);
#pragma unroll
        for (int i = 1; i < 4; ++i) v += *reinterpret_cast<const float4_t*>(&rows_out[i][orow][d]);
        v *= inv;
        if (whole) store_output(a, orow_at, d, v);
        else *reinterpret_cast<float4_t*>(slot + (16 * t + orow) * (32 * C) + d) = v;
      }
      if ((tid & 15) == 0) {
        if (!whole) {
          slot[TR * 32 * C + 2 * (16 * t + orow)] = mm;
          slot[TR * 32 * C + 2 * (16 * t + orow) + 1] = sum;
        } else if (a.lse) {
          a.lse[orow_at] = sum == 0.0f ? -__builtin_inff() : 0.69314718055994530942f * (mm + __builtin_amdgcn_logf(sum));
        }
      }
    }
    __syncthreads();
  }
}

// Defined for each width in a file of its own: launches the form for the cache's
// groups and the schedule's tile height.
template <int C>
hipError_t launch_attention_width(const AttentionArgs& a, const Schedule& s, const Workspace& ws, hipStream_t stream);

}  // namespace int4dq
