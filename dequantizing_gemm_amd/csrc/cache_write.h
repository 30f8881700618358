// cache_write.h -- 64 positions of a sequence written into the 4-bit cache: the
// codes of one token's channels, four threads a token, and how they leave. Shared by
// the kernel that writes rows as they are (cache_store.hip) and the one that normalises
// and rotates keys on the way (cache_append_prompts.hip).
#pragma once

#include "cache_rows.h"
#include "lanes.h"
#include "quantize_common.h"

namespace int4dq {

// The cache's units of the step's four 16-token units for head 0 (head h: h more
// pages of units), -1 where there is no page.
__device__ __forceinline__ void find_units(const CacheView& c, const RowsView& r, const StoreBlock& w,
                                           int64_t units[4]) {
  if (threadIdx.x < 4) {
    const int64_t pos = w.base + 16 * (int)threadIdx.x, page = find_page(r, c, w.b, pos);
    units[threadIdx.x] = page < 0 ? -1 : c.unit(page, 0, (int)(pos & (((int64_t)1 << c.page_shift) - 1)));
  }
  __syncthreads();
}

// Codes, scales and zero points of a thread's channels of one token.
template <int C>
struct Quantised {
  uint32_t word[C];
  uint16_t scale[C];         // of block i's group
  uint8_t zero[C];
};

// A thread's channels of one token: thread `a` of the token's four owns channels
// 32 i + 8 a + e for i < C, e < 8. 0 where there are no channels or no token.
template <int DT, int C>
struct Channels {
  Bits<DT> raw[C][8];

  __device__ __forceinline__ void load(const CacheView& c, const Bits<DT>* src, int wide, int a, bool there) {
    if (wide) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int d = 32 * i + 8 * a;
        const bool have = there && d < c.D;            // head_dim is a multiple of 8
        const auto v = *reinterpret_cast<const Pack<Bits<DT>, 8>*>(src + (have ? d : 0));
#pragma unroll
        for (int e = 0; e < 8; ++e) raw[i][e] = have ? v.v[e] : (Bits<DT>)0;
      }
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int d = 32 * i + 8 * a + e;
          const bool have = there && d < c.D;
          const Bits<DT> v = src[have ? d : 0];
          raw[i][e] = have ? v : (Bits<DT>)0;
        }
    }
  }
};

// Codes of the values value(i, e) of a thread's channels; the token's four threads take
// part together.
template <int C, bool AFF, typename V>
__device__ __forceinline__ Quantised<C> quantise(const CacheView& c, int a, V value) {
  // extremes of each block of 32 channels, then of each group
  float lo[C], hi[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    lo[i] = hi[i] = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = value(i, e);
      if constexpr (AFF) lo[i] = __builtin_fminf(lo[i], x);
      hi[i] = __builtin_fmaxf(hi[i], AFF ? x : __builtin_fabsf(x));
    }
    if constexpr (AFF) lo[i] = run_umax_bits<4>(lo[i]);
    hi[i] = run_umax_bits<4>(hi[i]);
  }
  const int blocks = c.G == 1 ? C : c.group / 32;    // of 32 channels, to a group
  Quantised<C> q;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int from = blocks == C ? 0 : i / blocks * blocks;
    float top = 0.0f, bottom = 0.0f;
#pragma unroll
    for (int k = 0; k < C; ++k)
      if (k >= from && k < from + blocks) {
        top = __builtin_fmaxf(top, hi[k]);
        if constexpr (AFF) bottom = __builtin_fminf(bottom, lo[k]);
      }
    const _Float16 s16 = (_Float16)(AFF ? (top - bottom) / 15.0f : top / 7.0f);
    const float sf = (float)s16, rsf = scale_rcp(sf);
    const uint32_t zp = AFF ? affine_zp(bottom, sf) : 0u;
    q.scale[i] = __builtin_bit_cast(uint16_t, s16);
    q.zero[i] = (uint8_t)zp;
    // code_of / affine_code of the 8 channels, with one branch around the divisions. As
    // code + 8 (affine: the code) on top of kOne, whose unit in the last place is 1, the sum
    // rounds to the code, and the 8 patterns can be added up, each 4 bits higher, with what
    // kOne adds to them taken off at the end. Clamped before, which is the same outside
    // the range; ties, rounded to even of the sum, are among those near a half. (Against
    // rounding, clamping, converting and shifting each: 28114 tokens, 8 heads of 128,
    // bfloat16, 39 -> 37.7 us, with zero points in groups of 32 54.9 -> 49.)
    constexpr float kOne = 0x1.8p23f;
    constexpr uint32_t kOnes = 0x11111111u * 0x4B400000u;
    const float base = AFF ? kOne + (float)zp : kOne + 8.0f;
    const float least = AFF ? -(float)zp : -8.0f, most = AFF ? 15.0f - (float)zp : 7.0f;
    float code[8], far = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float t = __builtin_amdgcn_fmed3f(value(i, e) * rsf, least, most);
      code[e] = base + t;
      far = __builtin_fmaxf(far, __builtin_fabsf(t - (code[e] - base)));
    }
    if (__builtin_expect(far > 0.5f - 0x1p-14f, 0)) {            // near_half_integer of one of them
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = value(i, e);
        if (near_half_integer(x * rsf))
          code[e] = AFF ? kOne + (float)affine_code(x, sf, rsf, zp)
                        : base + __builtin_fminf(__builtin_fmaxf(__builtin_rintf(x / sf), -8.0f), 7.0f);   // IEEE division
      }
    }
    uint32_t word = 0;
#pragma unroll
    for (int e = 7; e >= 0; --e) word = (word << 4) + __builtin_bit_cast(uint32_t, code[e]);
    word -= kOnes;
    if constexpr (AFF) {                               // padding channels have code 0
      const int have = c.D - (32 * i + 8 * a);
      word &= have >= 8 ? ~0u : have <= 0 ? 0u : (1u << (4 * have)) - 1;
    } else {
      word ^= 0x88888888u;
    }
    q.word[i] = word;
  }
  return q;
}

template <int C, bool AFF>
__device__ __forceinline__ void store_scales(const CacheView& c, const Quantised<C>& q, int64_t unit, int ts,
                                             uint16_t* scales, uint8_t* zeros) {
  const int blocks = c.G == 1 ? C : c.group / 32;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int g = blocks == C ? 0 : i / blocks;
    if (i == g * blocks && g < c.G) {
      scales[(unit * c.G + g) * 16 + ts] = q.scale[i];
      if constexpr (AFF) zeros[(unit * c.G + g) * 16 + ts] = q.zero[i];
    }
  }
}

// One head of the block's 64 positions, keys or values. codes(row, position, a, there):
// of the thread's channels of a row's key or value, all four threads of a token and all
// tokens of a wavefront together; may(position): whether the position is written at all.
template <int C, bool AFF, typename M, typename Q>
__device__ __forceinline__ void write_step(const CacheView& c, const RowsView& r, int block, int head, bool is_keys, M may,
                                           Q codes) {
  constexpr int DB = 16 * C;
  __shared__ __attribute__((aligned(16))) uint8_t bytes[4 * DB * 16];            // [unit][channel pair][token]
  __shared__ int64_t units[4];
  __shared__ uint32_t written[4];                    // a bit for each token of the unit
  StoreBlock w;
  if (!find_store_block(r, block, LaneSearch{}, &w)) return;
  find_units(c, r, w, units);
  const int tid = threadIdx.x, token = tid >> 2, a = tid & 3, ts = token & 15;
  const int64_t pos = w.base + token, at_row = pos - w.p0, unit0 = units[token >> 4];      // a wavefront is a unit
  const bool there = at_row >= 0 && at_row < w.rows && unit0 >= 0 && may(pos);
  const int64_t row = w.first + (there ? at_row : 0);
  const uint64_t tokens = __ballot(there);           // lanes 4 t + a
  if ((tid & (kWave - 1)) == 0) {
    uint32_t bits = 0;
#pragma unroll
    for (int t = 0; t < 16; ++t) bits |= (uint32_t)((tokens >> (4 * t)) & 1) << t;
    written[tid >> 6] = bits;
  }
  const int64_t up = (int64_t)head << (c.page_shift - 4), unit = unit0 + up;
  if (tokens) {                                      // the same for the wavefront
    const Quantised<C> q = codes(row, pos, a, there);
    if (there && a == 0)
      store_scales<C, AFF>(c, q, unit, ts, is_keys ? c.k_scales : c.v_scales, is_keys ? c.k_zeros : c.v_zeros);
    if (is_keys) {
      if (there) {
        uint32_t* const to = reinterpret_cast<uint32_t*>(c.k_packed + unit * (16 * DB) + ts * DB + a * 4 * C);
#pragma unroll
        for (int i = 0; i < C; ++i) to[i] = q.word[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          bytes[(token >> 4) * (DB * 16) + (16 * i + 4 * a + k) * 16 + ts] = (uint8_t)(q.word[i] >> (8 * k));
    }
  }
  if (is_keys) return;                               // the same for the block
  __syncthreads();
  for (int it = tid; it < 4 * DB; it += 256) {
    const int u = it / DB, j = it % DB;
    uint32_t mask = written[u];
    if (mask == 0) continue;
    uint8_t* const to = c.v_packed + (units[u] + up) * (16 * DB) + j * 16;
    if (mask == 0xFFFFu) {
      *reinterpret_cast<u32x4_t*>(to) = *reinterpret_cast<const u32x4_t*>(&bytes[it * 16]);
    } else {
      for (; mask; mask &= mask - 1) {
        const int t = __builtin_ctz(mask);
        to[t] = bytes[it * 16 + t];
      }
    }
  }
}

}  // namespace int4dq
