// cache_append.hip -- a projection's queries, keys and values on their way into
// attention over the 4-bit cache, in one pass: norms of queries and keys for each
// head, their rotation by position, and the cache's codes
// (include/int4dq_cache_step.h).
//
// Mathematics, for the channels x of one row and head at position p:
//   r = binary32(1 / sqrt(mean_d x_d^2 + eps)), mean and root in binary64,
//   y_d = (x_d r) w_d,
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin) for each pair (a, b),
// every product and sum rounded to binary32 by itself. The codes of a key go by the
// last bit of this where a value lies next to a border between two codes; stated so,
// and with a sum whose order does not show in binary32, they can be reproduced.
#include "cache_rows.h"
#include "cache_step.h"
#include "lanes.h"
#include "quantize_common.h"

namespace int4dq {

namespace {

// What the kernels take besides the caller's arguments.
struct AppendPlan {
  RowArray q, k, v;
  int out_wide;              // as RowArray::wide, of the output
  int turn_wide;             // weights, cosines and sines of 8 channels lie 16-byte aligned, and their partners are 8 channels side by side
  int group_lanes;           // lanes of a scale's group: 4, 8, 16 or 32
  int64_t kv_blocks;         // steps: the first blocks; the others take queries
  int q_heads_per_block, kv_heads_per_block;         // heads that a block takes in turn
};

// ---------------------------------------------------------------- norm and rotation

template <int CTRL>
__device__ __forceinline__ double add_dpp(double v) {
  const u32x2_t x = __builtin_bit_cast(u32x2_t, v);
  const uint32_t x0 = x.x, x1 = x.y;
  u32x2_t y;
  y.x = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x0, CTRL, 0xF, 0xF, true);
  y.y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x1, CTRL, 0xF, 0xF, true);
  return v + __builtin_bit_cast(double, y);
}
// Over LANES adjacent lanes (a power of two up to 32).
template <int LANES>
__device__ __forceinline__ double lanes_sum(double v) {
  v = add_dpp<0xB1>(v);
  v = add_dpp<0x4E>(v);
  if constexpr (LANES >= 8) v = add_dpp<0x141>(v);
  if constexpr (LANES >= 16) v = add_dpp<0x140>(v);
  if constexpr (LANES >= 32) v += __shfl_xor(v, 16);
  return v;
}

// binary32(1 / sqrt(m)): an estimate within 2^-20 and a step of third order, which
// leaves 2^-52. At 0 and infinity the estimate, infinity and 0, is the value.
__device__ __forceinline__ float norm_factor(double m) {
  const double y = __builtin_amdgcn_rsq(m);
  const double e = __builtin_fma(-m * y, y, 1.0);
  const double better = __builtin_fma(y * e, __builtin_fma(e, 0.375, 0.5), y);
  return (float)(m > 0.0 && m < __builtin_inf() ? better : y);
}

// The weights, cosines and sines of 8 channels from d on, and where their partners lie.
struct Turn {
  float w[8], wp[8], c[8], s[8];         // s: the sign of its product is in it
  uint32_t turned;                       // a bit for each channel that is rotated
  int partner;                           // of channel d, with halves; the others follow it

  __device__ __forceinline__ void load(const AppendArgs& a, const AppendPlan& p, const float* norm, int64_t pos, int d) {
    const int D = a.c.D, half = a.rope ? a.half : 0;
    turned = 0;
    partner = d;
    if (p.turn_wide) {                   // head_dim and half are multiples of 8
      const bool in = d < D, turn = d < 2 * half;
      const int at = in ? d : 0, pair = turn ? (a.interleaved ? d / 2 : d < half ? d : d - half) : 0;
      if (turn) turned = 0xFFu;
      if (turn && !a.interleaved) partner = d < half ? d + half : d - half;
      if (norm) {
        const int other = in ? partner : 0;
        const float4_t* const w4 = reinterpret_cast<const float4_t*>(norm + at);
        const float4_t* const v4 = reinterpret_cast<const float4_t*>(norm + other);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          w[e] = w4[e / 4][e % 4];
          wp[e] = a.interleaved ? w4[e / 4][(e ^ 1) % 4] : v4[e / 4][e % 4];
        }
      }
      if (half > 0) {
        const float* const row = a.rope + pos * a.rope_stride;
        const float4_t* const c4 = reinterpret_cast<const float4_t*>(row + pair);
        const float4_t* const s4 = reinterpret_cast<const float4_t*>(row + half + pair);
        if (a.interleaved) {
          const float4_t x = c4[0], y = s4[0];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            c[e] = x[e / 2];
            s[e] = e & 1 ? y[e / 2] : -y[e / 2];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            c[e] = c4[e / 4][e % 4];
            s[e] = d < half ? -s4[e / 4][e % 4] : s4[e / 4][e % 4];
          }
        }
      }
      return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int x = d + e;
      const bool in = x < D, turn = x < 2 * half;
      const int pair = !turn ? 0 : a.interleaved ? x / 2 : x < half ? x : x - half;
      const int other = !turn ? x : a.interleaved ? x ^ 1 : x < half ? x + half : x - half;
      if (turn) turned |= 1u << e;
      if (norm) {
        w[e] = norm[in ? x : 0];
        wp[e] = norm[in ? other : 0];
      }
      if (half > 0) {
        const float* const row = a.rope + pos * a.rope_stride;
        c[e] = row[pair];
        const float y = row[half + pair];
        s[e] = (a.interleaved ? (x & 1) : x >= half) ? y : -y;
      }
    }
  }
};

// The partners of 8 channels from d on in the halves' form (of a channel that has
// none, itself), from the row in memory: it was read just before.
template <int DT>
__device__ __forceinline__ void load_partners(const AppendArgs& a, const AppendPlan& p, const Turn& t, const Bits<DT>* src,
                                              int wide, int d, Bits<DT> raw[8]) {
  if (wide && p.turn_wide) {
    const auto v = *reinterpret_cast<const Pack<Bits<DT>, 8>*>(src + (t.partner < a.c.D ? t.partner : 0));
#pragma unroll
    for (int e = 0; e < 8; ++e) raw[e] = v.v[e];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int x = d + e, other = x >= 2 * a.half ? x : x < a.half ? x + a.half : x - a.half;
      raw[e] = src[other < a.c.D ? other : 0];
    }
  }
}

// Normalised and rotated values of 8 channels from d on; 0 from head_dim on.
__device__ __forceinline__ void turn8(const AppendArgs& a, const Turn& t, bool normed, float r, int d, const float x[8],
                                      const float xp[8], float y[8]) {
#pragma clang fp contract(off)
  float n[8], np[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    n[e] = normed ? (x[e] * r) * t.w[e] : x[e];
    np[e] = normed ? (xp[e] * r) * t.wp[e] : xp[e];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float own = n[e] * t.c[e], other = np[e] * t.s[e];
    const float z = (t.turned >> e) & 1u ? own + other : n[e];
    y[e] = d + e < a.c.D ? z : 0.0f;
  }
}

// The partners' values of a lane's 8 channels.
template <int DT>
__device__ __forceinline__ void partners_of(const AppendArgs& a, const AppendPlan& p, const Turn& t, const Bits<DT>* src,
                                            int wide, int d, const float x[8], float xp[8]) {
  if (a.interleaved || !a.rope) {
#pragma unroll
    for (int e = 0; e < 8; ++e) xp[e] = x[e ^ 1];
  } else {
    Bits<DT> raw[8];
    load_partners<DT>(a, p, t, src, wide, d, raw);
#pragma unroll
    for (int e = 0; e < 8; ++e) xp[e] = value_of<DT>(raw[e]);
  }
}

// A lane's 8 channels of a row; 0 from head_dim on.
template <int DT>
__device__ __forceinline__ void load_channels(const Bits<DT>* src, int wide, int d, int D, float x[8]) {
  if (wide) {
    const bool in = d < D;
    const auto v = *reinterpret_cast<const Pack<Bits<DT>, 8>*>(src + (in ? d : 0));
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = in ? value_of<DT>(v.v[e]) : 0.0f;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const Bits<DT> v = src[d + e < D ? d + e : 0];
      x[e] = d + e < D ? value_of<DT>(v) : 0.0f;
    }
  }
}

// A row's head of queries or keys: loads, normalises and rotates a lane's 8 channels.
template <int DT, int L>
__device__ __forceinline__ void transformed(const AppendArgs& a, const AppendPlan& p, const Turn& t, bool normed,
                                            const Bits<DT>* src, int wide, int d, float y[8]) {
  float x[8], xp[8];
  load_channels<DT>(src, wide, d, a.c.D, x);
  partners_of<DT>(a, p, t, src, wide, d, x, xp);
  float r = 1.0f;
  if (normed) {
    double sum = 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = __builtin_fma((double)x[e], (double)x[e], sum);
    r = norm_factor(lanes_sum<L>(sum) / (double)a.c.D + a.eps);
  }
  turn8(a, t, normed, r, d, x, xp, y);
}

// ---------------------------------------------------------------- codes

// Codes of a lane's 8 channels, with their group's scale and zero point: the
// arithmetic of quantize_common.h.
struct Codes {
  uint32_t word;
  uint16_t scale;
  uint8_t zero;
};

// The largest pattern (run_umax_bits) over the group's lanes.
__device__ __forceinline__ float group_umax(float v, int lanes) {
  uint32_t u = __builtin_bit_cast(uint32_t, v);
  u = dpp_umax<0xB1>(u);
  u = dpp_umax<0x4E>(u);
  if (lanes >= 8) u = dpp_umax<0x141>(u);
  if (lanes >= 16) u = dpp_umax<0x140>(u);
  if (lanes >= 32) {
    const uint32_t o = (uint32_t)__shfl_xor((int)u, 16);
    u = u > o ? u : o;
  }
  return __builtin_bit_cast(float, u);
}

template <bool AFF>
__device__ __forceinline__ Codes codes_of(const AppendArgs& a, const AppendPlan& p, int d, const float x[8]) {
  float lo = 0.0f, hi = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (AFF) lo = __builtin_fminf(lo, x[e]);
    hi = __builtin_fmaxf(hi, AFF ? x[e] : __builtin_fabsf(x[e]));
  }
  if constexpr (AFF) lo = group_umax(lo, p.group_lanes);
  hi = group_umax(hi, p.group_lanes);
  const _Float16 s16 = (_Float16)(AFF ? (hi - lo) / 15.0f : hi / 7.0f);
  const float sf = (float)s16, rsf = scale_rcp(sf);
  const uint32_t zp = AFF ? affine_zp(lo, sf) : 0u;
  float code[8];
  bool near = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = x[e] * rsf, n = __builtin_rintf(t);
    near |= __builtin_fabsf(__builtin_fabsf(t - n) - 0.5f) < 0x1p-14f;           // near_half_integer(t)
    code[e] = AFF ? __builtin_fminf(__builtin_fmaxf(n + (float)zp, 0.0f), 15.0f)
                  : __builtin_fminf(__builtin_fmaxf(n, -8.0f), 7.0f);
  }
  if (__builtin_expect(near, 0)) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (near_half_integer(x[e] * rsf))
        code[e] = AFF ? (float)affine_code(x[e], sf, rsf, zp)
                      : __builtin_fminf(__builtin_fmaxf(__builtin_rintf(x[e] / sf), -8.0f), 7.0f);   // IEEE division
  }
  Codes q{0, __builtin_bit_cast(uint16_t, s16), (uint8_t)zp};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t u = (uint32_t)(int)code[e] & 15u;
    q.word |= (!AFF || d + e < a.c.D ? u : 0u) << (4 * e);                         // padding channels have code 0
  }
  return q;
}
__device__ __forceinline__ Codes codes_of(const AppendArgs& a, const AppendPlan& p, int d, const float x[8]) {
  return a.c.affine ? codes_of<true>(a, p, d, x) : codes_of<false>(a, p, d, x);
}

__device__ __forceinline__ void store_scale(const AppendArgs& a, const AppendPlan& p, const Codes& q, bool keys, int64_t unit,
                                            int ts, int lane) {
  const int g = lane / p.group_lanes;
  if (lane % p.group_lanes == 0 && g < a.c.G) {
    const int64_t at = (unit * a.c.G + g) * 16 + ts;
    (keys ? a.c.k_scales : a.c.v_scales)[at] = q.scale;
    if (a.c.affine) (keys ? a.c.k_zeros : a.c.v_zeros)[at] = q.zero;
  }
}
// Lane 4 i + j of a row has word i of its key's part j.
__device__ __forceinline__ void store_key(const CacheView& c, const Codes& q, int64_t unit, int ts, int lane) {
  if (lane < 4 * c.C)
    *reinterpret_cast<uint32_t*>(c.k_packed + unit * (256 * c.C) + ts * (16 * c.C) + (lane & 3) * 4 * c.C + (lane >> 2) * 4) = q.word;
}

// ---------------------------------------------------------------- rows

__device__ __forceinline__ bool position_there(const AppendArgs& a, int64_t pos) {
  return pos >= 0 && (!a.rope || pos < a.positions);
}

// A lane's 8 channels of the output.
template <int DT>
__device__ __forceinline__ void store_query(const AppendArgs& a, const AppendPlan& p, int64_t row, int head, int d,
                                            const float y[8]) {
  Bits<DT>* const to = static_cast<Bits<DT>*>(a.out) + (row * a.q_heads + head) * a.c.D + d;
  Pack<Bits<DT>, 8> out;
#pragma unroll
  for (int e = 0; e < 8; ++e) out.v[e] = bits_of<DT>(y[e]);
  if (p.out_wide) {
    if (d < a.c.D) *reinterpret_cast<Pack<Bits<DT>, 8>*>(to) = out;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (d + e < a.c.D) to[e] = out.v[e];
  }
}

template <int DT>
__device__ __forceinline__ const Bits<DT>* at_row(const RowArray& x, int64_t row, int head) {
  return static_cast<const Bits<DT>*>(x.p) + row * x.row_stride + head * x.head_stride;
}

// Where sequences have few rows: L lanes for one head of a row's queries, keys or
// values, in this order. Value codes leave byte by byte.
template <int DT, int L>
__global__ __launch_bounds__(256) void cache_append_rows_kernel(AppendArgs a, AppendPlan p) {
  const CacheView& c = a.c;
  const int lane = threadIdx.x & (L - 1), d = 8 * lane, all = a.q_heads + 2 * c.heads;
  const int64_t index = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L, row = index / all;
  const int which = (int)(index - row * all);
  int seq = 0;
  int64_t pos = -1;
  if (row >= a.r.rows || !find_row(a.r, row, &seq, &pos)) return;                  // the same for the L lanes
  const bool there = position_there(a, pos);
  if (which < a.q_heads) {
    float y[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (there) {
      Turn t;
      t.load(a, p, a.q_norm, pos, d);
      transformed<DT, L>(a, p, t, a.q_norm != nullptr, at_row<DT>(p.q, row, which), p.q.wide, d, y);
    }
    return store_query<DT>(a, p, row, which, d, y);
  }
  const int64_t page = there ? find_page(a.r, c, seq, pos) : -1;
  if (page < 0) return;
  const bool keys = which < a.q_heads + c.heads;
  const int head = which - a.q_heads - (keys ? 0 : c.heads), ts = (int)(pos & 15);
  const int64_t unit = c.unit(page, head, (int)(pos & (((int64_t)1 << c.page_shift) - 1)));
  float y[8];
  if (keys) {
    Turn t;
    t.load(a, p, a.k_norm, pos, d);
    transformed<DT, L>(a, p, t, a.k_norm != nullptr, at_row<DT>(p.k, row, head), p.k.wide, d, y);
  } else {
    load_channels<DT>(at_row<DT>(p.v, row, head), p.v.wide, d, c.D, y);
  }
  const Codes q = codes_of(a, p, d, y);
  store_scale(a, p, q, keys, unit, ts, lane);
  if (keys) {
    store_key(c, q, unit, ts, lane);
  } else if (lane < 4 * c.C) {
    uint8_t* const to = c.v_packed + unit * (256 * c.C) + ts;
#pragma unroll
    for (int k = 0; k < 4; ++k) to[(4 * lane + k) * 16] = (uint8_t)(q.word >> (8 * k));
  }
}

// ---------------------------------------------------------------- prompts

// 64 positions of a sequence (find_store_block), several heads of one side in turn.
// Value codes go through LDS and leave as 16-byte rows of a unit; a unit of which
// some tokens are not written leaves byte by byte.
template <int DT, int L>
__device__ __forceinline__ void append_step(const AppendArgs& a, const AppendPlan& p, int64_t block, uint8_t (*bytes)[4 * 128 * 16],
                                            int64_t units[4], uint32_t* written) {
  constexpr int ROWS = 256 / L;
  const CacheView& c = a.c;
  const int chunks = (c.heads + p.kv_heads_per_block - 1) / p.kv_heads_per_block;
  const bool keys = block & 1;
  const int head0 = (int)((block >> 1) % chunks) * p.kv_heads_per_block;
  const int head1 = head0 + p.kv_heads_per_block < c.heads ? head0 + p.kv_heads_per_block : c.heads;
  StoreBlock w;
  if (!find_store_block(a.r, (int)((block >> 1) / chunks), LaneSearch{}, &w)) return;
  const int tid = threadIdx.x, lane = tid & (L - 1), d = 8 * lane, DB = 16 * c.C;
  const int page_units = 1 << (c.page_shift - 4);
  if (tid < 4) {
    const int64_t pos = w.base + 16 * tid, page = find_page(a.r, c, w.b, pos);
    units[tid] = page < 0 ? -1 : c.unit(page, 0, (int)(pos & (((int64_t)1 << c.page_shift) - 1)));
  }
  __syncthreads();
  auto token_there = [&](int token) {
    const int64_t pos = w.base + token, at = pos - w.p0;
    return at >= 0 && at < w.rows && units[token >> 4] >= 0 && position_there(a, pos);
  };
  if (keys) {
#pragma unroll 1
    for (int token = tid / L; token < 64; token += ROWS) {
      if (!token_there(token)) continue;
      const int64_t pos = w.base + token, row = w.first + (pos - w.p0);
      Turn t;
      t.load(a, p, a.k_norm, pos, d);
#pragma unroll 1
      for (int head = head0; head < head1; ++head) {
        float y[8];
        transformed<DT, L>(a, p, t, a.k_norm != nullptr, at_row<DT>(p.k, row, head), p.k.wide, d, y);
        const Codes q = codes_of(a, p, d, y);
        const int64_t unit = units[token >> 4] + (int64_t)head * page_units;
        store_scale(a, p, q, true, unit, token & 15, lane);
        store_key(c, q, unit, token & 15, lane);
      }
    }
    return;
  }
  if (tid < kWave) {
    const uint64_t there = __ballot(token_there(tid));
    if (tid < 4) written[tid] = (uint32_t)(there >> (16 * tid)) & 0xFFFFu;
  }
#pragma unroll 1
  for (int head = head0, turn = 0; head < head1; ++head, turn ^= 1) {
#pragma unroll 1
    for (int token = tid / L; token < 64; token += ROWS) {
      if (!token_there(token)) continue;
      const int64_t row = w.first + (w.base + token - w.p0);
      float y[8];
      load_channels<DT>(at_row<DT>(p.v, row, head), p.v.wide, d, c.D, y);
      const Codes q = codes_of(a, p, d, y);
      store_scale(a, p, q, false, units[token >> 4] + (int64_t)head * page_units, token & 15, lane);
      if (lane < 4 * c.C)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          bytes[turn][((token >> 4) * DB + 4 * lane + k) * 16 + (token & 15)] = (uint8_t)(q.word >> (8 * k));
    }
    __syncthreads();                     // two buffers: the one written next was read before this
    for (int it = tid; it < 4 * DB; it += 256) {
      const int u = it / DB, j = it % DB;
      uint32_t mask = written[u];
      if (mask == 0) continue;
      uint8_t* const to = c.v_packed + (units[u] + (int64_t)head * page_units) * (16 * DB) + j * 16;
      if (mask == 0xFFFFu) {
        *reinterpret_cast<u32x4_t*>(to) = *reinterpret_cast<const u32x4_t*>(&bytes[turn][it * 16]);
      } else {
        for (; mask; mask &= mask - 1) {
          const int t = __builtin_ctz(mask);
          to[t] = bytes[turn][it * 16 + t];
        }
      }
    }
  }
}

// Rows of queries, L lanes a row, several heads in turn.
template <int DT, int L>
__device__ __forceinline__ void append_queries(const AppendArgs& a, const AppendPlan& p, int64_t block) {
  const int chunks = (a.q_heads + p.q_heads_per_block - 1) / p.q_heads_per_block;
  const int64_t row = block / chunks * (256 / L) + threadIdx.x / L;
  const int head0 = (int)(block % chunks) * p.q_heads_per_block;
  const int head1 = head0 + p.q_heads_per_block < a.q_heads ? head0 + p.q_heads_per_block : a.q_heads;
  const int d = (threadIdx.x & (L - 1)) * 8;
  int seq = 0;
  int64_t pos = -1;
  if (row >= a.r.rows || !find_row(a.r, row, &seq, &pos)) return;                  // the same for the L lanes
  const bool there = position_there(a, pos);
  Turn t;
  t.load(a, p, a.q_norm, there ? pos : 0, d);
#pragma unroll 1
  for (int head = head0; head < head1; ++head) {
    float y[8];
    transformed<DT, L>(a, p, t, a.q_norm != nullptr, at_row<DT>(p.q, row, head), p.q.wide, d, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = there ? y[e] : 0.0f;
    store_query<DT>(a, p, row, head, d, y);
  }
}

template <int DT, int L>
__global__ __launch_bounds__(256) void cache_append_steps_kernel(AppendArgs a, AppendPlan p) {
  __shared__ __attribute__((aligned(16))) uint8_t bytes[2][4 * 128 * 16];            // [unit][channel pair][token]
  __shared__ int64_t units[4];
  __shared__ uint32_t written[4];                    // a bit for each token of the unit
  const int64_t block = blockIdx.x;
  if (block < p.kv_blocks) append_step<DT, L>(a, p, block, bytes, units, written);
  else append_queries<DT, L>(a, p, block - p.kv_blocks);
}

// ---------------------------------------------------------------- launches

template <int DT, int L>
void launch_lanes(const AppendArgs& a, AppendPlan p, hipStream_t stream) {
  constexpr int ROWS = 256 / L;
  if (!a.r.starts || a.r.rows < 8 * (int64_t)a.r.batch) {
    const int64_t items = a.r.rows * (a.q_heads + 2 * a.c.heads);
    hipLaunchKernelGGL((cache_append_rows_kernel<DT, L>), dim3((unsigned)((items + ROWS - 1) / ROWS)), dim3(256), 0, stream,
                       a, p);
    return;
  }
  // Several heads a block, which share cosines and sines, as long as that leaves twice
  // the 2048 blocks that the GPU holds at once.
  auto per_block = [](int64_t blocks, int heads) {
    int n = 1;
    while (n < 8 && blocks * (heads / (2 * n)) >= 4096) n *= 2;
    return n;
  };
  const int64_t units = store_units(a.r), row_blocks = (a.r.rows + ROWS - 1) / ROWS;
  p.kv_heads_per_block = per_block(2 * units, a.c.heads);
  p.q_heads_per_block = per_block(row_blocks, a.q_heads);
  p.kv_blocks = 2 * units * ((a.c.heads + p.kv_heads_per_block - 1) / p.kv_heads_per_block);
  const int64_t blocks = p.kv_blocks + row_blocks * ((a.q_heads + p.q_heads_per_block - 1) / p.q_heads_per_block);
  hipLaunchKernelGGL((cache_append_steps_kernel<DT, L>), dim3((unsigned)blocks), dim3(256), 0, stream, a, p);
}

template <int DT>
hipError_t launch_type(const AppendArgs& a, const AppendPlan& p, hipStream_t stream) {
  if (a.c.C <= 2) launch_lanes<DT, 8>(a, p, stream);
  else if (a.c.C <= 4) launch_lanes<DT, 16>(a, p, stream);
  else launch_lanes<DT, 32>(a, p, stream);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_append(const AppendArgs& a, int dtype, hipStream_t stream) {
  const int per16 = dtype == INT4DQ_ROWS_F32 ? 4 : 8;          // elements of 16 bytes
  auto rows = [&](const void* x, int64_t row_stride, int64_t head_stride) {
    const int wide = a.c.D % 8 == 0 && (uintptr_t)x % 16 == 0 && row_stride % per16 == 0 && head_stride % per16 == 0;
    return RowArray{const_cast<void*>(x), row_stride, head_stride, wide};
  };
  AppendPlan p{rows(a.q, a.q_row_stride, a.q_head_stride), rows(a.k, a.k_row_stride, a.k_head_stride),
               rows(a.v, a.v_row_stride, a.v_head_stride), a.c.D % 8 == 0 && (uintptr_t)a.out % 16 == 0, 0, 0, 0, 1, 1};
  p.turn_wide = a.c.D % 8 == 0 && ((uintptr_t)a.q_norm | (uintptr_t)a.k_norm | (uintptr_t)a.rope) % 16 == 0 &&
                (!a.rope || (a.half % 8 == 0 && a.rope_stride % 4 == 0));
  p.group_lanes = a.c.G > 1 ? a.c.group / 8 : a.c.C <= 2 ? 8 : a.c.C <= 4 ? 16 : 32;
  if (dtype == INT4DQ_ROWS_F32) return launch_type<INT4DQ_ROWS_F32>(a, p, stream);
  if (dtype == INT4DQ_ROWS_F16) return launch_type<INT4DQ_ROWS_F16>(a, p, stream);
  return launch_type<INT4DQ_ROWS_BF16>(a, p, stream);
}

}  // namespace int4dq
