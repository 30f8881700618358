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
// last bit of this where a value lies next to a border between two codes: the squares are
// summed in one order in all forms, 8 channels one after the other and then in pairs, so
// that a code does not depend on the call that wrote it. (Before it is rounded, r is that of
// the binary64 sum within 2^-52; another order of the sum can give another last bit of r.)
//
// Work. L lanes (8, 16 or 32) take a row's head, 8 channels each: 16 bytes a load, the
// sum over the lanes by DPP, the partner of a channel from the lane that has it, and one
// word of 8 codes a lane. Single tokens, drafts and short prompts go so, queries, keys
// and values side by side in one launch; one token of 8 + 32 heads of 128 takes 4.4 us,
// 128 of them 5.3 us, bound by the chain of dependent loads. Of long prompts the queries
// go so, several heads a block, which share cosines and sines, and keys and values in
// the write kernel's arrangement (cache_append_prompts.hip).
//
// What bounds long prompts (28114 tokens of 8 + 32 heads of 128, bfloat16, symmetric codes
// in groups of 128): the queries memory, 460 MB in 101 us, 4.6 TB/s; keys and values the
// latency of their loads and the VALU (busy for half of 73 us): a block is 64 tokens of
// one head, and four wavefronts a SIMD is what its 122 registers leave. Both in one
// launch with their blocks in turns took 187 us, one after the other 175. Summing in
// binary64 costs nothing that shows (without norms 154 us, without rotation 147 of 175).
#include "cache_append.h"
#include "quantize_common.h"

namespace int4dq {

namespace {

// ---------------------------------------------------------------- 8 channels a lane

// The weights, cosines and sines of 8 channels from d on, and where their partners
// lie. WIDE, here and below: the rows' 8 channels lie 16-byte aligned in every array,
// weights, cosines and sines as well, head_dim and half are multiples of 8, so that the
// partners of 8 channels are 8 channels side by side.
template <bool WIDE>
struct Turn {
  float w[8], c[8], s[8];                // s: the sign of its product is in it
  float wp[WIDE ? 1 : 8];                // of the partners
  uint32_t turned;                       // a bit for each channel that is rotated
  int partner;                           // WIDE, in halves: the lane of the wavefront that has the channels' partners

  __device__ __forceinline__ void load(const AppendArgs& a, const float* norm, int64_t pos, int d) {
    const int D = a.c.D, half = a.rope ? a.half : 0;
    turned = 0;
    partner = threadIdx.x & (kWave - 1);
    if constexpr (WIDE) {
      const bool in = d < D, turn = d < 2 * half;
      const int at = in ? d : 0, pair = turn ? (a.interleaved ? d / 2 : d < half ? d : d - half) : 0;
      if (turn) turned = 0xFFu;
      if (turn && !a.interleaved) partner += d < half ? half / 8 : -(half / 8);
      if (norm) {
        const float4_t w0 = reinterpret_cast<const float4_t*>(norm + at)[0], w1 = reinterpret_cast<const float4_t*>(norm + at)[1];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = e < 4 ? w0[e % 4] : w1[e % 4];
      }
      if (half > 0) {
        const float* const row = a.rope + pos * a.rope_stride;
        const float4_t* const c4 = reinterpret_cast<const float4_t*>(row + pair);
        const float4_t* const s4 = reinterpret_cast<const float4_t*>(row + half + pair);
        const float4_t c0 = c4[0], s0 = s4[0];
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            c[e] = c0[e / 2];
            s[e] = e & 1 ? s0[e / 2] : -s0[e / 2];
          }
        } else {
          const float4_t c1 = c4[1], s1 = s4[1];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float x = e < 4 ? s0[e % 4] : s1[e % 4];
            c[e] = e < 4 ? c0[e % 4] : c1[e % 4];
            s[e] = d < half ? -x : x;
          }
        }
      }
    } else {
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
  }
};

// From the lane that has the partners of a lane's channels.
template <int L>
__device__ __forceinline__ float of_partner(const AppendArgs& a, int partner, float v) {
  if (L == 16 && a.half == 64)                       // the same for all: 128 channels in halves of a row's 16 lanes
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x128, 0xF, 0xF, true));
  return __builtin_bit_cast(float, __builtin_amdgcn_ds_bpermute(4 * partner, __builtin_bit_cast(int, v)));
}

// A lane's 8 channels of a row as they lie in memory (from head_dim on, some other
// channel), and where not WIDE their partners in the halves' form (of a channel that
// has none, itself).
template <int DT, bool WIDE>
struct Raw {
  Bits<DT> v[8], p[WIDE ? 1 : 8];

  __device__ __forceinline__ void load(const Bits<DT>* src, int d, int D) {
    if constexpr (WIDE) {
      const auto x = *reinterpret_cast<const Pack<Bits<DT>, 8>*>(src + (d < D ? d : 0));
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = x.v[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = src[d + e < D ? d + e : 0];
    }
  }
  __device__ __forceinline__ void load_partners(const AppendArgs& a, const Bits<DT>* src, int d) {
    if constexpr (!WIDE) {
      if (a.interleaved || !a.rope) return;          // the same for all
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int x = d + e, other = x >= 2 * a.half ? x : x < a.half ? x + a.half : x - a.half;
        p[e] = src[other < a.c.D ? other : 0];
      }
    }
  }
  // 0 from head_dim on
  __device__ __forceinline__ void values(int d, int D, float x[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (WIDE ? d : d + e) < D ? value_of<DT>(v[e]) : 0.0f;
  }
};

// A row's head of queries or keys: normalises and rotates a lane's 8 channels; 0 from
// head_dim on. All L lanes take part.
template <int DT, int L, bool WIDE>
__device__ __forceinline__ void transformed(const AppendArgs& a, const AppendPlan& p, const Turn<WIDE>& t, bool normed,
                                            const Raw<DT, WIDE>& raw, int d, float y[8]) {
#pragma clang fp contract(off)
  float r = 1.0f;
  raw.values(d, a.c.D, y);
  if (normed) {
    double sum = 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = __builtin_fma((double)y[e], (double)y[e], sum);
    r = norm_factor(lanes_sum<L>(sum) * p.mean + a.eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = (y[e] * r) * t.w[e];
  }
  if (a.rope) {
    float other[8];
    if (a.interleaved) {
#pragma unroll
      for (int e = 0; e < 8; ++e) other[e] = y[e ^ 1];
    } else if constexpr (WIDE) {
#pragma unroll
      for (int e = 0; e < 8; ++e) other[e] = of_partner<L>(a, t.partner, y[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        other[e] = value_of<DT>(raw.p[e]);
        if (normed) other[e] = (other[e] * r) * t.wp[e];
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = y[e] * t.c[e], z = other[e] * t.s[e], turned = x + z;
      y[e] = (WIDE ? t.turned != 0 : (t.turned >> e) & 1u) ? turned : y[e];
    }
  }
  if constexpr (!WIDE) {                             // weights of other channels have been there
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = d + e < a.c.D ? y[e] : 0.0f;
  } else if (a.c.D < 8 * L) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = d < a.c.D ? y[e] : 0.0f;
  }
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
  // codes of quantize_common.h's code_of and affine_code, from 0 up (symmetric ones plus
  // 8), with one branch around the divisions: |t - rint(t)| is at most a half, and
  // where it is that within 2^-14 the quotient decides
  constexpr float kZero = AFF ? 0.0f : 8.0f;
  const float up = AFF ? (float)zp : kZero;
  float code[8], most = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = x[e] * rsf, n = __builtin_rintf(t);
    most = __builtin_fmaxf(most, __builtin_fabsf(t - n));
    code[e] = __builtin_amdgcn_fmed3f(n + up, 0.0f, 15.0f);
  }
  if (__builtin_expect(most > 0.5f - 0x1p-14f, 0)) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (near_half_integer(x[e] * rsf))
        code[e] = AFF ? (float)affine_code(x[e], sf, rsf, zp)
                      : __builtin_fminf(__builtin_fmaxf(__builtin_rintf(x[e] / sf), -8.0f), 7.0f) + kZero;   // IEEE division
  }
  if (AFF && a.c.D % 8 != 0)                         // padding channels have code 0
#pragma unroll
    for (int e = 0; e < 8; ++e) code[e] = d + e < a.c.D ? code[e] : 0.0f;
  // four nibbles are a whole number below 2^16, exact in binary32
  auto four = [&](int e) {
    return (uint32_t)__builtin_fmaf(__builtin_fmaf(__builtin_fmaf(code[e + 3], 16.0f, code[e + 2]), 16.0f, code[e + 1]), 16.0f, code[e]);
  };
  const uint32_t word = four(0) | four(4) << 16;
  // two's complement: the highest bit of a nibble the other way round; code 0 is 8 from 0 up
  return Codes{AFF ? (d < a.c.D ? word : 0u) : word ^ 0x88888888u, __builtin_bit_cast(uint16_t, s16), (uint8_t)zp};
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

// Two outputs as binary16 or bfloat16 patterns, rounded to nearest even.
template <int DT>
__device__ __forceinline__ uint32_t pair_of(float x, float y) {
  if constexpr (DT == INT4DQ_ROWS_BF16) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    const bf16x2_t v = {(__bf16)x, (__bf16)y};
    return __builtin_bit_cast(uint32_t, v);
  } else {
    const half2_t v = {(_Float16)x, (_Float16)y};
    return __builtin_bit_cast(uint32_t, v);
  }
}

// A lane's 8 channels of the output.
template <int DT, bool WIDE>
__device__ __forceinline__ void store_query(const AppendArgs& a, int64_t row, int head, int d, const float y[8]) {
  Bits<DT>* const to = static_cast<Bits<DT>*>(a.out) + (row * a.q_heads + head) * a.c.D + d;
  if constexpr (WIDE) {
    if (d >= a.c.D) return;
    if constexpr (DT == INT4DQ_ROWS_F32) {
      reinterpret_cast<float4_t*>(to)[0] = float4_t{y[0], y[1], y[2], y[3]};
      reinterpret_cast<float4_t*>(to)[1] = float4_t{y[4], y[5], y[6], y[7]};
    } else {
      *reinterpret_cast<u32x4_t*>(to) = u32x4_t{pair_of<DT>(y[0], y[1]), pair_of<DT>(y[2], y[3]), pair_of<DT>(y[4], y[5]),
                                                pair_of<DT>(y[6], y[7])};
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (d + e < a.c.D) to[e] = bits_of<DT>(y[e]);
  }
}

// Where sequences have few rows: L lanes for one head of a row's queries, keys or
// values, in this order. Value codes leave byte by byte.
template <int DT, int L, bool WIDE>
__global__ __launch_bounds__(256) void cache_append_rows_kernel(AppendArgs a, AppendPlan p) {
  const CacheView& c = a.c;
  const int lane = threadIdx.x & (L - 1), d = 8 * lane, all = a.q_heads + 2 * c.heads;
  const int64_t index = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L, row = index / all;
  const int which = (int)(index - row * all);
  int seq = 0;
  int64_t pos = -1;
  if (row >= a.r.rows || !find_row(a.r, row, &seq, &pos)) return;                  // the same for the L lanes
  const bool there = position_there(a, pos), query = which < a.q_heads, keys = !query && which < a.q_heads + c.heads;
  const int head = query ? which : which - a.q_heads - (keys ? 0 : c.heads);
  const RowArray& in = query ? p.q : keys ? p.k : p.v;
  const float* const norm = query ? a.q_norm : a.k_norm;
  const Bits<DT>* const src = at_row<DT>(in, row, head);
  float y[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (there) {
    Raw<DT, WIDE> raw;
    raw.load(src, d, c.D);
    if (query || keys) {
      Turn<WIDE> t;
      t.load(a, norm, pos, d);
      raw.load_partners(a, src, d);
      transformed<DT, L, WIDE>(a, p, t, norm != nullptr, raw, d, y);
    } else {
      raw.values(d, c.D, y);
    }
  }
  if (query) return store_query<DT, WIDE>(a, row, head, d, y);
  const int64_t page = there ? find_page(a.r, c, seq, pos) : -1;
  if (page < 0) return;
  const int ts = (int)(pos & 15);
  const int64_t unit = c.unit(page, head, (int)(pos & (((int64_t)1 << c.page_shift) - 1)));
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

// Keys whose pairs lie in two threads of cache_append_prompts.hip: 64 positions of a
// sequence (find_store_block), one head, L lanes a row.
template <int DT, int L, bool WIDE>
__device__ __forceinline__ void append_keys(const AppendArgs& a, const AppendPlan& p, int64_t block) {
  const CacheView& c = a.c;
  const int head = (int)(block % c.heads);
  StoreBlock w;
  if (!find_store_block(a.r, (int)(block / c.heads), LaneSearch{}, &w)) return;
  const int lane = threadIdx.x & (L - 1), d = 8 * lane;
#pragma unroll 1
  for (int token = threadIdx.x / L; token < 64; token += 256 / L) {
    const int64_t pos = w.base + token, at = pos - w.p0;
    if (at < 0 || at >= w.rows || !position_there(a, pos)) continue;               // the same for the L lanes
    const int64_t page = find_page(a.r, c, w.b, pos);
    if (page < 0) continue;
    const int64_t unit = c.unit(page, head, (int)(pos & (((int64_t)1 << c.page_shift) - 1)));
    const Bits<DT>* const src = at_row<DT>(p.k, w.first + at, head);
    Raw<DT, WIDE> raw;
    raw.load(src, d, c.D);
    raw.load_partners(a, src, d);
    Turn<WIDE> t;
    t.load(a, a.k_norm, pos, d);
    float y[8];
    transformed<DT, L, WIDE>(a, p, t, a.k_norm != nullptr, raw, d, y);
    const Codes q = codes_of(a, p, d, y);
    store_scale(a, p, q, true, unit, token & 15, lane);
    store_key(c, q, unit, token & 15, lane);
  }
}

// Rows of queries, L lanes a row, several heads in turn.
template <int DT, int L, bool WIDE>
__device__ __forceinline__ void append_queries(const AppendArgs& a, const AppendPlan& p, int64_t block) {
  const int chunks = (a.q_heads + p.heads_per_block - 1) / p.heads_per_block;
  const int64_t row = block / chunks * (256 / L) + threadIdx.x / L;
  const int head0 = (int)(block % chunks) * p.heads_per_block;
  const int head1 = head0 + p.heads_per_block < a.q_heads ? head0 + p.heads_per_block : a.q_heads;
  const int d = (threadIdx.x & (L - 1)) * 8;
  int seq = 0;
  int64_t pos = -1;
  if (row >= a.r.rows || !find_row(a.r, row, &seq, &pos)) return;                  // the same for the L lanes
  const bool there = position_there(a, pos);
  Turn<WIDE> t;
  t.load(a, a.q_norm, there ? pos : 0, d);
  const Bits<DT>* src = at_row<DT>(p.q, row, head0);
  Raw<DT, WIDE> next;
  next.load(src, d, a.c.D);
  next.load_partners(a, src, d);
#pragma unroll 1
  for (int head = head0; head < head1; ++head) {
    const Raw<DT, WIDE> raw = next;
    src += head + 1 < head1 ? p.q.head_stride : 0;               // (the last one's again, for no one)
    next.load(src, d, a.c.D);
    next.load_partners(a, src, d);
    float y[8];
    transformed<DT, L, WIDE>(a, p, t, a.q_norm != nullptr, raw, d, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = there ? y[e] : 0.0f;
    store_query<DT, WIDE>(a, row, head, d, y);
  }
}

// The queries, and behind them the keys that cache_append_prompts.hip leaves.
template <int DT, int L, bool WIDE>
__global__ __launch_bounds__(256) void cache_append_steps_kernel(AppendArgs a, AppendPlan p) {
  const int64_t block = blockIdx.x;
  if (block < p.query_blocks) append_queries<DT, L, WIDE>(a, p, block);
  else append_keys<DT, L, WIDE>(a, p, block - p.query_blocks);
}

// ---------------------------------------------------------------- launches

template <int DT, int L, bool WIDE>
hipError_t launch_lanes(const AppendArgs& a, AppendPlan p, int dtype, hipStream_t stream) {
  constexpr int ROWS = 256 / L;
  // Row by row while that takes one short launch or a block of 64 positions would hold
  // few rows. Measured, row by row against by positions, 8 + 32 heads of 128: 8 sequences
  // of 32 rows 7 and 12 us, of 256 23 and 25, of 512 39 and 34, of 2000 185 and 108; 64
  // of 48 33 and 41, of 64 42 and 40; 512 of 16 86 and 96, of 24 148 and 123.
  const int64_t items = a.r.rows * (a.q_heads + 2 * a.c.heads);
  if (!a.r.starts || a.r.rows < 20 * (int64_t)a.r.batch || items * a.c.D <= 20000000) {
    hipLaunchKernelGGL((cache_append_rows_kernel<DT, L, WIDE>), dim3((unsigned)((items + ROWS - 1) / ROWS)), dim3(256), 0,
                       stream, a, p);
    return hipGetLastError();
  }
  const bool keys = WIDE && keys_in_thread(a);
  const hipError_t e = launch_cache_append_prompts(a, p, dtype, keys, stream);
  if (e != hipSuccess) return e;
  // Several heads a block, which share cosines and sines, as long as that leaves twice
  // the 2048 blocks that the GPU holds at once.
  const int64_t row_blocks = (a.r.rows + ROWS - 1) / ROWS;
  p.heads_per_block = 1;
  while (p.heads_per_block < 8 && row_blocks * (a.q_heads / (2 * p.heads_per_block)) >= 4096) p.heads_per_block *= 2;
  p.query_blocks = row_blocks * ((a.q_heads + p.heads_per_block - 1) / p.heads_per_block);
  const int64_t blocks = p.query_blocks + (keys ? 0 : store_units(a.r) * a.c.heads);
  hipLaunchKernelGGL((cache_append_steps_kernel<DT, L, WIDE>), dim3((unsigned)blocks), dim3(256), 0, stream, a, p);
  return hipGetLastError();
}

template <int DT, bool WIDE>
hipError_t launch_width(const AppendArgs& a, const AppendPlan& p, int dtype, hipStream_t stream) {
  if (a.c.C <= 2) return launch_lanes<DT, 8, WIDE>(a, p, dtype, stream);
  if (a.c.C <= 4) return launch_lanes<DT, 16, WIDE>(a, p, dtype, stream);
  return launch_lanes<DT, 32, WIDE>(a, p, dtype, stream);
}

template <int DT>
hipError_t launch_type(const AppendArgs& a, const AppendPlan& p, int dtype, hipStream_t stream) {
  const bool turn_wide = ((uintptr_t)a.q_norm | (uintptr_t)a.k_norm | (uintptr_t)a.rope) % 16 == 0 &&
                         (!a.rope || (a.half % 8 == 0 && a.rope_stride % 4 == 0));
  if (p.q.wide && p.k.wide && p.v.wide && turn_wide && (uintptr_t)a.out % 16 == 0)
    return launch_width<DT, true>(a, p, dtype, stream);
  return launch_width<DT, false>(a, p, dtype, stream);
}

}  // namespace

hipError_t launch_cache_append(const AppendArgs& a, int dtype, hipStream_t stream) {
  const int per16 = dtype == INT4DQ_ROWS_F32 ? 4 : 8;          // elements of 16 bytes
  auto rows = [&](const void* x, int64_t row_stride, int64_t head_stride) {
    const int wide = a.c.D % 8 == 0 && (uintptr_t)x % 16 == 0 && row_stride % per16 == 0 && head_stride % per16 == 0;
    return RowArray{const_cast<void*>(x), row_stride, head_stride, wide};
  };
  const int lanes = a.c.G > 1 ? a.c.group / 8 : a.c.C <= 2 ? 8 : a.c.C <= 4 ? 16 : 32;
  const AppendPlan p{rows(a.q, a.q_row_stride, a.q_head_stride), rows(a.k, a.k_row_stride, a.k_head_stride),
                     rows(a.v, a.v_row_stride, a.v_head_stride), lanes, 1.0 / a.c.D, 1, 0};
  if (dtype == INT4DQ_ROWS_F32) return launch_type<INT4DQ_ROWS_F32>(a, p, dtype, stream);
  if (dtype == INT4DQ_ROWS_F16) return launch_type<INT4DQ_ROWS_F16>(a, p, dtype, stream);
  return launch_type<INT4DQ_ROWS_BF16>(a, p, dtype, stream);
}

}  // namespace int4dq
