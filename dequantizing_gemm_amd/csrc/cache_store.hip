// cache_store.hip -- writing keys and values into the 4-bit cache and reading
// them back (include/int4dq_cache.h).
//
// Mathematics: the group quantizer of quantize.hip on rows of head_dim
// channels, one row per (token, head) of the keys and of the values. Reading back
// is bound by memory (4 sequences of 9001 to 40961 tokens, 8 heads of 128, to
// bfloat16: 679 MB in 186 us, 3.7 TB/s), writing by the rounding's instructions (12
// prompts of 300 to 4100 tokens, 8 heads of 128, groups of 32 with zero points, from
// bfloat16: 58 us, the VALU busy for 74% of it), one token of one sequence by the
// chain of dependent loads (5 us either way).
//
// Work decomposition: a block of 256 threads takes 64 positions (a step: four of
// the cache's 16-token units) of a sequence, blockIdx.z the keys or the values, for
// one head or, when much is read back, several in turn: finding the step, its
// pages and their codes is a chain of dependent loads that one head's 20 KB would
// not pay for (131072 tokens: 227 us a head a block, 181 us with up to 8). For
// quantising, thread 4 t + a owns channels 32 i + 8 a .. + 7 of token t for all i:
// its key codes are then 4 C adjacent bytes of the cache, and a group's extremes
// are the thread's own and a DPP butterfly over the token's four threads. Value
// codes, whose bytes lie a token apart, go through LDS and leave as 16-byte rows of
// a unit; a unit of which some tokens are not written (a run's ragged ends) leaves
// byte by byte. Reading back, a thread takes 8 channels of a token's keys, so that a
// wavefront's store is 64 bytes (of two-byte elements) in each of 16 rows, or one
// 16-token byte row of the values (two channels of 16 tokens), whose stores cover
// whole rows.
#include <type_traits>

#include "cache.h"
#include "lanes.h"
#include "quantize_common.h"

#include "../../include/int4dq_cache.h"

namespace int4dq {

namespace {

// Keys or values in the caller's arrays: what a launch takes.
struct RowArray {
  void* p;
  int64_t row_stride, head_stride;
  int wide;                  // 8 channels lie 16-byte aligned (binary32: 32 bytes from a 16-byte boundary)
};

// ---------------------------------------------------------------- elements

template <int DT>
using Bits = typename std::conditional<DT == INT4DQ_ROWS_F32, uint32_t, uint16_t>::type;

template <int DT>
__device__ __forceinline__ float value_of(Bits<DT> v) {
  if constexpr (DT == INT4DQ_ROWS_F32) return __builtin_bit_cast(float, v);
  else if constexpr (DT == INT4DQ_ROWS_F16) return half_bits_to_float(v);
  else return __builtin_bit_cast(float, (uint32_t)v << 16);
}

// Rounded to nearest even; bfloat16 for finite values and infinities.
template <int DT>
__device__ __forceinline__ Bits<DT> bits_of(float v) {
  if constexpr (DT == INT4DQ_ROWS_F32) return __builtin_bit_cast(uint32_t, v);
  else if constexpr (DT == INT4DQ_ROWS_F16) return __builtin_bit_cast(uint16_t, (_Float16)v);
  else {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40u);
    return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
  }
}

// N adjacent elements from or to memory that is aligned to all of them (at most 16 bytes).
template <typename T, int N>
struct __attribute__((aligned(N * sizeof(T) < 16 ? N * sizeof(T) : 16))) Pack {
  T v[N];
};

// Past the caches' allocation: what is read back streams out.
template <typename T, int N>
__device__ __forceinline__ void store_nt(T* p, const Pack<T, N>& v) {
  if constexpr (N * sizeof(T) == 4) __builtin_nontemporal_store(__builtin_bit_cast(uint32_t, v), reinterpret_cast<uint32_t*>(p));
  else if constexpr (N * sizeof(T) == 8) __builtin_nontemporal_store(__builtin_bit_cast(u32x2_t, v), reinterpret_cast<u32x2_t*>(p));
  else if constexpr (N * sizeof(T) == 16) __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, v), reinterpret_cast<u32x4_t*>(p));
  else *reinterpret_cast<Pack<T, N>*>(p) = v;
}

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

// ---------------------------------------------------------------- write

// Codes, scales and zero points of a thread's channels of one token.
template <int C>
struct Quantised {
  uint32_t word[C];
  uint16_t scale[C];         // of block i's group
  uint8_t zero[C];
};

template <int DT, int C, bool AFF>
__device__ __forceinline__ Quantised<C> quantise(const CacheView& c, const RowArray& in, int64_t row, int head, int a,
                                                 bool there) {
  Bits<DT> raw[C][8];        // 0 where there are no channels
  const Bits<DT>* const src = static_cast<const Bits<DT>*>(in.p) + row * in.row_stride + head * in.head_stride;
  if (in.wide) {
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
  // extremes of each block of 32 channels, then of each group
  float lo[C], hi[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    lo[i] = hi[i] = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = value_of<DT>(raw[i][e]);
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
    // code_of / affine_code of the 8 channels, with one branch around the divisions
    float code[8];
    bool near = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float t = value_of<DT>(raw[i][e]) * rsf, n = __builtin_rintf(t);
      near |= __builtin_fabsf(__builtin_fabsf(t - n) - 0.5f) < 0x1p-14f;         // near_half_integer(t)
      code[e] = AFF ? __builtin_fminf(__builtin_fmaxf(n + (float)zp, 0.0f), 15.0f)
                    : __builtin_fminf(__builtin_fmaxf(n, -8.0f), 7.0f);
    }
    if (__builtin_expect(near, 0)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = value_of<DT>(raw[i][e]);
        if (near_half_integer(x * rsf))
          code[e] = AFF ? (float)affine_code(x, sf, rsf, zp)
                        : __builtin_fminf(__builtin_fmaxf(__builtin_rintf(x / sf), -8.0f), 7.0f);   // IEEE division
      }
    }
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t u = (uint32_t)(int)code[e] & 15u;
      // padding channels have code 0
      word |= (!AFF || 32 * i + 8 * a + e < c.D ? u : 0u) << (4 * e);
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

template <int DT, int C, bool AFF>
__global__ __launch_bounds__(256) void cache_write_kernel(CacheView c, RowsView r, RowArray keys, RowArray values) {
  constexpr int DB = 16 * C;
  __shared__ __attribute__((aligned(16))) uint8_t bytes[4 * DB * 16];            // [unit][channel pair][token]
  __shared__ int64_t units[4];
  __shared__ uint32_t written[4];                    // a bit for each token of the unit
  StoreBlock w;
  if (!find_store_block(r, blockIdx.x, LaneSearch{}, &w)) return;
  find_units(c, r, w, units);
  const int tid = threadIdx.x, token = tid >> 2, a = tid & 3, ts = token & 15;
  const int64_t at_row = w.base + token - w.p0, unit0 = units[token >> 4];       // a wavefront is a unit
  const bool there = at_row >= 0 && at_row < w.rows && unit0 >= 0;
  const int64_t row = w.first + (there ? at_row : 0);
  const uint64_t tokens = __ballot(there);           // lanes 4 t + a
  if ((tid & (kWave - 1)) == 0) {
    uint32_t bits = 0;
#pragma unroll
    for (int t = 0; t < 16; ++t) bits |= (uint32_t)((tokens >> (4 * t)) & 1) << t;
    written[tid >> 6] = bits;
  }
  const int head = blockIdx.y;
  const int64_t up = (int64_t)head << (c.page_shift - 4), unit = unit0 + up;
  const bool is_keys = blockIdx.z == 0;
  if (tokens) {                                      // the same for the wavefront
    const Quantised<C> q = quantise<DT, C, AFF>(c, is_keys ? keys : values, row, head, a, there);
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

// ---------------------------------------------------------------- read

template <int DT, int C, bool AFF>
__global__ __launch_bounds__(256) void cache_read_kernel(CacheView c, RowsView r, RowArray keys, RowArray values,
                                                         int heads_per_block) {
  constexpr int DB = 16 * C;
  StoreBlock w;
  if (!find_store_block(r, blockIdx.x, LaneSearch{}, &w)) return;
  const int tid = threadIdx.x, slots = (1 << c.page_shift) - 1;
  const int head0 = blockIdx.y * heads_per_block;
  const int head1 = head0 + heads_per_block < c.heads ? head0 + heads_per_block : c.heads;
  const int page_units = 1 << (c.page_shift - 4);
  if (blockIdx.z == 0) {                             // thread: channels 32 i + 8 a .. of a token
    const int token = tid >> 2, a = tid & 3, ts = token & 15;
    const int64_t pos = w.base + token, at_row = pos - w.p0;
    if (at_row < 0 || at_row >= w.rows) return;
    const int64_t page = find_page(r, c, w.b, pos);
    int64_t unit = page < 0 ? 0 : c.unit(page, head0, (int)(pos & slots));
    Bits<DT>* to = static_cast<Bits<DT>*>(keys.p) + (w.first + at_row) * keys.row_stride + head0 * keys.head_stride;
#pragma unroll 1
    for (int head = head0; head < head1; ++head, to += keys.head_stride, unit += page < 0 ? 0 : page_units) {
      const uint32_t* const from = reinterpret_cast<const uint32_t*>(c.k_packed + unit * (16 * DB) + ts * DB + a * 4 * C);
      uint32_t word[C];
      uint16_t scale[C];
      uint8_t zero[C];
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int d = 32 * i + 8 * a;
        const int64_t at = (unit * c.G + (d < c.D ? d / c.group : 0)) * 16 + ts;
        word[i] = from[i];
        scale[i] = c.k_scales[at];
        zero[i] = AFF ? c.k_zeros[at] : (uint8_t)0;
      }
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int d = 32 * i + 8 * a;
        if (d >= c.D) break;
        const float s = half_bits_to_float(scale[i]);
        Pack<Bits<DT>, 8> out;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t u = (word[i] >> (4 * e)) & 15u;
          out.v[e] = bits_of<DT>(page < 0 ? 0.0f : (float)(AFF ? (int)u - (int)zero[i] : sx4(u)) * s);
        }
        if (keys.wide) {
          store_nt(to + d, out);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (d + e < c.D) to[d + e] = out.v[e];
        }
      }
    }
    return;
  }
  for (int it = tid; it < 4 * DB; it += 256) {       // thread: two channels of 16 tokens
    const int u = it / DB, j = it % DB, d = 2 * j;
    const int64_t pos0 = w.base + 16 * u, row0 = pos0 - w.p0;
    if (d >= c.D || row0 + 15 < 0 || row0 >= w.rows) continue;
    const int64_t page = find_page(r, c, w.b, pos0);
    int64_t unit = page < 0 ? 0 : c.unit(page, head0, (int)(pos0 & slots));
    const int first = row0 < 0 ? (int)-row0 : 0, last = w.rows - row0 < 16 ? (int)(w.rows - row0) : 16;
    Bits<DT>* at_head = static_cast<Bits<DT>*>(values.p) + (w.first + row0) * values.row_stride + head0 * values.head_stride + d;
#pragma unroll 1
    for (int head = head0; head < head1; ++head, at_head += values.head_stride, unit += page < 0 ? 0 : page_units) {
      const u32x4_t bytes = *reinterpret_cast<const u32x4_t*>(c.v_packed + unit * (16 * DB) + j * 16);
      const int64_t at = (unit * c.G + d / c.group) * 16;
      const u32x4_t s0 = *reinterpret_cast<const u32x4_t*>(c.v_scales + at);
      const u32x4_t s1 = *reinterpret_cast<const u32x4_t*>(c.v_scales + at + 8);
      u32x4_t z = {0, 0, 0, 0};
      if constexpr (AFF) z = *reinterpret_cast<const u32x4_t*>(c.v_zeros + at);
      Bits<DT>* to = at_head;
#pragma unroll
      for (int t = 0; t < 16; ++t, to += values.row_stride) {
        const uint32_t b = (bytes[t / 4] >> (8 * (t % 4))) & 0xFFu;
        const float s = half_bits_to_float((uint16_t)((t < 8 ? s0[t / 2] : s1[t / 2 - 4]) >> (16 * (t % 2))));
        const int zp = AFF ? (z[t / 4] >> (8 * (t % 4))) & 0xFFu : 0;
        const int q0 = AFF ? (int)(b & 15u) - zp : sx4(b & 15u), q1 = AFF ? (int)(b >> 4) - zp : sx4(b >> 4);
        const Pack<Bits<DT>, 2> out = {bits_of<DT>(page < 0 ? 0.0f : (float)q0 * s),
                                       bits_of<DT>(page < 0 ? 0.0f : (float)q1 * s)};
        if (t < first || t >= last) continue;
        if (values.wide) {
          store_nt(to, out);
        } else {
          to[0] = out.v[0];
          if (d + 1 < c.D) to[1] = out.v[1];
        }
      }
    }
  }
}

// ---------------------------------------------------------------- launches

template <int DT, int C>
void launch_store(bool write, const CacheView& c, const RowsView& r, const RowArray& k, const RowArray& v,
                  hipStream_t stream) {
  const int64_t units = store_units(r);
  const dim3 block(256);
  if (write) {
    const dim3 grid((unsigned)units, (unsigned)c.heads, 2);
    if (c.k_zeros) hipLaunchKernelGGL((cache_write_kernel<DT, C, true>), grid, block, 0, stream, c, r, k, v);
    else hipLaunchKernelGGL((cache_write_kernel<DT, C, false>), grid, block, 0, stream, c, r, k, v);
    return;
  }
  // Several heads a block as long as that leaves twice the 2048 blocks that the GPU
  // holds at once.
  int per = 1;
  while (per < 8 && per < c.heads && units * c.heads / per >= 4096) per *= 2;
  const dim3 grid((unsigned)units, (unsigned)((c.heads + per - 1) / per), 2);
  if (c.k_zeros) hipLaunchKernelGGL((cache_read_kernel<DT, C, true>), grid, block, 0, stream, c, r, k, v, per);
  else hipLaunchKernelGGL((cache_read_kernel<DT, C, false>), grid, block, 0, stream, c, r, k, v, per);
}

template <int DT>
void launch_width(bool write, const CacheView& c, const RowsView& r, const RowArray& k, const RowArray& v,
                  hipStream_t stream) {
  switch (c.C) {
    case 2: return launch_store<DT, 2>(write, c, r, k, v, stream);
    case 3: return launch_store<DT, 3>(write, c, r, k, v, stream);
    case 4: return launch_store<DT, 4>(write, c, r, k, v, stream);
    case 6: return launch_store<DT, 6>(write, c, r, k, v, stream);
    default: return launch_store<DT, 8>(write, c, r, k, v, stream);
  }
}

hipError_t launch_type(bool write, const CacheView& c, const RowsView& r, RowArray k, RowArray v, int dtype,
                       hipStream_t stream) {
  const int per16 = dtype == INT4DQ_ROWS_F32 ? 4 : 8;          // elements of 16 bytes
  for (RowArray* x : {&k, &v})
    x->wide = c.D % 8 == 0 && (uintptr_t)x->p % 16 == 0 && x->row_stride % per16 == 0 && x->head_stride % per16 == 0;
  if (dtype == INT4DQ_ROWS_F32) launch_width<INT4DQ_ROWS_F32>(write, c, r, k, v, stream);
  else if (dtype == INT4DQ_ROWS_F16) launch_width<INT4DQ_ROWS_F16>(write, c, r, k, v, stream);
  else launch_width<INT4DQ_ROWS_BF16>(write, c, r, k, v, stream);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_write(const CacheView& c, const RowsView& r, const void* k, int64_t k_row_stride,
                              int64_t k_head_stride, const void* v, int64_t v_row_stride, int64_t v_head_stride,
                              int dtype, hipStream_t stream) {
  return launch_type(true, c, r, RowArray{const_cast<void*>(k), k_row_stride, k_head_stride, 0},
                     RowArray{const_cast<void*>(v), v_row_stride, v_head_stride, 0}, dtype, stream);
}

hipError_t launch_cache_read(const CacheView& c, const RowsView& r, void* k, void* v, int dtype, hipStream_t stream) {
  const int64_t row = (int64_t)c.heads * c.D;
  return launch_type(false, c, r, RowArray{k, row, c.D, 0}, RowArray{v, row, c.D, 0}, dtype, stream);
}

}  // namespace int4dq
