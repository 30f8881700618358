// cache_store.hip -- writing keys and values into the 4-bit cache and reading
// them back (include/int4dq_cache.h).
//
// Mathematics: the group quantizer of quantize.hip on rows of head_dim
// channels, one row per (token, head) of the keys and of the values. Bound by
// memory.
//
// Work decomposition: a block of 256 threads takes 64 positions (a step: four of
// the cache's 16-token units) of one head of one sequence, blockIdx.z the keys
// or the values. For quantising, thread 4 t + a owns channels 32 i + 8 a .. + 7 of
// token t for all i: its key codes are then 4 C adjacent bytes of the cache, and
// a group's extremes are the thread's own and a DPP butterfly over the token's four
// threads. Value codes, whose bytes lie a token apart, go through LDS and leave as
// 16-byte rows of a unit; a unit of which some tokens are not written (a run's
// ragged ends) leaves byte by byte. Reading back, a thread takes 4 C bytes of a
// token's key row, or one 16-token byte row of the values (two channels of 16
// tokens), so that a wavefront's stores cover whole rows.
#include <type_traits>

#include "cache.h"
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

// ---------------------------------------------------------------- the block's share

// 64 positions from `base` of sequence b; its rows start at position p0 with row
// `first` of the call, `rows` of them.
struct StoreBlock {
  int b, first, rows;
  int64_t p0, base;
};

__device__ __forceinline__ int lane_sum_upto(int v) {          // inclusive, over the wavefront
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int x = __shfl_up(v, o);
    if ((int)(threadIdx.x & (kWave - 1)) >= o) v += x;
  }
  return v;
}

__device__ __forceinline__ StoreBlock store_rows(const RowsView& r, int b) {
  const int s0 = r.starts ? r.starts[b] : b, s1 = r.starts ? r.starts[b + 1] : b + 1;
  StoreBlock x;
  x.b = b;
  x.first = s0 > 0 ? s0 : 0;
  const int last = s1 < r.rows ? s1 : (int)r.rows;
  x.rows = last > x.first ? last - x.first : 0;
  x.p0 = (int64_t)r.lengths[b] - s1 + x.first;
  x.base = (x.p0 >> 6) << 6;
  return x;
}

// Steps that a sequence's rows touch. Over a batch they number at most
// rows / 64 + 2 batch, the grid's size; without starts, one row touches one.
__device__ __forceinline__ int store_steps(const StoreBlock& x) {
  return x.rows > 0 ? (int)(((x.p0 + x.rows - 1) >> 6) - (x.p0 >> 6)) + 1 : 0;
}

__device__ __forceinline__ bool find_store_block(const RowsView& r, int unit, StoreBlock* out) {
  if (!r.starts) {
    *out = store_rows(r, unit);
    return true;
  }
  const int lane = threadIdx.x & (kWave - 1);
  int before = 0;
  for (int b0 = 0; b0 < r.batch; b0 += kWave) {
    const int steps = b0 + lane < r.batch ? store_steps(store_rows(r, b0 + lane)) : 0;
    const int upto = before + lane_sum_upto(steps);
    const uint64_t hit = __ballot(unit >= upto - steps && unit < upto);
    if (hit) {
      const int at = __builtin_ctzll(hit);
      *out = store_rows(r, b0 + at);
      out->base += (int64_t)(unit - __builtin_amdgcn_readlane(upto - steps, at)) * 64;
      return true;
    }
    before = __builtin_amdgcn_readlane(upto, kWave - 1);
  }
  return false;
}

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

// ---------------------------------------------------------------- write

template <int DT, int C, bool AFF>
__global__ __launch_bounds__(256) void cache_write_kernel(CacheView c, RowsView r, RowArray keys, RowArray values) {
  constexpr int DB = 16 * C;
  StoreBlock w;
  if (!find_store_block(r, blockIdx.x, &w)) return;
  const int head = blockIdx.y, tid = threadIdx.x, token = tid >> 2, a = tid & 3;
  const bool is_keys = blockIdx.z == 0;
  const RowArray in = is_keys ? keys : values;
  uint8_t* const packed = is_keys ? c.k_packed : c.v_packed;
  uint16_t* const scales = is_keys ? c.k_scales : c.v_scales;
  uint8_t* const zeros = is_keys ? c.k_zeros : c.v_zeros;

  const int64_t pos = w.base + token, at_row = pos - w.p0;
  const int64_t page = at_row >= 0 && at_row < w.rows ? find_page(r, c, w.b, pos) : -1;
  const bool there = page >= 0;

  // --- the thread's channels, 0 where there are none
  Bits<DT> raw[C][8];
  const Bits<DT>* const src = static_cast<const Bits<DT>*>(in.p) + (w.first + (there ? at_row : 0)) * in.row_stride +
                              head * in.head_stride;
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

  // --- extremes of each block of 32 channels, then of each group
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
  uint32_t word[C];
  const int slot = (int)(pos & (((int64_t)1 << c.page_shift) - 1)), ts = slot & 15;
  const int64_t unit = c.unit(page, head, slot);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int g = blocks == C ? 0 : i / blocks, from = g * blocks;
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
    word[i] = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = value_of<DT>(raw[i][e]);
      const uint32_t u = AFF ? affine_code(x, sf, rsf, zp) : code_of(x, sf, rsf);
      // padding channels have code 0
      if (!AFF || 32 * i + 8 * a + e < c.D) word[i] |= u << (4 * e);
    }
    if (there && a == 0 && i == from && g < c.G) {
      scales[(unit * c.G + g) * 16 + ts] = __builtin_bit_cast(uint16_t, s16);
      if constexpr (AFF) zeros[(unit * c.G + g) * 16 + ts] = (uint8_t)zp;
    }
  }

  if (is_keys) {
    if (there) {
      uint32_t* const to = reinterpret_cast<uint32_t*>(packed + unit * (16 * DB) + ts * DB + a * 4 * C);
#pragma unroll
      for (int i = 0; i < C; ++i) to[i] = word[i];
    }
    return;
  }
  // --- values: bytes to [unit][channel pair][token]
  __shared__ __attribute__((aligned(16))) uint8_t bytes[4 * DB * 16];
  __shared__ int64_t units[4];
  __shared__ uint32_t written[4];                    // a bit for each token of the unit
  const uint64_t tokens = __ballot(there);           // lanes 4 t + a: a wavefront is a unit
  if ((tid & (kWave - 1)) == 0) {
    uint32_t bits = 0;
#pragma unroll
    for (int t = 0; t < 16; ++t) bits |= (uint32_t)((tokens >> (4 * t)) & 1) << t;
    written[tid >> 6] = bits;
  }
  if (there) units[tid >> 6] = unit;                 // the same for all its tokens
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      bytes[(token >> 4) * (DB * 16) + (16 * i + 4 * a + k) * 16 + (token & 15)] = (uint8_t)(word[i] >> (8 * k));
  __syncthreads();
  for (int it = tid; it < 4 * DB; it += 256) {
    const int u = it / DB, j = it % DB;
    const uint32_t mask = written[u];
    if (mask == 0) continue;
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(&bytes[it * 16]);
    uint8_t* const to = packed + units[u] * (16 * DB) + j * 16;
    if (mask == 0xFFFFu) {
      *reinterpret_cast<u32x4_t*>(to) = v;
    } else {
#pragma unroll
      for (int t = 0; t < 16; ++t)
        if ((mask >> t) & 1u) to[t] = (uint8_t)(v[t / 4] >> (8 * (t % 4)));
    }
  }
}

// ---------------------------------------------------------------- read

template <int DT, int C, bool AFF>
__global__ __launch_bounds__(256) void cache_read_kernel(CacheView c, RowsView r, RowArray keys, RowArray values) {
  constexpr int DB = 16 * C;
  StoreBlock w;
  if (!find_store_block(r, blockIdx.x, &w)) return;
  const int head = blockIdx.y, tid = threadIdx.x;
  if (blockIdx.z == 0) {
    const int token = tid >> 2, a = tid & 3;
    const int64_t pos = w.base + token, at_row = pos - w.p0;
    if (at_row < 0 || at_row >= w.rows) return;
    const int64_t page = find_page(r, c, w.b, pos);
    const int slot = (int)(pos & (((int64_t)1 << c.page_shift) - 1)), ts = slot & 15;
    const int64_t unit = page < 0 ? 0 : c.unit(page, head, slot);
    const uint32_t* const from = reinterpret_cast<const uint32_t*>(c.k_packed + unit * (16 * DB) + ts * DB + a * 4 * C);
    Bits<DT>* const to = static_cast<Bits<DT>*>(keys.p) + (w.first + at_row) * keys.row_stride + head * keys.head_stride;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int d = 32 * i + 8 * a;
      if (d >= c.D) break;
      const uint32_t word = from[i];
      const int64_t at = (unit * c.G + d / c.group) * 16 + ts;
      const float s = half_bits_to_float(c.k_scales[at]);
      const int zp = AFF ? c.k_zeros[at] : 0;
      Pack<Bits<DT>, 8> out;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t u = (word >> (4 * e)) & 15u;
        out.v[e] = bits_of<DT>(page < 0 ? 0.0f : (float)(AFF ? (int)u - zp : sx4(u)) * s);
      }
      if (keys.wide) {
        *reinterpret_cast<Pack<Bits<DT>, 8>*>(to + d) = out;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (d + e < c.D) to[d + e] = out.v[e];
      }
    }
    return;
  }
  for (int it = tid; it < 4 * DB; it += 256) {
    const int u = it / DB, j = it % DB, d = 2 * j;
    const int64_t pos0 = w.base + 16 * u, row0 = pos0 - w.p0;
    if (d >= c.D || row0 + 15 < 0 || row0 >= w.rows) continue;
    const int64_t page = find_page(r, c, w.b, pos0);
    const int slot = (int)(pos0 & (((int64_t)1 << c.page_shift) - 1));
    const int64_t unit = page < 0 ? 0 : c.unit(page, head, slot);
    const u32x4_t bytes = *reinterpret_cast<const u32x4_t*>(c.v_packed + unit * (16 * DB) + j * 16);
    const int64_t at = (unit * c.G + d / c.group) * 16;
    const u32x4_t s0 = *reinterpret_cast<const u32x4_t*>(c.v_scales + at);
    const u32x4_t s1 = *reinterpret_cast<const u32x4_t*>(c.v_scales + at + 8);
    u32x4_t z = {0, 0, 0, 0};
    if constexpr (AFF) z = *reinterpret_cast<const u32x4_t*>(c.v_zeros + at);
    Bits<DT>* const to = static_cast<Bits<DT>*>(values.p) + (w.first + row0) * values.row_stride + head * values.head_stride + d;
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      const uint32_t b = (bytes[t / 4] >> (8 * (t % 4))) & 0xFFu;
      const float s = half_bits_to_float((uint16_t)((t < 8 ? s0[t / 2] : s1[t / 2 - 4]) >> (16 * (t % 2))));
      const int zp = AFF ? (z[t / 4] >> (8 * (t % 4))) & 0xFFu : 0;
      const int q0 = AFF ? (int)(b & 15u) - zp : sx4(b & 15u), q1 = AFF ? (int)(b >> 4) - zp : sx4(b >> 4);
      const Pack<Bits<DT>, 2> out = {bits_of<DT>(page < 0 ? 0.0f : (float)q0 * s),
                                     bits_of<DT>(page < 0 ? 0.0f : (float)q1 * s)};
      if (row0 + t < 0 || row0 + t >= w.rows) continue;
      if (values.wide) {
        *reinterpret_cast<Pack<Bits<DT>, 2>*>(to + t * values.row_stride) = out;
      } else {
        to[t * values.row_stride] = out.v[0];
        if (d + 1 < c.D) to[t * values.row_stride + 1] = out.v[1];
      }
    }
  }
}

// ---------------------------------------------------------------- launches

dim3 store_grid(const CacheView& c, const RowsView& r) {
  const int64_t units = r.starts ? r.rows / 64 + 2 * (int64_t)r.batch : r.batch;
  return dim3((unsigned)units, (unsigned)c.heads, 2);
}

template <int DT, int C>
void launch_store(bool write, const CacheView& c, const RowsView& r, const RowArray& k, const RowArray& v,
                  hipStream_t stream) {
  const dim3 grid = store_grid(c, r), block(256);
  if (write) {
    if (c.k_zeros) hipLaunchKernelGGL((cache_write_kernel<DT, C, true>), grid, block, 0, stream, c, r, k, v);
    else hipLaunchKernelGGL((cache_write_kernel<DT, C, false>), grid, block, 0, stream, c, r, k, v);
  } else {
    if (c.k_zeros) hipLaunchKernelGGL((cache_read_kernel<DT, C, true>), grid, block, 0, stream, c, r, k, v);
    else hipLaunchKernelGGL((cache_read_kernel<DT, C, false>), grid, block, 0, stream, c, r, k, v);
  }
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
