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
#include "cache_write.h"

namespace int4dq {

namespace {

// ---------------------------------------------------------------- write

template <int DT, int C, bool AFF>
__global__ __launch_bounds__(256) void cache_write_kernel(CacheView c, RowsView r, RowArray keys, RowArray values) {
  const int head = blockIdx.y;
  const bool is_keys = blockIdx.z == 0;
  write_step<C, AFF>(c, r, blockIdx.x, head, is_keys, [](int64_t) { return true; },
                     [&](int64_t row, int64_t, int a, bool there) {
                       const RowArray& in = is_keys ? keys : values;
                       Channels<DT, C> x;
                       x.load(c, static_cast<const Bits<DT>*>(in.p) + row * in.row_stride + head * in.head_stride, in.wide,
                              a, there);
                       return quantise<C, AFF>(c, a, [&](int i, int e) { return value_of<DT>(x.raw[i][e]); });
                     });
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
