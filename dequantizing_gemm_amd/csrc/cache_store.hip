// cache_store.hip -- writing keys and values into the 4-bit cache and reading
// them back (include/int4dq_cache.h).
//
// Mathematics: the group quantizer of quantize.hip on rows of head_dim
// channels, one row per (token, head) of the keys and of the values.
//
// Work decomposition: a lane owns 8 channels of a row, LP lanes a row (the
// power of two that holds 4 C), 256 threads a block of 16 or more consecutive
// rows of one head, blockIdx.z the keys or the values. A group's extremes are
// a DPP butterfly over its lanes. A lane's 8 key codes are 4 adjacent bytes of
// the token's row; its 8 value codes lie in 4 byte rows of the token's unit.
#include "cache.h"
#include "quantize_common.h"

#include "../../include/int4dq_cache.h"

namespace int4dq {

namespace {

template <int DT>
__device__ __forceinline__ float load_row(const void* p, int64_t i) {
  if constexpr (DT == INT4DQ_ROWS_F32) return static_cast<const float*>(p)[i];
  else if constexpr (DT == INT4DQ_ROWS_F16) return (float)static_cast<const _Float16*>(p)[i];
  else return __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

// Round to nearest even; the values here are finite.
__device__ __forceinline__ uint16_t bf16_bits(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

template <int DT>
__device__ __forceinline__ void store_row(void* p, int64_t i, float v) {
  if constexpr (DT == INT4DQ_ROWS_F32) static_cast<float*>(p)[i] = v;
  else if constexpr (DT == INT4DQ_ROWS_F16) static_cast<_Float16*>(p)[i] = (_Float16)v;
  else static_cast<uint16_t*>(p)[i] = bf16_bits(v);
}

struct RowArray {
  const void* p;
  int64_t row_stride, head_stride;
};

template <int DT, int LP, int LANES, bool AFF>
__global__ __launch_bounds__(256) void cache_write_kernel(CacheView c, RowsView r, RowArray k, RowArray v) {
  const int rl = threadIdx.x / LP, lane = threadIdx.x % LP;
  const int head = blockIdx.y;
  const bool keys = blockIdx.z == 0;
  const RowArray in = keys ? k : v;
  uint8_t* const packed = keys ? c.k_packed : c.v_packed;
  uint16_t* const scales = keys ? c.k_scales : c.v_scales;
  uint8_t* const zeros = keys ? c.k_zeros : c.v_zeros;
  const int64_t t = (int64_t)blockIdx.x * (256 / LP) + rl;
  int b;
  int64_t pos, page = -1;
  if (t < r.rows && find_row(r, t, &b, &pos)) page = find_page(r, c, b, pos);
  const int d0 = lane * 8;
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    x[e] = page >= 0 && d0 + e < c.D ? load_row<DT>(in.p, t * in.row_stride + head * in.head_stride + d0 + e) : 0.0f;
  uint32_t word = 0, zp = 0;
  _Float16 s16;
  if constexpr (!AFF) {
    float amax = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = __builtin_fmaxf(amax, __builtin_fabsf(x[e]));
    s16 = (_Float16)(run_umax_bits<LANES>(amax) / 7.0f);
    const float sf = (float)s16, rsf = scale_rcp(sf);
#pragma unroll
    for (int e = 0; e < 8; ++e) word |= code_of(x[e], sf, rsf) << (4 * e);
  } else {
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo = __builtin_fminf(lo, x[e]);
      hi = __builtin_fmaxf(hi, x[e]);
    }
    lo = run_umax_bits<LANES>(lo);
    hi = run_umax_bits<LANES>(hi);
    s16 = (_Float16)((hi - lo) / 15.0f);
    const float sf = (float)s16, rsf = scale_rcp(sf);
    zp = affine_zp(lo, sf);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (d0 + e < c.D) word |= affine_code(x[e], sf, rsf, zp) << (4 * e);
  }
  if (page < 0 || lane >= 4 * c.C) return;
  const int slot = (int)(pos & (((int64_t)1 << c.page_shift) - 1));
  const int64_t unit = c.unit(page, head, slot);
  const int DB = c.row_bytes(), ts = slot & 15;
  if (keys) {
    const int64_t at = unit * 16 * DB + ts * DB + (lane & 3) * 4 * c.C + (lane >> 2) * 4;
    *reinterpret_cast<uint32_t*>(packed + at) = word;
  } else {
    uint8_t* const at = packed + unit * 16 * DB + (int64_t)lane * 64 + ts;
#pragma unroll
    for (int j = 0; j < 4; ++j) at[16 * j] = (uint8_t)(word >> (8 * j));
  }
  if (lane % LANES == 0 && d0 < c.D) {
    const int64_t at = (unit * c.G + lane / LANES) * 16 + ts;
    scales[at] = __builtin_bit_cast(uint16_t, s16);
    if constexpr (AFF) zeros[at] = (uint8_t)zp;
  }
}

template <int DT, int LP>
__global__ __launch_bounds__(256) void cache_read_kernel(CacheView c, RowsView r, void* k, void* v) {
  const int rl = threadIdx.x / LP, lane = threadIdx.x % LP;
  const int head = blockIdx.y;
  const bool keys = blockIdx.z == 0;
  const int64_t t = (int64_t)blockIdx.x * (256 / LP) + rl;
  int b;
  int64_t pos;
  const int d0 = lane * 8;
  if (t >= r.rows || d0 >= c.D || !find_row(r, t, &b, &pos)) return;
  void* const out = keys ? k : v;
  const int64_t o = (t * c.heads + head) * c.D + d0;
  const int64_t page = find_page(r, c, b, pos);
  uint32_t word = 0, zp = 0;
  float s = 0.0f;
  const uint8_t* const zeros = keys ? c.k_zeros : c.v_zeros;
  if (page >= 0) {
    const int slot = (int)(pos & (((int64_t)1 << c.page_shift) - 1));
    const int64_t unit = c.unit(page, head, slot);
    const int DB = c.row_bytes(), ts = slot & 15;
    if (keys) {
      const int64_t at = unit * 16 * DB + ts * DB + (lane & 3) * 4 * c.C + (lane >> 2) * 4;
      word = *reinterpret_cast<const uint32_t*>(c.k_packed + at);
    } else {
      const uint8_t* const at = c.v_packed + unit * 16 * DB + (int64_t)lane * 64 + ts;
#pragma unroll
      for (int j = 0; j < 4; ++j) word |= (uint32_t)at[16 * j] << (8 * j);
    }
    const int64_t at = (unit * c.G + d0 / c.group) * 16 + ts;
    s = half_bits_to_float((keys ? c.k_scales : c.v_scales)[at]);
    if (zeros) zp = zeros[at];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t u = (word >> (4 * e)) & 15u;
    const int q = zeros ? (int)u - (int)zp : sx4(u);
    if (d0 + e < c.D) store_row<DT>(out, o + e, (float)q * s);
  }
}

template <int DT, int LP, int LANES>
void write_form(const CacheView& c, const RowsView& r, const RowArray& k, const RowArray& v, hipStream_t stream) {
  const dim3 grid((unsigned)((r.rows + 256 / LP - 1) / (256 / LP)), (unsigned)c.heads, 2);
  if (c.k_zeros) hipLaunchKernelGGL((cache_write_kernel<DT, LP, LANES, true>), grid, dim3(256), 0, stream, c, r, k, v);
  else hipLaunchKernelGGL((cache_write_kernel<DT, LP, LANES, false>), grid, dim3(256), 0, stream, c, r, k, v);
}

template <int DT, int LP>
void write_group(const CacheView& c, const RowsView& r, const RowArray& k, const RowArray& v, hipStream_t stream) {
  // one group: the butterfly runs over all lanes of the row
  const int lanes = c.G == 1 ? LP : c.group / 8;
  if (lanes == 4) write_form<DT, LP, 4>(c, r, k, v, stream);
  else if (lanes == 8) write_form<DT, LP, 8>(c, r, k, v, stream);
  else if constexpr (LP >= 16) {
    if (lanes == 16) write_form<DT, LP, 16>(c, r, k, v, stream);
    else write_form<DT, LP, LP>(c, r, k, v, stream);
  }
}

template <int DT>
void write_width(const CacheView& c, const RowsView& r, const RowArray& k, const RowArray& v, hipStream_t stream) {
  if (c.C == 2) write_group<DT, 8>(c, r, k, v, stream);
  else if (c.C <= 4) write_group<DT, 16>(c, r, k, v, stream);
  else write_group<DT, 32>(c, r, k, v, stream);
}

template <int DT>
void read_width(const CacheView& c, const RowsView& r, void* k, void* v, hipStream_t stream) {
  const int LP = c.C == 2 ? 8 : c.C <= 4 ? 16 : 32;
  const dim3 grid((unsigned)((r.rows + 256 / LP - 1) / (256 / LP)), (unsigned)c.heads, 2);
  if (LP == 8) hipLaunchKernelGGL((cache_read_kernel<DT, 8>), grid, dim3(256), 0, stream, c, r, k, v);
  else if (LP == 16) hipLaunchKernelGGL((cache_read_kernel<DT, 16>), grid, dim3(256), 0, stream, c, r, k, v);
  else hipLaunchKernelGGL((cache_read_kernel<DT, 32>), grid, dim3(256), 0, stream, c, r, k, v);
}

}  // namespace

hipError_t launch_cache_write(const CacheView& c, const RowsView& r, const void* k, int64_t k_row_stride,
                              int64_t k_head_stride, const void* v, int64_t v_row_stride, int64_t v_head_stride,
                              int dtype, hipStream_t stream) {
  const RowArray ka{k, k_row_stride, k_head_stride}, va{v, v_row_stride, v_head_stride};
  if (dtype == INT4DQ_ROWS_F32) write_width<INT4DQ_ROWS_F32>(c, r, ka, va, stream);
  else if (dtype == INT4DQ_ROWS_F16) write_width<INT4DQ_ROWS_F16>(c, r, ka, va, stream);
  else write_width<INT4DQ_ROWS_BF16>(c, r, ka, va, stream);
  return hipGetLastError();
}

hipError_t launch_cache_read(const CacheView& c, const RowsView& r, void* k, void* v, int dtype, hipStream_t stream) {
  if (dtype == INT4DQ_ROWS_F32) read_width<INT4DQ_ROWS_F32>(c, r, k, v, stream);
  else if (dtype == INT4DQ_ROWS_F16) read_width<INT4DQ_ROWS_F16>(c, r, k, v, stream);
  else read_width<INT4DQ_ROWS_BF16>(c, r, k, v, stream);
  return hipGetLastError();
}

}  // namespace int4dq
