// cache_append.h -- what the kernels of int4_cache_append share: the norm's factor, and
// what a launch takes.
#pragma once

#include "cache_rows.h"
#include "cache_step.h"
#include "lanes.h"

namespace int4dq {

// What the kernels take besides the caller's arguments.
struct AppendPlan {
  RowArray q, k, v;
  int group_lanes;           // lanes of a scale's group: 4, 8, 16 or 32
  double mean;               // 1 / head_dim
  int heads_per_block;       // prompts: query heads that a block takes in turn
  int64_t query_blocks;
};

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

__device__ __forceinline__ bool position_there(const AppendArgs& a, int64_t pos) {
  return pos >= 0 && (!a.rope || pos < a.positions);
}

template <int DT>
__device__ __forceinline__ const Bits<DT>* at_row(const RowArray& x, int64_t row, int head) {
  return static_cast<const Bits<DT>*>(x.p) + row * x.row_stride + head * x.head_stride;
}

// Prompts' values and, with `keys`, their keys: those whose pairs one thread has, WIDE.
inline bool keys_in_thread(const AppendArgs& a) {
  return !a.rope || a.interleaved || (a.c.C % 2 == 0 && a.half == 16 * a.c.C);
}
hipError_t launch_cache_append_prompts(const AppendArgs& a, const AppendPlan& p, int dtype, bool keys, hipStream_t stream);

}  // namespace int4dq
