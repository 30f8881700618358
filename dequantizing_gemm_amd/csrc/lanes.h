// lanes.h -- sums over a wavefront's lanes, and a search by all of them.
#pragma once

#include <type_traits>

#include "device_common.h"

namespace int4dq {

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

// The largest over the lanes, of numbers from 0 up.
__device__ __forceinline__ int lane_max(int v) {
#pragma unroll
  for (int x = 1; x < kWave; x <<= 1) {
    const int o = __shfl_xor(v, x);
    v = o > v ? o : v;
  }
  return __builtin_amdgcn_readfirstlane(v);
}

// The last i in [0, n) with f(i) <= x, where f does not decrease; 0 if there is
// none, and some i in range whatever f does. The lanes try 64 places at a time, so
// that up to 64 take one load and 4096 two.
template <typename F>
__device__ __forceinline__ int lane_search(int n, int64_t x, F f) {
  const int lane = threadIdx.x & (kWave - 1);
  int from = 0;
  while (n > 1) {
    const int apart = (n + kWave - 1) / kWave;
    const uint64_t below = __ballot(lane * apart < n && f(from + lane * apart) <= x);
    const int at = below ? 63 - __builtin_clzll(below) : 0;
    from += at * apart;
    n = n - at * apart < apart ? n - at * apart : apart;
  }
  return from;
}

}  // namespace int4dq
