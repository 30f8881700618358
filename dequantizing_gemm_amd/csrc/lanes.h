// lanes.h -- sums over a wavefront's lanes, and a search by all of them (whose steps
// are host code too, for checks without a GPU).
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

// A search by 64 lanes, 64 places at a time, so that up to 64 take one load and 4096
// two. below(from, apart, n): a bit for each lane l with l * apart < n and place
// from + l * apart at or below what is searched for.
template <typename B>
__host__ __device__ __forceinline__ int search_by_lanes(int n, B below) {
  int from = 0;
  while (n > 1) {
    const int apart = (n + kWave - 1) / kWave;
    const uint64_t bits = below(from, apart, n);
    const int at = bits ? 63 - __builtin_clzll(bits) : 0;
    from += at * apart;
    n = n - at * apart < apart ? n - at * apart : apart;
  }
  return from;
}

// The last i in [0, n) with f(i) <= x, where f does not decrease; 0 if there is
// none, and some i in range whatever f does.
template <typename F>
__device__ __forceinline__ int lane_search(int n, int64_t x, F f) {
  const int lane = threadIdx.x & (kWave - 1);
  return search_by_lanes(n, [&](int from, int apart, int left) -> uint64_t {
    return __ballot(lane * apart < left && f(from + lane * apart) <= x);
  });
}
struct LaneSearch {
  template <typename F>
  __device__ __forceinline__ int operator()(int n, int64_t x, F f) const { return lane_search(n, x, f); }
};

}  // namespace int4dq
