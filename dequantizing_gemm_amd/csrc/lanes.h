// lanes.h -- sums over a wavefront's lanes.
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

}  // namespace int4dq
