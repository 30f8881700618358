// cache_rows.h -- the caller's row-wise arrays as the kernels that write and read
// the 4-bit cache take them: elements of the three types, side by side or not.
#pragma once

#include <type_traits>

#include "cache.h"
#include "device_common.h"

#include "../../include/int4dq_cache.h"

namespace int4dq {

// Rows of queries, keys or values in the caller's arrays: what a launch takes.
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

}  // namespace int4dq
