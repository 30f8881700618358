// cache_attention_launch.h -- the choice among one width's forms of the
// attention kernel.
#pragma once

#include "cache_attention_kernel.h"

namespace int4dq {

template <int C, int GC, bool AFF>
void launch_attention_form(const AttentionArgs& a, const Schedule& s, const Workspace& ws, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)s.units * a.c.heads));
  if (s.tile_rows == kWideRows) {                    // plan_of asks for the forms that there are
    constexpr int QT = wide_tiles(C, C / GC, AFF);
    if constexpr (QT > 0)
      hipLaunchKernelGGL((cache_attention_wide_kernel<C, GC, QT, AFF>), grid, dim3(512 / QT), 0, stream, a, s, ws);
  } else if (s.tile_rows == 16) {
    hipLaunchKernelGGL((cache_attention_kernel<C, GC, 1, AFF>), grid, dim3(256), 0, stream, a, s, ws);
  } else if constexpr (max_tiles(C, C / GC, AFF) == 2) {
    hipLaunchKernelGGL((cache_attention_kernel<C, GC, 2, AFF>), grid, dim3(256), 0, stream, a, s, ws);
  }
}

template <int C, int GC>
void launch_attention_codes(const AttentionArgs& a, const Schedule& s, const Workspace& ws, hipStream_t stream) {
  if (a.c.k_zeros) launch_attention_form<C, GC, true>(a, s, ws, stream);
  else launch_attention_form<C, GC, false>(a, s, ws, stream);
}

template <int C>
hipError_t launch_attention_width(const AttentionArgs& a, const Schedule& s, const Workspace& ws, hipStream_t stream) {
  const int blocks = scale_blocks(a.c);
  if (blocks == C) launch_attention_codes<C, C>(a, s, ws, stream);
  if constexpr (C > 4 && C % 4 == 0)
    if (blocks == 4) launch_attention_codes<C, 4>(a, s, ws, stream);
  if constexpr (C > 2 && C % 2 == 0)
    if (blocks == 2) launch_attention_codes<C, 2>(a, s, ws, stream);
  if (blocks == 1) launch_attention_codes<C, 1>(a, s, ws, stream);
  return hipGetLastError();
}

}  // namespace int4dq
