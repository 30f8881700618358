// cache_attention_launch.h -- the choice among one width's forms of the
// attention kernel.
#pragma once

#include "cache_attention_kernel.h"

namespace int4dq {

template <int C, int GC, bool AFF, bool MORE>
void launch_attention_form(const AttentionArgs& a, const Schedule& s, const Workspace& ws,
                           const Second<MORE>& second, hipStream_t stream) {
  int64_t units = s.units;
  if constexpr (MORE)
    if (second.blocks > 0) units += second.sched.units;
  const dim3 grid((unsigned)(units * a.c.heads));
  if (s.tile_rows == kWideRows) {                    // plan_of asks for the forms that there are
    constexpr int QT = wide_tiles(C, C / GC, AFF);
    if constexpr (QT > 0)
      hipLaunchKernelGGL((cache_attention_wide_kernel<C, GC, QT, AFF, MORE>), grid, dim3(512 / QT), 0, stream, a, s, ws, second);
  } else if (s.tile_rows == 16) {
    hipLaunchKernelGGL((cache_attention_kernel<C, GC, 1, AFF, MORE>), grid, dim3(256), 0, stream, a, s, ws, second);
  } else if constexpr (max_tiles(C, C / GC, AFF) == 2) {
    hipLaunchKernelGGL((cache_attention_kernel<C, GC, 2, AFF, MORE>), grid, dim3(256), 0, stream, a, s, ws, second);
  }
}

template <int C, int GC, bool MORE>
void launch_attention_codes(const AttentionArgs& a, const Schedule& s, const Workspace& ws,
                           const Second<MORE>& second, hipStream_t stream) {
  if (a.c.k_zeros) launch_attention_form<C, GC, true, MORE>(a, s, ws, second, stream);
  else launch_attention_form<C, GC, false, MORE>(a, s, ws, second, stream);
}

template <int C, bool MORE>
hipError_t launch_attention_width(const AttentionArgs& a, const Schedule& s, const Workspace& ws,
                           const Second<MORE>& second, hipStream_t stream) {
  const int blocks = scale_blocks(a.c);
  if (blocks == C) launch_attention_codes<C, C, MORE>(a, s, ws, second, stream);
  if constexpr (C > 4 && C % 4 == 0)
    if (blocks == 4) launch_attention_codes<C, 4, MORE>(a, s, ws, second, stream);
  if constexpr (C > 2 && C % 2 == 0)
    if (blocks == 2) launch_attention_codes<C, 2, MORE>(a, s, ws, second, stream);
  if (blocks == 1) launch_attention_codes<C, 1, MORE>(a, s, ws, second, stream);
  return hipGetLastError();
}

}  // namespace int4dq
