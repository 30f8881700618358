// cache_attention_launch.h -- the choice among one width's forms of the
// attention kernel.
#pragma once

#include "cache_attention_kernel.h"

namespace int4dq {

template <int C, int GC, int QT>
void launch_attention_form(const AttentionArgs& a, const Schedule& s, const Workspace& ws, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)s.units * a.c.heads));
  if (a.c.k_zeros) hipLaunchKernelGGL((cache_attention_kernel<C, GC, QT, true>), grid, dim3(256), 0, stream, a, s, ws);
  else hipLaunchKernelGGL((cache_attention_kernel<C, GC, QT, false>), grid, dim3(256), 0, stream, a, s, ws);
}

// s.tile_rows is at most 16 max_tiles: plan_of sees to that.
template <int C, int GC>
void launch_attention_tile(const AttentionArgs& a, const Schedule& s, const Workspace& ws, hipStream_t stream) {
  constexpr int most = max_tiles(C, C / GC);
  if (s.tile_rows == 16) launch_attention_form<C, GC, 1>(a, s, ws, stream);
  if constexpr (most >= 2)
    if (s.tile_rows == 32) launch_attention_form<C, GC, 2>(a, s, ws, stream);
}

template <int C>
hipError_t launch_attention_width(const AttentionArgs& a, const Schedule& s, const Workspace& ws, hipStream_t stream) {
  const int blocks = scale_blocks(a.c);
  if (blocks == C) launch_attention_tile<C, C>(a, s, ws, stream);
  if constexpr (C > 4 && C % 4 == 0)
    if (blocks == 4) launch_attention_tile<C, 4>(a, s, ws, stream);
  if constexpr (C > 2 && C % 2 == 0)
    if (blocks == 2) launch_attention_tile<C, 2>(a, s, ws, stream);
  if (blocks == 1) launch_attention_tile<C, 1>(a, s, ws, stream);
  return hipGetLastError();
}

}  // namespace int4dq
