// cache_append_prompts.hip -- prompts' keys, normalised and rotated, and values on their way
// into the 4-bit cache (include/int4dq_cache_step.h), in the write kernel's
// arrangement: four threads a token, so that the norm's factor, a group's extremes and
// the places are found once for 8 C channels a thread, and both channels of a pair are
// in one thread. (The mathematics is in cache_append.hip.) 28114 tokens, 8 heads of 128,
// bfloat16: 73 us; with the lanes' arrangement of cache_append.hip and all in one launch
// the whole call took 233 us instead of 175.
#include "cache_append.h"
#include "cache_write.h"

namespace int4dq {

namespace {

// Normalised and rotated channels of a thread; 0 from head_dim on. Weights, cosines and
// sines lie 16-byte aligned, head_dim and half are multiples of 8.
template <int DT, int C>
__device__ __forceinline__ void transform_key(const AppendArgs& a, const AppendPlan& p, const Channels<DT, C>& x, int64_t pos,
                                              int lane4, float y[C][8]) {
#pragma clang fp contract(off)
  const int D = a.c.D, half = a.half;
  // Cosines and sines are asked for first, to come while the norm is summed. Halves: of
  // the pairs of blocks i and i + C / 2; interleaved: of block i's four pairs.
  constexpr int H = C / 2;
  float4_t c[C], s[C];
  const bool halves = C % 2 == 0 && !a.interleaved;
  if (a.rope) {
    const float* const row = a.rope + pos * a.rope_stride;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int d = 32 * (halves ? i / 2 : i) + 8 * lane4;
      const int at = halves ? d + 4 * (i % 2) : d < 2 * half ? d / 2 : 0;
      c[i] = *reinterpret_cast<const float4_t*>(row + at);
      s[i] = *reinterpret_cast<const float4_t*>(row + half + at);
    }
  }
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) y[i][e] = value_of<DT>(x.raw[i][e]);
  if (a.k_norm) {
    // in the order of cache_append.hip: 8 channels one after the other, then block by block
    // the four threads as four of its lanes, then the blocks pair by pair as its other steps
    double sum[8] = {};
#pragma unroll
    for (int i = 0; i < C; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[i] = __builtin_fma((double)y[i][e], (double)y[i][e], sum[i]);
      sum[i] = lanes_sum<4>(sum[i]);
    }
#pragma unroll
    for (int n = 4; n >= 1; n /= 2)
#pragma unroll
      for (int i = 0; i < n; ++i) sum[i] = sum[2 * i] + sum[2 * i + 1];         // (0 past C: the same)
    const float r = norm_factor(sum[0] * p.mean + a.eps);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int d = 32 * i + 8 * lane4;
      const float4_t* const w4 = reinterpret_cast<const float4_t*>(a.k_norm + (d < D ? d : 0));
      const float4_t w0 = w4[0], w1 = w4[1];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[i][e] = (y[i][e] * r) * (e < 4 ? w0[e % 4] : w1[e % 4]);
    }
  }
  if (!a.rope) return;
  if (!halves) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const bool turn = 32 * i + 8 * lane4 < 2 * half;
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float u = y[i][e], v = y[i][e + 1], ce = c[i][e / 2], se = s[i][e / 2];
        const float u0 = u * ce, u1 = v * se, v0 = v * ce, v1 = u * se;
        const float left = u0 - u1, right = v0 + v1;
        y[i][e] = turn ? left : u;
        y[i][e + 1] = turn ? right : v;
      }
    }
  } else if constexpr (C % 2 == 0) {                 // all channels, in halves of 16 C
#pragma unroll
    for (int i = 0; i < H; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float u = y[i][e], v = y[i + H][e], ce = c[2 * i + e / 4][e % 4], se = s[2 * i + e / 4][e % 4];
        const float u0 = u * ce, u1 = v * se, v0 = v * ce, v1 = u * se;
        y[i][e] = u0 - u1;
        y[i + H][e] = v0 + v1;
      }
  }
}

template <int DT, int C, bool AFF>
__device__ __forceinline__ void append_step(const AppendArgs& a, const AppendPlan& p, int block, int head, bool is_keys) {
  write_step<C, AFF>(a.c, a.r, block, head, is_keys, [&](int64_t pos) { return position_there(a, pos); },
                     [&](int64_t row, int64_t pos, int lane4, bool there) {
                       const RowArray& in = is_keys ? p.k : p.v;
                       Channels<DT, C> x;
                       x.load(a.c, at_row<DT>(in, row, head), in.wide, lane4, there);
                       if (!is_keys) return quantise<C, AFF>(a.c, lane4, [&](int i, int e) { return value_of<DT>(x.raw[i][e]); });
                       float y[C][8];
                       transform_key<DT, C>(a, p, x, there ? pos : 0, lane4, y);
                       return quantise<C, AFF>(a.c, lane4, [&](int i, int e) { return y[i][e]; });
                     });
}

// A row's heads and sides lie side by side in one projection's output, and are read
// together by blocks next to each other.
template <int DT, int C, bool AFF>
__global__ __launch_bounds__(256) void cache_append_prompts_kernel(AppendArgs a, AppendPlan p) {
  const int which = blockIdx.x % (2 * a.c.heads), head = which % a.c.heads;
  append_step<DT, C, AFF>(a, p, blockIdx.x / (2 * a.c.heads), head, which < a.c.heads);
}

template <int DT, int C, bool AFF>
__global__ __launch_bounds__(256) void cache_append_values_kernel(AppendArgs a, AppendPlan p) {
  append_step<DT, C, AFF>(a, p, blockIdx.x / a.c.heads, blockIdx.x % a.c.heads, false);
}

template <int DT, int C, bool AFF>
void launch_form(const AppendArgs& a, const AppendPlan& p, bool keys, hipStream_t stream) {
  const int64_t blocks = store_units(a.r) * a.c.heads;
  if (keys)
    hipLaunchKernelGGL((cache_append_prompts_kernel<DT, C, AFF>), dim3((unsigned)(2 * blocks)), dim3(256), 0, stream, a, p);
  else
    hipLaunchKernelGGL((cache_append_values_kernel<DT, C, AFF>), dim3((unsigned)blocks), dim3(256), 0, stream, a, p);
}

template <int DT, int C>
void launch_width(const AppendArgs& a, const AppendPlan& p, bool keys, hipStream_t stream) {
  if (a.c.k_zeros) launch_form<DT, C, true>(a, p, keys, stream);
  else launch_form<DT, C, false>(a, p, keys, stream);
}

template <int DT>
void launch_type(const AppendArgs& a, const AppendPlan& p, bool keys, hipStream_t stream) {
  switch (a.c.C) {
    case 2: return launch_width<DT, 2>(a, p, keys, stream);
    case 3: return launch_width<DT, 3>(a, p, keys, stream);
    case 4: return launch_width<DT, 4>(a, p, keys, stream);
    case 6: return launch_width<DT, 6>(a, p, keys, stream);
    default: return launch_width<DT, 8>(a, p, keys, stream);
  }
}

}  // namespace

hipError_t launch_cache_append_prompts(const AppendArgs& a, const AppendPlan& p, int dtype, bool keys, hipStream_t stream) {
  if (dtype == INT4DQ_ROWS_F32) launch_type<INT4DQ_ROWS_F32>(a, p, keys, stream);
  else if (dtype == INT4DQ_ROWS_F16) launch_type<INT4DQ_ROWS_F16>(a, p, keys, stream);
  else launch_type<INT4DQ_ROWS_BF16>(a, p, keys, stream);
  return hipGetLastError();
}

}  // namespace int4dq
