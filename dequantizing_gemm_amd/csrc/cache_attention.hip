// cache_attention.hip -- softmax attention over the 4-bit cache
// (include/int4dq_cache.h): the plan of a call, and the kernel that joins the
// partial results of tiles whose keys were shared out over several blocks. The
// attention kernel itself is in cache_attention_kernel.h.
#include "cache_attention_kernel.h"

namespace int4dq {

namespace {

// out = sum_i exp2(m_i - M) o_i / sum_i exp2(m_i - M) l_i over the chunks of the
// row's tile; one block for each (row, query head), blocks of rows that are
// whole already leave at once. A channel quadruple a thread, the chunks dealt to
// 256 / (8 C) groups of threads and joined through LDS.
template <int C>
__global__ __launch_bounds__(256) void cache_attention_join_kernel(AttentionArgs a, Schedule sched,
                                                                   const float* __restrict__ part) {
  constexpr int T = 8 * C, GROUPS = 256 / T;
  const int H = a.c.heads * a.ratio;
  __shared__ __attribute__((aligned(16))) float4_t sums[GROUPS][T];
  for (int64_t item = blockIdx.x; item < a.r.rows * H; item += gridDim.x) {
    const int64_t t = item / H;
    const int h = (int)(item % H), kh = h / a.ratio;
    BlockWork work;
    int first;
    const bool got = find_sequence(
        a, sched, [&](const SequenceWork& w, int, int, int) { return t >= w.first && t < w.first + w.rows; }, &work, &first);
    if (!got || work.chunks == 1) continue;       // the same for the whole block
    const int flat = (int)(t - work.w.first) * a.ratio + h % a.ratio;
    const int tile = flat / sched.tile_rows, in_tile = flat % sched.tile_rows;
    const int slot0 = work.slot + (work.w.tiles - 1 - tile) * work.chunks;
    const int64_t size = partial_floats(sched.tile_rows, C), next = size * a.c.heads;
    const float* const base = part + ((int64_t)slot0 * a.c.heads + kh) * size;
    const float* const ml = base + (int64_t)sched.tile_rows * 32 * C + 2 * in_tile;

    const int lane = threadIdx.x & (kWave - 1);
    float top = -1e30f;
    for (int i = lane; i < work.chunks; i += kWave) top = __builtin_fmaxf(top, ml[i * next]);
#pragma unroll
    for (int x = 1; x < kWave; x <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, x));
    float sum = 0.0f;
    for (int i = lane; i < work.chunks; i += kWave)
      sum += ml[i * next + 1] * __builtin_amdgcn_exp2f(ml[i * next] - top);
#pragma unroll
    for (int x = 1; x < kWave; x <<= 1) sum += __shfl_xor(sum, x);

    const int group = threadIdx.x / T, d = threadIdx.x % T * 4;
    float4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (group < GROUPS) {
#pragma unroll 4
      for (int i = group; i < work.chunks; i += GROUPS) {
        const float f = __builtin_amdgcn_exp2f(ml[i * next] - top);
        v += *reinterpret_cast<const float4_t*>(base + i * next + in_tile * (32 * C) + d) * f;
      }
    }
    __syncthreads();                              // the item before is read
    if (group < GROUPS) sums[group][threadIdx.x % T] = v;
    __syncthreads();
    if (threadIdx.x < T) {
      v = sums[0][threadIdx.x];
#pragma unroll
      for (int i = 1; i < GROUPS; ++i) v += sums[i][threadIdx.x];
      store_output(a, t * H + h, d, v * (sum == 0.0f ? 0.0f : 1.0f / sum));
    }
    if (threadIdx.x == 0 && a.lse)
      a.lse[t * H + h] = sum == 0.0f ? -__builtin_inff() : 0.69314718055994530942f * (top + __builtin_amdgcn_logf(sum));
  }
}

template <int C>
hipError_t launch_width(const AttentionArgs& a, const Schedule& s, float* part, hipStream_t stream) {
  hipError_t e = launch_attention_width<C>(a, s, part, stream);
  if (e != hipSuccess || s.target == 0) return e;
  hipLaunchKernelGGL(cache_attention_join_kernel<C>, dim3(stride_grid(a.r.rows * a.c.heads * a.ratio)), dim3(256), 0,
                     stream, a, s, part);
  return hipGetLastError();
}

}  // namespace

extern template hipError_t launch_attention_width<2>(const AttentionArgs&, const Schedule&, float*, hipStream_t);
extern template hipError_t launch_attention_width<3>(const AttentionArgs&, const Schedule&, float*, hipStream_t);
extern template hipError_t launch_attention_width<4>(const AttentionArgs&, const Schedule&, float*, hipStream_t);
extern template hipError_t launch_attention_width<6>(const AttentionArgs&, const Schedule&, float*, hipStream_t);
extern template hipError_t launch_attention_width<8>(const AttentionArgs&, const Schedule&, float*, hipStream_t);

int64_t cache_attention_workspace(const CacheView& c, const RowsView& r, int ratio) {
  const Schedule s = plan_of(c, r, ratio);
  return workspace_slots(s) * c.heads * partial_floats(s.tile_rows, c.C) * 4;
}

hipError_t launch_cache_attention(const AttentionArgs& a, void* workspace, int64_t workspace_bytes,
                                  hipStream_t stream) {
  Schedule s = plan_of(a.c, a.r, a.ratio);
  if (workspace_bytes < cache_attention_workspace(a.c, a.r, a.ratio)) {
    s.units -= s.target;
    s.target = 0;
  }
  float* const part = static_cast<float*>(workspace);
  switch (a.c.C) {
    case 2: return launch_width<2>(a, s, part, stream);
    case 3: return launch_width<3>(a, s, part, stream);
    case 4: return launch_width<4>(a, s, part, stream);
    case 6: return launch_width<6>(a, s, part, stream);
    default: return launch_width<8>(a, s, part, stream);
  }
}

}  // namespace int4dq
