// cache_attention.hip -- softmax attention over the 4-bit cache
// (include/int4dq_cache.h).
//
// One wavefront per (row, query head): 64 keys at a time, one a lane, their
// scores in binary32 with the running maximum and sum of the softmax; then each
// lane sums the values of its channels over those keys.
#include "cache.h"
#include "device_common.h"

namespace int4dq {

namespace {

__device__ __forceinline__ float row_value(const void* p, int64_t i, int bf16) {
  if (bf16) return __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  return (float)static_cast<const _Float16*>(p)[i];
}

__device__ __forceinline__ float code_value(uint32_t byte, int odd, const uint8_t* zeros, int64_t at) {
  const uint32_t u = (byte >> (4 * odd)) & 15u;
  return zeros ? (float)((int)u - (int)zeros[at]) : (float)sx4(u);
}

__global__ __launch_bounds__(64) void cache_attention_kernel(AttentionArgs a) {
  const CacheView& c = a.c;
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y, kh = h / a.ratio, DB = c.row_bytes();
  int b;
  int64_t pos;
  if (!find_row(a.r, t, &b, &pos)) return;
  int64_t hi = a.r.lengths[b];
  if (a.causal && pos + 1 < hi) hi = pos + 1;
  if (hi > a.r.max_pages << c.page_shift) hi = a.r.max_pages << c.page_shift;
  const int64_t lo = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
  __shared__ float q[kMaxHeadDim], p[64];
  __shared__ int64_t units[64];
  for (int d = lane; d < c.D; d += 64) q[d] = row_value(a.q, t * a.q_row_stride + h * a.q_head_stride + d, a.bf16);
  __syncthreads();
  float m = -__builtin_inff(), l = 0.0f, o[kMaxHeadDim / 64] = {};
  for (int64_t j0 = lo; j0 < hi; j0 += 64) {
    const int64_t j = j0 + lane;
    const int64_t page = j < hi ? find_page(a.r, c, b, j) : -1;
    const int slot = (int)(j & (((int64_t)1 << c.page_shift) - 1)), ts = slot & 15;
    const int64_t unit = page >= 0 ? c.unit(page, kh, slot) : -1;
    float s = -__builtin_inff();
    if (unit >= 0) {
      float acc = 0.0f;
      for (int d = 0; d < c.D; ++d) {
        const int64_t at = (unit * c.G + d / c.group) * 16 + ts;
        const uint32_t byte = c.k_packed[unit * 16 * DB + ts * DB + 4 * c.C * (d % 32 / 8) + 4 * (d / 32) + d % 8 / 2];
        acc += q[d] * (code_value(byte, d % 2, c.k_zeros, at) * half_bits_to_float(c.k_scales[at]));
      }
      s = acc * a.scale;
    }
    float top = s;
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, x));
    top = __builtin_fmaxf(top, m);
    if (top == -__builtin_inff()) continue;
    const float alpha = expf(m - top), e = expf(s - top);
    m = top;
    float sum = e;
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) sum += __shfl_xor(sum, x);
    l = l * alpha + sum;
    __syncthreads();
    p[lane] = e;
    units[lane] = unit;
    __syncthreads();
    for (int i = 0; i < kMaxHeadDim / 64; ++i) {
      const int d = lane + 64 * i;
      if (d >= c.D) break;
      o[i] *= alpha;
      for (int n = 0; n < 64; ++n) {
        const int64_t un = units[n];
        if (un < 0) continue;
        const int tn = (int)((j0 + n) & 15);
        const int64_t at = (un * c.G + d / c.group) * 16 + tn;
        const uint32_t byte = c.v_packed[un * 16 * DB + (d / 2) * 16 + tn];
        o[i] += p[n] * (code_value(byte, d % 2, c.v_zeros, at) * half_bits_to_float(c.v_scales[at]));
      }
    }
  }
  const int H = c.heads * a.ratio;
  for (int i = 0; i < kMaxHeadDim / 64; ++i) {
    const int d = lane + 64 * i;
    if (d >= c.D) break;
    const float v = l > 0.0f ? o[i] / l : 0.0f;
    const int64_t at = (t * H + h) * c.D + d;
    if (a.bf16) {
      const uint32_t u = __builtin_bit_cast(uint32_t, v);
      static_cast<uint16_t*>(a.out)[at] = (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
    } else {
      static_cast<_Float16*>(a.out)[at] = (_Float16)v;
    }
  }
  if (a.lse && lane == 0) a.lse[t * H + h] = l > 0.0f ? m + logf(l) : -__builtin_inff();
}

}  // namespace

hipError_t launch_cache_attention(const AttentionArgs& a, void*, int64_t, hipStream_t stream) {
  hipLaunchKernelGGL(cache_attention_kernel, dim3((unsigned)a.r.rows, (unsigned)(a.c.heads * a.ratio)), dim3(64), 0,
                     stream, a);
  return hipGetLastError();
}

int64_t cache_attention_workspace(const CacheView&, const RowsView&, int) { return 0; }

}  // namespace int4dq
