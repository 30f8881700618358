// cache_attention_shared.hip -- attention over the 4-bit cache for a batch whose
// sequences begin with the same tokens (include/int4dq_cache_step.h).
//
// Mathematics: softmax attention over the union of two sets of keys is the sum of
// both parts' sums, each taken with its own reference m: with partial sums o_i and
// l_i over chunks i of either part, out = sum_i exp2(m_i - M) o_i / sum_i exp2(m_i - M) l_i.
//
// Work. The shared tokens are one sequence whose rows are those of the whole batch,
// side by side: a tile of 16, 32 or 128 of them reads and takes apart the shared codes
// once, where the sequences by themselves would do so for a tile of 16 each, of which
// one token fills only as many rows as there are query heads to a key head. Each
// sequence's own tokens are cut as in a call of its own. Both leave partial results, and
// one join adds them row by row: bound by the latency of a chain of four loads (64
// sequences, 32 query heads of 128, 15 chunks a row: 6.8 us).
//
// What bounds it (8 x 4 heads of 128, groups of 64, bfloat16, 64 sequences of 10 to 1500
// own tokens on 32768 shared ones, 95 us in all). The shared part in tiles of 32 rows 73 us,
// 470 TFLOP/s: the VALU, busy for 65% of it, which takes codes apart for four tiles of a
// head and block; in tiles of 128 it is 60 us and a longer join. The own part 23 us:
// latency, at most 24 steps of 64 tokens on four wavefronts. Both in one kernel, with
// tiles of 32 and 16 rows, was 92 us here, but 67 against 46 for 200 sequences of few own
// tokens, whose blocks then have the registers of the taller tiles.
#include "cache_attention_kernel.h"
#include "cache_parts.h"
#include "cache_step.h"

namespace int4dq {

namespace {

// A wavefront for each row of a tile of the own part; a block for each slot and head
// (those whose slot is no tile's first leave at once) and, in y, a share of the rows.
template <int C>
__global__ __launch_bounds__(256) void cache_attention_parts_kernel(AttentionArgs a, Schedule own, Workspace ws,
                                                                    Schedule shared, Workspace ws2) {
  constexpr int T = 8 * C, GROUPS = kWave / T;       // lanes for a row's channels, chunks at a time
  const int heads = a.c.heads, slot = blockIdx.x / heads, kh = blockIdx.x % heads;
  const PartRecord tile = ws.record[slot];           // read together with the counts
  const PartRecord all = ws2.record[0];
  const int used = *ws2.used;
  if (slot >= *ws.used || tile.chunk != 0) return;
  // starts that decrease can leave slots unwritten: whatever they hold stays inside the arrays
  if (tile.first < 0 || tile.flat0 < 0 || tile.flats < 0 || tile.chunks < 1 || tile.chunks > own.units - slot ||
      (int64_t)tile.first * a.ratio + tile.flats > a.r.rows * a.ratio)
    return;
  const bool has = used > 0 && used <= shared.units && all.chunks >= 1 && all.chunks <= used;
  const int chunks2 = has ? all.chunks : 0, tiles2 = has ? used / all.chunks : 0;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave, group = lane / T, d = lane % T * 4;
  const int64_t size = partial_floats(own.tile_rows, C), size2 = partial_floats(shared.tile_rows, C);
  const int rows = tile.flats - tile.flat0 < own.tile_rows ? tile.flats - tile.flat0 : own.tile_rows;
  const uint32_t ratio = a.ratio;
  for (int row = blockIdx.y * 4 + wave; row < rows; row += gridDim.y * 4) {
    const uint32_t flat = tile.flat0 + row;
    const int64_t token = tile.first + flat / ratio;
    const int64_t flat2 = (token - all.first) * ratio + flat % ratio;
    const int64_t tile2 = flat2 >= 0 ? flat2 / shared.tile_rows : -1;
    const int more = tile2 >= 0 && tile2 < tiles2 ? chunks2 : 0, n = tile.chunks + more;
    const int row2 = (int)(flat2 % shared.tile_rows);
    const int64_t slot2 = more ? (tiles2 - 1 - tile2) * chunks2 : 0;
    const float* const base = ws.part + ((int64_t)slot * heads + kh) * size;
    const float* const base2 = ws2.part + (slot2 * heads + kh) * size2;
    auto sums = [&](int i) {             // of chunk i
      return i < tile.chunks ? base + i * size * heads + row * (32 * C)
                             : base2 + (i - tile.chunks) * size2 * heads + row2 * (32 * C);
    };
    auto stats = [&](int i) {
      return i < tile.chunks ? base + i * size * heads + own.tile_rows * (32 * C) + 2 * row
                             : base2 + (i - tile.chunks) * size2 * heads + shared.tile_rows * (32 * C) + 2 * row2;
    };
    float top = -1e30f;
    for (int i = lane; i < n; i += kWave) top = __builtin_fmaxf(top, stats(i)[0]);
#pragma unroll
    for (int x = 1; x < kWave; x <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, x));
    float sum = 0.0f;
    for (int i = lane; i < n; i += kWave) sum += stats(i)[1] * __builtin_amdgcn_exp2f(stats(i)[0] - top);
    sum = lane_value(lane_scan(sum), kWave - 1);
    float4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (group < GROUPS) {
#pragma unroll 4
      for (int i = group; i < n; i += GROUPS)
        v += *reinterpret_cast<const float4_t*>(sums(i) + d) * __builtin_amdgcn_exp2f(stats(i)[0] - top);
    }
    float o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = o[e];
#pragma unroll
      for (int g = 1; g < GROUPS; ++g) o[e] += __shfl(x, lane + g * T);
      o[e] *= sum == 0.0f ? 0.0f : 1.0f / sum;
    }
    const int64_t at = token * heads * ratio + kh * ratio + flat % ratio;
    if (lane < T) store_output<4>(a, at, d, o);
    if (lane == 0 && a.lse) a.lse[at] = lse_of(top, sum);
  }
}

template <int C>
hipError_t launch_width(const AttentionArgs& whole, const Parts& p, const Workspace& ws, const Workspace& ws2,
                        hipStream_t stream) {
  AttentionArgs a = whole;
  a.part = kOwnPart;
  if (p.own.planned) {
    const hipError_t e = launch_cache_attention_plan(a, p.own, ws, stream);
    if (e != hipSuccess) return e;
  }
  // one launch where tiles are as high, so that the sequences' own tokens fill in; not with
  // the form for prompts, which fills the GPU (917 us together, 850 apart)
  const bool together = p.own.tile_rows == p.shared.tile_rows && p.own.tile_rows != kWideRows &&
                        ((int64_t)p.own.units + p.shared.units) * a.c.heads < (1 << 24);          // 2^32 threads
  const Second<true> second{together ? (unsigned)(p.shared.units * a.c.heads) : 0, p.shared, ws2};
  hipError_t e = launch_attention_width<C, true>(a, p.own, ws, second, stream);
  if (e != hipSuccess) return e;
  if (!together) {
    a.part = kSharedPart;
    a.all = a.r.batch;
    a.r.batch = 1;
    e = launch_attention_width<C, true>(a, p.shared, ws2, {}, stream);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(cache_attention_parts_kernel<C>, dim3((unsigned)(p.own.units * whole.c.heads), (unsigned)(p.own.tile_rows / 16)),
                     dim3(256), 0, stream, whole, p.own, ws, p.shared, ws2);
  return hipGetLastError();
}

}  // namespace

extern template hipError_t launch_attention_width<2, true>(const AttentionArgs&, const Schedule&, const Workspace&,
                                                    const Second<true>&, hipStream_t);
extern template hipError_t launch_attention_width<3, true>(const AttentionArgs&, const Schedule&, const Workspace&,
                                                    const Second<true>&, hipStream_t);
extern template hipError_t launch_attention_width<4, true>(const AttentionArgs&, const Schedule&, const Workspace&,
                                                    const Second<true>&, hipStream_t);
extern template hipError_t launch_attention_width<6, true>(const AttentionArgs&, const Schedule&, const Workspace&,
                                                    const Second<true>&, hipStream_t);
extern template hipError_t launch_attention_width<8, true>(const AttentionArgs&, const Schedule&, const Workspace&,
                                                    const Second<true>&, hipStream_t);

int64_t cache_attention_shared_workspace(const CacheView& c, const RowsView& r, int ratio, int64_t from) {
  return parts_workspace(c, r, ratio, from);
}

hipError_t launch_cache_attention_shared(const AttentionArgs& args, int64_t from, void* workspace, int64_t bytes,
                                         hipStream_t stream) {
  Parts p;
  if (!plan_parts(args.c, args.r, args.ratio, from, &p) || bytes < p.bytes())
    return launch_cache_attention(args, workspace, bytes, stream);
  AttentionArgs a = args;
  a.least_shared = p.from;
  const Workspace ws = workspace_at(workspace, p.own, a.c.heads, a.c.C);
  const Workspace ws2 = workspace_at(static_cast<uint8_t*>(workspace) + p.own_bytes, p.shared, a.c.heads, a.c.C);
  switch (a.c.C) {
    case 2: return launch_width<2>(a, p, ws, ws2, stream);
    case 3: return launch_width<3>(a, p, ws, ws2, stream);
    case 4: return launch_width<4>(a, p, ws, ws2, stream);
    case 6: return launch_width<6>(a, p, ws, ws2, stream);
    default: return launch_width<8>(a, p, ws, ws2, stream);
  }
}

}  // namespace int4dq
