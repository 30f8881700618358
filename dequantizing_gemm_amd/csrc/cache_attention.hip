// cache_attention.hip -- softmax attention over the 4-bit cache
// (include/int4dq_cache.h): the plan of a call, and the kernel that joins the
// partial results of tiles whose keys were shared out over several blocks. The
// attention kernel itself is in cache_attention_kernel.h.
#include "cache_attention_kernel.h"

namespace int4dq {

namespace {

// The blocks and slots of the sequences before each, for batches that a wavefront
// does not look through at once: one block, a thread a sequence.
__global__ __launch_bounds__(1024) void cache_attention_plan_kernel(AttentionArgs a, Schedule sched, Workspace ws) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid >> 6;
  __shared__ float works[2][16];
  __shared__ int longest[16], adds[2][16];
  __shared__ PlanEntry sums[2][16];
  const bool parts = sched.partial && leaves_parts(a, sched);
  const SequenceWork own = tid < a.r.batch ? sequence_work(a, sched.tile_rows, tid) : SequenceWork{};
  auto of = [&](int b) { return b == tid ? own : sequence_work(a, sched.tile_rows, b); };
  float work = 0.0f, tiles = 0.0f;
  int most = 0;
  for (int b = tid; b < a.r.batch; b += 1024) {
    const SequenceWork w = of(b);
    work += (float)w.tiles * (float)w.steps;
    tiles += (float)w.tiles;
    most = w.tiles > 0 && w.steps > most ? w.steps : most;
  }
  work = lane_scan(work);
  tiles = lane_scan(tiles);
  most = lane_max(most);
  if (lane == kWave - 1) {
    works[0][wave] = work;
    works[1][wave] = tiles;
    longest[wave] = most;
  }
  __syncthreads();
  work = tiles = 0.0f;
  for (int i = 0; i < 16; ++i) {
    work += works[0][i];
    tiles += works[1][i];
    most = longest[i] > most ? longest[i] : most;
  }
  int turn = 0;
  const int per = steps_per_block(sched, work, tiles, most, [&](int x) {
    int sum = 0;
    for (int b = tid; b < a.r.batch; b += 1024) {
      const SequenceWork w = of(b);
      sum += w.tiles > 0 ? (chunks_of(w.steps, x) - 1) * w.tiles : 0;
    }
    sum = lane_scan(sum);
    if (lane == kWave - 1) adds[turn][wave] = sum;
    __syncthreads();                     // two buffers: the one written next was read before this
    sum = 0;
    for (int i = 0; i < 16; ++i) sum += adds[turn][i];
    turn ^= 1;
    return sum;
  });
  int blocks = 0, slots = 0;
  for (int b0 = 0; b0 < a.r.batch; b0 += 1024, turn ^= 1) {
    const int b = b0 + tid;
    int mine = 0, mine_slots = 0;
    if (b < a.r.batch) {
      const SequenceWork w = of(b);
      const int chunks = w.tiles > 0 ? chunks_of(w.steps, per) : 0;
      mine = chunks * w.tiles;
      mine_slots = chunks > 1 || parts ? mine : 0;
    }
    int upto = lane_scan(mine), slots_upto = lane_scan(mine_slots);
    if (lane == kWave - 1) sums[turn][wave] = PlanEntry{upto, slots_upto};
    __syncthreads();                     // (two buffers here too)
    upto += blocks;
    slots_upto += slots;
    for (int i = 0; i < 16; ++i) {
      const PlanEntry x = sums[turn][i];
      upto += i < wave ? x.blocks : 0;
      slots_upto += i < wave ? x.slots : 0;
      blocks += x.blocks;
      slots += x.slots;
    }
    if (b < a.r.batch) ws.plan[b] = PlanEntry{upto - mine, slots_upto - mine_slots};
  }
  if (tid == 0) {
    ws.plan[a.r.batch] = PlanEntry{blocks, slots};
    *ws.used = slots;
  }
}

// out = sum_i exp2(m_i - M) o_i / sum_i exp2(m_i - M) l_i over the chunks of a
// tile that was shared out, for each of its rows. One block for each slot and head
// (those whose slot is no tile's first leave at once) and, in y, a share of the
// tile's rows; a channel quadruple a thread, 256 / (8 C) groups of threads. Up to 8
// chunks: each group has a row of its own. More: the groups share out the chunks
// of one row and are joined through LDS.
template <int C>
__global__ __launch_bounds__(256) void cache_attention_join_kernel(AttentionArgs a, Schedule sched, Workspace ws) {
  constexpr int T = 8 * C, GROUPS = 256 / T;
  const int slot = blockIdx.x / a.c.heads, kh = blockIdx.x % a.c.heads;
  const PartRecord tile = ws.record[slot];          // read together with the count
  if (slot >= *ws.used || tile.chunk != 0) return;
  // starts that decrease can make more tiles than the grid has blocks, and leave
  // this slot unwritten: whatever it holds then stays inside the arrays
  if (tile.first < 0 || tile.flat0 < 0 || tile.flats < 0 || tile.chunks < 1 ||
      tile.chunks > workspace_slots(sched) - slot || (int64_t)tile.first * a.ratio + tile.flats > a.r.rows * a.ratio)
    return;
  const int64_t size = partial_floats(sched.tile_rows, C), next = size * a.c.heads;
  const float* const base = ws.part + ((int64_t)slot * a.c.heads + kh) * size;
  const int lane = threadIdx.x & (kWave - 1), group = threadIdx.x / T, d = threadIdx.x % T * 4;
  __shared__ __attribute__((aligned(16))) float4_t sums[GROUPS][T];
  const int rows = tile.flats - tile.flat0 < sched.tile_rows ? tile.flats - tile.flat0 : sched.tile_rows;
  const uint32_t ratio = a.ratio;
  if (tile.chunks <= 8) {
    for (int row = blockIdx.y * GROUPS + group; row < rows && group < GROUPS; row += gridDim.y * GROUPS) {
      const float* const ml = base + (int64_t)sched.tile_rows * 32 * C + 2 * row;
      float m[8], top = -1e30f, sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m[i] = ml[(i < tile.chunks ? i : 0) * next];
        top = __builtin_fmaxf(top, m[i]);
      }
      float4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < tile.chunks) {
          const float f = __builtin_amdgcn_exp2f(m[i] - top);
          sum += ml[i * next + 1] * f;
          v += *reinterpret_cast<const float4_t*>(base + i * next + row * (32 * C) + d) * f;
        }
      v *= sum == 0.0f ? 0.0f : 1.0f / sum;
      const uint32_t flat = tile.flat0 + row;
      const int64_t at = (int64_t)(tile.first + flat / ratio) * a.c.heads * ratio + kh * ratio + flat % ratio;
      const float o[4] = {v.x, v.y, v.z, v.w};
      store_output<4>(a, at, d, o);
      if (d == 0 && a.lse) a.lse[at] = lse_of(top, sum);
    }
    return;
  }
  for (int row = blockIdx.y; row < rows; row += gridDim.y) {
    const float* const ml = base + (int64_t)sched.tile_rows * 32 * C + 2 * row;
    float top = -1e30f;
    for (int i = lane; i < tile.chunks; i += kWave) top = __builtin_fmaxf(top, ml[i * next]);
#pragma unroll
    for (int x = 1; x < kWave; x <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, x));
    float sum = 0.0f;
    for (int i = lane; i < tile.chunks; i += kWave) sum += ml[i * next + 1] * __builtin_amdgcn_exp2f(ml[i * next] - top);
    sum = lane_value(lane_scan(sum), kWave - 1);

    float4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (group < GROUPS) {
#pragma unroll 4
      for (int i = group; i < tile.chunks; i += GROUPS) {
        const float f = __builtin_amdgcn_exp2f(ml[i * next] - top);
        v += *reinterpret_cast<const float4_t*>(base + i * next + row * (32 * C) + d) * f;
      }
      sums[group][threadIdx.x % T] = v;
    }
    __syncthreads();
    const uint32_t flat = tile.flat0 + row;
    const int64_t at = (int64_t)(tile.first + flat / ratio) * a.c.heads * ratio + kh * ratio + flat % ratio;
    if (threadIdx.x < T) {
      v = sums[0][threadIdx.x];
#pragma unroll
      for (int i = 1; i < GROUPS; ++i) v += sums[i][threadIdx.x];
      v *= sum == 0.0f ? 0.0f : 1.0f / sum;
      const float o[4] = {v.x, v.y, v.z, v.w};
      store_output<4>(a, at, d, o);
    }
    if (threadIdx.x == 0 && a.lse)
      a.lse[at] = lse_of(top, sum);
    __syncthreads();                                 // the sums are read
  }
}

}  // namespace

hipError_t launch_cache_attention_plan(const AttentionArgs& a, const Schedule& s, const Workspace& ws, hipStream_t stream) {
  hipLaunchKernelGGL(cache_attention_plan_kernel, dim3(1), dim3(1024), 0, stream, a, s, ws);
  return hipGetLastError();
}

namespace {

template <int C>
hipError_t launch_width(const AttentionArgs& a, const Schedule& s, const Workspace& ws, hipStream_t stream) {
  hipError_t e = s.planned ? launch_cache_attention_plan(a, s, ws, stream) : hipSuccess;
  if (e == hipSuccess)
    e = sink_end(a) > 0 ? launch_attention_width<C, true>(a, s, ws, {}, stream) : launch_attention_width<C, false>(a, s, ws, {}, stream);
  if (e != hipSuccess || s.target == 0) return e;
  // few tiles of many rows after a last round: more blocks for each (18 tiles in 7 chunks, 4
  // blocks 172 us with the attention, 16 blocks 166)
  const unsigned rows = s.last_round ? 16 : (unsigned)(a.r.starts || a.ratio > 4 ? 4 : a.ratio);
  hipLaunchKernelGGL(cache_attention_join_kernel<C>, dim3((unsigned)(workspace_slots(s) * a.c.heads), rows), dim3(256),
                     0, stream, a, s, ws);
  return hipGetLastError();
}

}  // namespace

extern template hipError_t launch_attention_width<2, false>(const AttentionArgs&, const Schedule&, const Workspace&,
                                                    const Second<false>&, hipStream_t);
extern template hipError_t launch_attention_width<2, true>(const AttentionArgs&, const Schedule&, const Workspace&,
                                                    const Second<true>&, hipStream_t);
extern template hipError_t launch_attention_width<3, false>(const AttentionArgs&, const Schedule&, const Workspace&,
                                                    const Second<false>&, hipStream_t);
extern template hipError_t launch_attention_width<3, true>(const AttentionArgs&, const Schedule&, const Workspace&,
                                                    const Second<true>&, hipStream_t);
extern template hipError_t launch_attention_width<4, false>(const AttentionArgs&, const Schedule&, const Workspace&,
                                                    const Second<false>&, hipStream_t);
extern template hipError_t launch_attention_width<4, true>(const AttentionArgs&, const Schedule&, const Workspace&,
                                                    const Second<true>&, hipStream_t);
extern template hipError_t launch_attention_width<6, false>(const AttentionArgs&, const Schedule&, const Workspace&,
                                                    const Second<false>&, hipStream_t);
extern template hipError_t launch_attention_width<6, true>(const AttentionArgs&, const Schedule&, const Workspace&,
                                                    const Second<true>&, hipStream_t);
extern template hipError_t launch_attention_width<8, false>(const AttentionArgs&, const Schedule&, const Workspace&,
                                                    const Second<false>&, hipStream_t);
extern template hipError_t launch_attention_width<8, true>(const AttentionArgs&, const Schedule&, const Workspace&,
                                                    const Second<true>&, hipStream_t);

int64_t cache_attention_workspace(const CacheView& c, const RowsView& r, int ratio) {
  const Schedule s = plan_of(c, r, ratio);
  return s.target == 0 ? 0 : workspace_bytes(s, c.heads, c.C, r.batch);
}

hipError_t launch_cache_attention(const AttentionArgs& a, void* workspace, int64_t bytes, hipStream_t stream) {
  const int tile_rows = tile_rows_of(a.c, a.r, a.ratio);
  // With a window and first tokens few blocks are busy where there are few tiles, and
  // prompts' tiles are short: blocks of 8 steps. One sequence, window 8192, 64 first
  // tokens, groups of 32 with zero points, 24.0 -> 18.9 us; window 1000 20.1 -> 17.5; 4
  // prompts in chunks, window 1500, 142 -> 137; but 8 sequences of one row each 15.5 -> 16.4,
  // of 3 to 5 rows 20.2 -> 22.8.
  const bool few = a.r.batch <= 4 && a.r.rows * a.ratio <= 4 * tile_rows;
  Schedule s = plan_for(a.c, a.r, a.ratio, tile_rows, sink_end(a) > 0 && (few || tile_rows == kWideRows) ? 8 : 16);
  if (sink_end(a) > 0 && tile_rows == kWideRows) {
    // Prompts' tiles with a window are about as long as each other: with more tiles than
    // places only those of the last round are cut, over all places. 149 tiles on 128
    // places, against as many cuts as without first tokens and none at all: window 1500,
    // 148, 129 and 108 us, 3000 205, 207 and 170, 6000 321, 332 and 278; 274 tiles 194, 194
    // and 166. Where fewer tiles are cut for a short window, the join costs more than the
    // empty places, and so it does for the last round where a tile has less than two
    // blocks' steps: 77 tiles, window 1500, 80 us and uncut 77, 122 tiles 83 and 79; 149
    // tiles, window 300, 83 and 55.
    const int64_t tiles = a.r.rows * a.ratio / tile_rows, run = a.window / kStep + (sink_end(a) - 1) / kStep + 2;
    const bool last_round = tiles >= s.target && !s.planned && run >= 2 * s.min_steps;
    if (last_round) {
      cut_last_round(&s);
    } else if (a.window < 2560 && 3 * tiles >= s.target) {
      s.units -= s.target * (s.crowded ? 2 : 1);
      s.target = s.crowded = s.planned = 0;
    }
  }
  auto fits = [&] { return s.target == 0 || bytes >= workspace_bytes(s, a.c.heads, a.c.C, a.r.batch); };
  if (s.crowded && !fits()) {            // a workspace made for a larger call may have room for fewer cuts
    s.units -= s.target;
    s.crowded = 0;
  }
  if (!fits()) {
    s.units -= s.target;
    s.target = s.planned = 0;
  }
  const Workspace ws = workspace_at(workspace, s, a.c.heads, a.c.C);
  switch (a.c.C) {
    case 2: return launch_width<2>(a, s, ws, stream);
    case 3: return launch_width<3>(a, s, ws, stream);
    case 4: return launch_width<4>(a, s, ws, stream);
    case 6: return launch_width<6>(a, s, ws, stream);
    default: return launch_width<8>(a, s, ws, stream);
  }
}

}  // namespace int4dq
