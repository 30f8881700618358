// cache_schedule.h -- how the attention kernel's work is cut into blocks.
//
// A sequence with n rows gives n * ratio query rows per key/value head (row i,
// head r of the head's `ratio` query heads: flat row i * ratio + r), cut into
// tiles of tile_rows. A tile sees a run of keys, cut into steps of 64 tokens;
// the steps of a tile are shared out over `chunks` blocks. How many is decided
// on the GPU from the lengths: with W the steps of all tiles of one head and
// `target` the blocks per head that fill the GPU, a block takes about
// per_block = max(min_steps, W / target) steps, so a long sequence gets many
// blocks and a short one a single one, whatever mixture the batch is. Hence
//   blocks per head <= W / per_block + tiles <= target + tiles
// (the size of the grid, known on the host), and the blocks of tiles with more
// than one chunk, which leave partial results in the workspace, number at most
// 2 target: such a tile has over per_block steps, so there are at most target of
// them.
#pragma once

#include "cache.h"

namespace int4dq {

constexpr int kStep = 64;                // tokens of a wavefront's step

struct Schedule {
  int tile_rows;
  int target;                            // 0: every tile in one block
  int min_steps;
  int units;                             // blocks per key/value head
};

// One sequence's share of the call.
struct SequenceWork {
  int64_t first;                         // its first row
  int64_t end;                           // one past its last row, as starts has it
  int rows;
  int keys;                              // its cached tokens that the page table covers
  int tiles;
  int steps;                             // of a tile, at most; 1 where there are none
};

__host__ __device__ inline SequenceWork sequence_work(const AttentionArgs& a, int tile_rows, int b) {
  SequenceWork w;
  const int64_t s0 = a.r.start(b);
  w.end = a.r.start(b + 1);
  w.first = s0 > 0 ? s0 : 0;
  const int64_t last = w.end < a.r.rows ? w.end : a.r.rows;
  w.rows = last > w.first ? (int)(last - w.first) : 0;
  const int64_t cover = a.r.max_pages << a.c.page_shift;
  const int64_t len = a.r.lengths[b];
  w.keys = (int)(len < 0 ? 0 : len < cover ? len : cover);
  w.tiles = (int)(((uint32_t)w.rows * (uint32_t)a.ratio + tile_rows - 1) / (uint32_t)tile_rows);
  w.steps = w.keys / kStep + (w.keys % kStep != 0);
  if (a.window > 0 && a.window < w.keys) {
    // a tile's rows lie on at most tile_rows / ratio + 2 positions
    const int run = ((int)a.window + tile_rows / a.ratio + 2) / kStep + 2;
    if (run < w.steps) w.steps = run;
  }
  if (w.steps < 1) w.steps = 1;
  return w;
}

// Steps of a block, from the steps of all tiles of one head (a binary32 sum,
// taken the same way in every kernel; the margin covers its rounding, so that
// the bounds above hold).
__host__ __device__ inline int steps_per_block(const Schedule& s, float all_steps) {
  if (s.target == 0) return 1 << 30;
  const float per = all_steps * 1.001f / (float)s.target;
  return per < (float)s.min_steps ? s.min_steps : per > 1e9f ? 1 << 30 : (int)per + 1;
}

__host__ __device__ inline int chunks_of(int steps, int per_block) {
  return (int)((uint32_t)(steps - 1) / (uint32_t)per_block) + 1;
}

// Keys [lo, hi) that flat row `row` of a sequence sees.
__host__ __device__ inline void visible(const AttentionArgs& a, const SequenceWork& w, int length, int row,
                                        int* lo, int* hi) {
  const int64_t pos = length - (w.end - (w.first + (uint32_t)row / (uint32_t)a.ratio));
  const int64_t top = a.causal && pos + 1 < w.keys ? pos + 1 : w.keys;
  const int64_t low = a.window > 0 ? pos - a.window + 1 : 0;
  *hi = top > 0 ? (int)top : 0;
  *lo = low < 0 ? 0 : low < *hi ? (int)low : *hi;
}

// The steps [begin, end) of chunk `chunk` of a tile that sees keys [lo, hi).
__host__ __device__ inline void chunk_steps(int lo, int hi, int chunk, int chunks, int* begin, int* end) {
  const int s0 = lo / kStep, s1 = hi > lo ? (hi - 1) / kStep + 1 : s0;
  const int per = (int)((uint32_t)(s1 - s0 + chunks - 1) / (uint32_t)chunks);
  const int64_t from = s0 + (int64_t)chunk * per;
  *begin = from < s1 ? (int)from : s1;
  *end = from + per < s1 ? (int)(from + per) : s1;
}

// Blocks of 32 channels to a scale in the kernel's form for this cache: all C, the
// group's where that divides C, or else 1.
inline int scale_blocks(const CacheView& c) {
  const int blocks = c.G == 1 ? c.C : c.group / 32;
  return c.C % blocks == 0 ? blocks : 1;
}

// The tallest tile (in 16 rows) whose accumulators, scores and operands stay in
// registers: wide heads and many groups take more of them a row.
constexpr int max_tiles(int C, int groups) {
  return C <= 2 || (C <= 4 && groups == 1) ? 4 : groups * C <= 24 ? 2 : 1;
}

// A partial result: the rows of a tile, then for each row its reference and sum.
__host__ __device__ inline int64_t partial_floats(int tile_rows, int C) { return (int64_t)tile_rows * (32 * C + 2); }

// Partial results of one head, at most.
inline int64_t workspace_slots(const Schedule& s) { return 2 * (int64_t)s.target; }

constexpr int kComputeUnits = 256;

// Tiles of 16 rows for token generation, 32 or 64 where the sequences' rows
// fill them.
inline Schedule plan_of(const CacheView& c, const RowsView& r, int ratio) {
  Schedule s{};
  const int64_t mean = (r.rows * ratio + r.batch - 1) / r.batch;
  const int most = 16 * max_tiles(c.C, c.C / scale_blocks(c));
  s.tile_rows = mean <= 16 ? 16 : mean <= 32 ? 32 : 64;
  if (s.tile_rows > most) s.tile_rows = most;
  const int resident = s.tile_rows == 16 ? 3 : s.tile_rows == 32 ? 2 : 1;      // blocks on a CU
  s.target = (resident * kComputeUnits + c.heads - 1) / c.heads;
  s.min_steps = 4;
  s.units = (int)(s.target + r.rows * ratio / s.tile_rows + r.batch);
  return s;
}

}  // namespace int4dq
