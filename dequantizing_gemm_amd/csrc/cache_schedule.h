// cache_schedule.h -- how the attention kernel's work is cut into blocks.
//
// A sequence with n rows gives n * ratio query rows per key/value head (row i,
// head r of the head's `ratio` query heads: flat row i * ratio + r), cut into
// tiles of tile_rows. A tile sees a run of keys, cut into steps of 64 tokens;
// the steps of a tile are shared out over `chunks` blocks of equal length. How many
// is decided on the GPU from the lengths, whatever mixture the batch is: `target`
// blocks per head fill the GPU once, and the longest block is made as short as
// their number allows (steps_per_block), so that all run at once and end together;
// with more tiles than that, tiles are cut down to the average share; and with a
// few more, which would leave most of the GPU idle for their length, all are cut
// further, to at most 3 target blocks (4 prompts in chunks, 149 tiles and a target of
// 128: 260 us uncut, 237 so).
// So cuts add at most `target` blocks, and a tile of c > 1 chunks adds
// c - 1 >= c / 2 of them, or the blocks are at most 3 target: that bounds the grid
// and the number of partial results, which the host has to know.
#pragma once

#include "cache.h"

namespace int4dq {

constexpr int kStep = 64;                // tokens of a wavefront's step

constexpr int kWideRows = 128;           // rows of a tile in the form for prompts

struct Schedule {
  int tile_rows;                         // kWideRows: that form
  int target;                            // 0: every tile in one block
  int min_steps;
  int units;                             // blocks per key/value head
  int crowded;                           // tiles may be more than the target by up to half
  int planned;                           // the blocks of each sequence are counted by a kernel of its own
};

// From more sequences than a wavefront looks through at once, their blocks are
// counted once for all, by a kernel before the attention kernel (when that came in, 1024
// sequences of 512 tokens: 185 us; looked through by every block, 402 us; 256 of them:
// 51 and 63; 1024 of them take 129 us now).
constexpr int kScanBatch = 64;

// The first token of the 16-token unit u of a step. Unsigned: loads run a few steps
// ahead, past 2^31 where a sequence ends just below.
__host__ __device__ inline uint32_t unit_token(int step, int u) { return (uint32_t)step * kStep + 16u * (uint32_t)u; }

// Whether some row of a tile does not see some token of the step, where all rows see
// keys [lo, hi).
__host__ __device__ inline bool step_masked(int step, int lo, int hi) {
  return unit_token(step, 0) < (uint32_t)lo || unit_token(step + 1, 0) > (uint32_t)hi;
}

// One sequence's share of the call.
struct SequenceWork {
  int first;                             // its first row
  int end;                               // one past its last row, as starts has it
  int rows;
  int length;                            // as lengths has it
  int keys;                              // its cached tokens that the page table covers
  int tiles;
  int steps;                             // of a tile, at most; 1 where there are none
};

__host__ __device__ inline SequenceWork sequence_work(const AttentionArgs& a, int tile_rows, int b) {
  SequenceWork w;
  const int s0 = a.r.starts ? a.r.starts[b] : b;
  w.end = a.r.starts ? a.r.starts[b + 1] : b + 1;
  w.length = a.r.lengths[b];
  w.first = s0 > 0 ? s0 : 0;
  const int last = w.end < a.r.rows ? w.end : (int)a.r.rows;
  w.rows = last > w.first ? last - w.first : 0;
  const int64_t cover = a.r.max_pages << a.c.page_shift;
  w.keys = w.length < 0 ? 0 : w.length < cover ? w.length : (int)cover;
  w.tiles = (int)(((uint32_t)w.rows * (uint32_t)a.ratio + tile_rows - 1) / (uint32_t)tile_rows);
  w.steps = w.keys / kStep + (w.keys % kStep != 0);
  if (a.window > 0 && a.window < w.keys) {
    // a tile's rows lie on at most tile_rows / ratio + 2 positions
    const int64_t run = (a.window + tile_rows / a.ratio + 2) / kStep + 2;
    if (run < w.steps) w.steps = (int)run;
  }
  if (w.steps < 1) w.steps = 1;
  return w;
}

// Where every tile is left to one block: before sequence b come at most this many
// blocks, a number that needs no other sequence's length.
__host__ __device__ inline int64_t tiles_before(const AttentionArgs& a, const Schedule& s, int b) {
  const int64_t x = a.r.starts[b] < 0 ? 0 : a.r.starts[b] < a.r.rows ? a.r.starts[b] : a.r.rows;
  return (uint32_t)(x * a.ratio) / (uint32_t)s.tile_rows + b;
}

// Chunks of a tile when no block takes more than `per` steps.
__host__ __device__ inline int chunks_of(int steps, int per) { return (int)((uint32_t)(steps + per - 1) / (uint32_t)per); }

// The fewest steps for the longest block with which the cuts add no more blocks
// than there is room for: what `tiles` leave of the target, or the target where they
// exceed it (by much). `work`: the steps of all tiles of one head, `most` those of the
// longest; added(per): the blocks that chunks_of adds with `per`, at most
// work / per, so that work / room is enough (1.001: the sum's rounding).
template <typename F>
__host__ __device__ inline int steps_per_block(const Schedule& s, float work, float tiles, int most, F added) {
  const bool fits = tiles <= (float)s.target, few_over = !fits && s.crowded && tiles <= 1.5f * (float)s.target;
  const int room = fits ? s.target - (int)tiles : few_over ? 3 * s.target - (int)tiles : s.target;
  int from = (int)(work / (float)(few_over ? 3 * s.target : s.target)), to = most;
  if (from < s.min_steps) from = s.min_steps;
  if (room > 0) {
    const float enough = work * 1.001f / (float)room + 1.0f;
    if (enough < (float)to) to = (int)enough;
  }
  while (from < to) {
    const int per = (int)(((uint32_t)from + (uint32_t)to) / 2);
    if (added(per) <= room) to = per;
    else from = per + 1;
  }
  return from;
}

// Keys [lo, hi) that row `token` of a sequence's rows sees.
__host__ __device__ inline void visible(const AttentionArgs& a, const SequenceWork& w, int token, int* lo,
                                        int* hi) {
  const int64_t pos = (int64_t)w.length - w.end + w.first + token;
  const int64_t top = a.causal && pos + 1 < w.keys ? pos + 1 : w.keys;
  const int64_t low = a.window > 0 ? pos - a.window + 1 : 0;
  *hi = top > 0 ? (int)top : 0;
  *lo = low < 0 ? 0 : low < *hi ? (int)low : *hi;
}

// The steps [begin, end) of chunk `chunk` of a tile that sees keys [lo, hi).
__host__ __device__ inline void chunk_steps(int lo, int hi, int chunk, int chunks, int* begin, int* end) {
  const int s0 = lo / kStep, s1 = hi > lo ? (hi - 1) / kStep + 1 : s0;
  const int per = chunks == 1 ? s1 - s0 : (int)((uint32_t)(s1 - s0 + chunks - 1) / (uint32_t)chunks);
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

// Tiles of 16 rows a wavefront whose accumulators, scores and operands stay in
// registers, in the form for few rows (at most) and in the one for prompts: wide
// heads and many groups, affine ones above all, take more registers a row.
constexpr int max_tiles(int C, int groups, bool affine) { return groups * C <= (affine ? 4 : 8) && C <= 4 ? 2 : 1; }
constexpr int wide_tiles(int C, int groups, bool affine) {
  return groups * C >= (affine ? 32 : 64) ? 0 : C <= 4 && !(affine && groups > 1) ? 2 : 1;      // 0: no such form
}

// Blocks of a form that a CU holds at once, by their registers and LDS; the form for
// few rows is compiled to fit that many.
constexpr int resident_blocks(int C, int groups, bool affine, int tile_rows) {
  if (tile_rows == kWideRows) return wide_tiles(C, groups, affine);              // of 4 wavefronts, or 1 of 8
  if (tile_rows == 32) return C == 2 && !affine && groups == 1 ? 3 : 2;
  return C == 2 ? 4 : C == 3 ? (groups == 1 && !affine ? 4 : 3) : C == 4 ? (groups > 2 ? 2 : 3) : groups * C >= (affine ? 32 : 64) ? 1 : 2;
}

// The workspace: `slots` partial results for each head (the rows of a tile, then
// for each row its reference and sum), a record for each slot, the number of slots
// in use, and the plan of a large batch.
struct PartRecord {
  int first, flat0, flats;               // the sequence's first row, the tile's first flat row, the sequence's flat rows
  int chunk, chunks;
  int unused[3];
};

// Blocks and slots of the sequences before one.
struct PlanEntry {
  int blocks, slots;
};

struct Workspace {
  float* part;
  PartRecord* record;
  int* used;
  PlanEntry* plan;                       // [batch + 1], where planned
};

__host__ __device__ inline int64_t partial_floats(int tile_rows, int C) { return (int64_t)tile_rows * (32 * C + 2); }

__host__ __device__ inline int workspace_slots(const Schedule& s) { return (s.crowded ? 3 : 2) * s.target; }

inline int64_t workspace_bytes(const Schedule& s, int heads, int C, int batch) {
  return workspace_slots(s) * (heads * partial_floats(s.tile_rows, C) * 4 + (int64_t)sizeof(PartRecord)) + 16 +
         (s.planned ? (batch + 1) * (int64_t)sizeof(PlanEntry) : 0);
}

__host__ __device__ inline Workspace workspace_at(void* p, const Schedule& s, int heads, int C) {
  float* const part = static_cast<float*>(p);
  PartRecord* const record =
      reinterpret_cast<PartRecord*>(part + workspace_slots(s) * (heads * partial_floats(s.tile_rows, C)));
  int* const used = reinterpret_cast<int*>(record + workspace_slots(s));
  return Workspace{part, record, used, reinterpret_cast<PlanEntry*>(used + 4)};
}

constexpr int kComputeUnits = 256;

// Tiles of 16 rows for token generation, of 32 where the sequences' rows fill
// them, and the form for prompts where a sequence's rows fill a tile of it, or two
// where tiles of 32 are the other choice. Measured on 8 sequences of 2650 tokens on
// average, 8 key/value heads, few rows' form and prompts': head width 128, 128 rows
// 39 us and 52, 256 rows 60 and 60, 512 rows 91 and 90; width 256 (tiles of 16),
// 128 rows 69 and 71, 192 rows 96 and 90.
inline Schedule plan_of(const CacheView& c, const RowsView& r, int ratio) {
  Schedule s{};
  const int64_t mean = (r.rows * ratio + r.batch - 1) / r.batch;
  const int groups = c.C / scale_blocks(c), most = 16 * max_tiles(c.C, groups, c.affine);
  const bool wide = mean > most / 16 * kWideRows && wide_tiles(c.C, groups, c.affine) > 0;
  s.tile_rows = wide ? kWideRows : mean <= 16 ? 16 : most;
  const int resident = resident_blocks(c.C, groups, c.affine, s.tile_rows);
  s.target = (resident * kComputeUnits + c.heads - 1) / c.heads;
  // Four for each wavefront of the form for few rows (16 sequences of 2650 tokens, 3 to
  // 6 rows each, with at least one each: 40 us, four: 35; one row of 2000 tokens 18.7
  // and 17.7). The form for prompts has the same number, though its wavefronts all take
  // every step: that suits many rows (8 sequences, 512 rows each: 87 us with 16, 10 and
  // 6) better than few on one sequence (400 rows on 3000 tokens 47, 37 and 35 us; 1200
  // rows on 1500 tokens 41, 36 and 40).
  s.min_steps = 16;
  // Where no sequence can have more, every tile is left to one block and the join
  // kernel's launch is saved.
  if ((r.max_pages << c.page_shift) <= s.min_steps * kStep) s.target = 0;
  s.planned = s.target > 0 && r.batch > kScanBatch;
  const int64_t fewest = (r.rows * ratio + s.tile_rows - 1) / s.tile_rows, tiles = r.rows * ratio / s.tile_rows + r.batch;
  s.crowded = tiles > s.target && 2 * fewest <= 3 * (int64_t)s.target;
  s.units = (int)(s.target * (s.crowded ? 2 : 1) + tiles);
  return s;
}

}  // namespace int4dq
