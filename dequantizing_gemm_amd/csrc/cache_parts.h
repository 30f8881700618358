// cache_parts.h -- attention for a batch whose sequences begin with the same tokens: whether the
// shared tokens are computed once, and how both parts are cut then. Host code, and checked
// as such on a machine without a GPU.
#pragma once

#include "cache_schedule.h"

namespace int4dq {

struct Parts {
  Schedule own, shared;
  int64_t own_bytes, shared_bytes;
  int from;                  // shared tokens, at least
  int64_t bytes() const { return own_bytes + shared_bytes; }
};

// From how many shared tokens on sharing pays; 0: never. Measured, 8 x 4 heads of 128,
// shared against not.
//  - Few rows, tiles of 16 at most half filled by a sequence: 200 own tokens, 4 sequences
//    18 and 21 us with 8192 shared tokens, 16 and 15 with 1984; 16 sequences 24 and 32,
//    18 and 19; 64 sequences 44 and 88, 32 and 32, with 512 30 and 16; 2 sequences, 18 and
//    17.5, with 32768 tokens 30 and 27.5.
//  - More rows take codes apart as often either way; what is saved is what the
//    sequences' last tiles leave empty, which has to pay for the join: 16 sequences
//    of 30 to 250 rows 850 and 1040 us with 20011 shared tokens (64 tiles and 72),
//    519 and 510 with 8192; 16 of 16 to 64 rows 330 and 368, 182 and 177; but 4 of 30 to 250
//    rows 434 and 417, 16 of 100 to 500 2108 and 1999, 16 of 4 rows each, whose tiles are
//    full, 68 and 58.
//  - What this rule leaves to share_from: many sequences with full tiles, for which the
//    shared part's tiles of 128 rows of the whole batch take codes apart less often. 64 of
//    one row with 16 query heads a key head (4 of these) 123 and 150 us with 32768 shared
//    tokens, 59 and 48 with 8192; 128 of 4 rows 374 and 543, with 4096 104 and 102; 32 of 4
//    rows 132 and 146; 128 of 8 rows 699 and 736, 32 of them 206 and 205, 8 of them 75 and 67.
//  - It does not go by a window, which the shared part's cut does not know either, so that
//    a short one loses: 64 sequences of 10 to 1500 own tokens on 32768, window 1000, 44 and
//    24 us, 2048 47 and 33, 8192 57 and 84, 40000 86 and 354.
inline int64_t sharing_pays(const RowsView& r, int ratio) {
  const int64_t rows = r.rows * ratio, tokens = 24576 / (r.batch > 0 ? r.batch : 1);
  if (rows <= 8 * (int64_t)r.batch) return r.batch < 4 ? 0 : tokens > 1536 ? tokens : 1536;
  return r.batch >= 8 && rows > 64 * (int64_t)r.batch && rows <= 640 * (int64_t)r.batch && rows <= 16384 ? 16384 : 0;
}

// The tiles of the shared part, for the number of its rows and of the tokens that the
// page table covers, which the shared ones may be. Measured, 300 own tokens, in tiles of 16
// (one launch with the sequences' own), 32 and 128 rows: 128 rows 24, 30 and 42 us with
// 4032 shared tokens, 55, 55 and 61 with 32768; 256 rows 29, 33 and 45 with 1984, 44, 45 and
// 51 with 8192, 87, 81 and 82 with 32768; 512 rows 47, 52 and 61, 68, 69 and 73, 154, 141
// and 132; 1024 rows 70, 75 and 78, 109, 108 and 106, 300, 249 and 224.
constexpr int64_t kLongTable = 16384;
inline int shared_tile_rows(const CacheView& c, int64_t rows, int64_t cover) {
  const int groups = c.C / scale_blocks(c), most = 16 * max_tiles(c.C, groups, c.affine);
  if (rows >= (cover < kLongTable ? 2048 : 1024) && wide_tiles(c.C, groups, c.affine) > 0) return kWideRows;
  return rows >= 256 && cover >= kLongTable ? most : 16;
}

// False: sharing would not pay, or cannot be. from < 0: where it pays.
inline bool plan_parts(const CacheView& c, const RowsView& r, int ratio, int64_t from, Parts* p) {
  if (from < 0) from = sharing_pays(r, ratio);
  else if (from == 0) from = 1;
  if (from == 0 || (r.max_pages << c.page_shift) < from) return false;
  p->from = from < INT32_MAX ? (int)from : INT32_MAX;
  RowsView one = r;
  one.batch = 1;
  // A join follows in any case: blocks of 8 steps, not 16 (24 sequences' rows, 1984
  // shared tokens: 21.1 -> 17.3 us; of 4: 16.2, but 33.1 -> 37.5 with 32768).
  p->own = plan_for(c, r, ratio, tile_rows_of(c, r, ratio), 8);
  p->shared = plan_for(c, one, ratio, shared_tile_rows(c, r.rows * ratio, r.max_pages << c.page_shift), 8);
  if (p->own.target == 0 || p->shared.target == 0) return false;
  p->own.partial = p->shared.partial = 1;
  p->own_bytes = (workspace_bytes(p->own, c.heads, c.C, r.batch) + 255) / 256 * 256;
  p->shared_bytes = workspace_bytes(p->shared, c.heads, c.C, 1);
  return true;
}

// What a call of these sizes takes at most, whatever its page table's length up to r's; 0: it does not share.
inline int64_t parts_workspace(const CacheView& c, const RowsView& r, int ratio, int64_t from) {
  Parts p;
  int64_t most = plan_parts(c, r, ratio, from, &p) ? p.bytes() : 0;
  if ((r.max_pages << c.page_shift) >= kLongTable) { // a call whose table is shorter may cut finer
    RowsView shorter = r;
    shorter.max_pages = (kLongTable - 1) >> c.page_shift;
    if (plan_parts(c, shorter, ratio, from, &p) && p.bytes() > most) most = p.bytes();
  }
  return most;
}

}  // namespace int4dq
