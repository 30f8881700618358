// store_driver.cpp -- the arithmetic by which the 4-bit cache's write and read kernels
// find their rows (StoreBlock in cache.h, the search in lanes.h), and the attention
// kernel's shares, under AddressSanitizer and UndefinedBehaviorSanitizer: with starts
// that do not decrease, every row that a sequence owns is in exactly one block of the
// grid, at its own position, and no other row in any; with any contents of starts,
// lengths and page table, every row, code and scale of a block lies inside its array,
// and every share of the attention kernel inside the grid, the rows and the workspace.
//
// Test infrastructure: built and run only by tests/test_sanitize_store_cpu.py.
// Exit status 0 when every check holds.
#include <limits.h>
#include <stdio.h>

#include <random>
#include <vector>

#include "../../dequantizing_gemm_amd/csrc/cache.h"
#include "../../dequantizing_gemm_amd/csrc/cache_schedule.h"
#include "../../dequantizing_gemm_amd/csrc/lanes.h"

using namespace int4dq;

static int failures = 0;
#define CHECK(cond, what)                                        \
  do {                                                           \
    if (!(cond)) {                                               \
      if (++failures < 20) fprintf(stderr, "FAIL line %d: %s\n", __LINE__, what); \
    }                                                            \
  } while (0)

static std::mt19937_64 rng(2);
static int64_t pick(int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); }

// lane_search with the lanes one after another.
struct HostSearch {
  template <typename F>
  int operator()(int n, int64_t x, F f) const {
    return search_by_lanes(n, [&](int from, int apart, int left) {
      uint64_t bits = 0;
      for (int lane = 0; lane < kWave; ++lane)
        if (lane * apart < left && f(from + lane * apart) <= x) bits |= uint64_t(1) << lane;
      return bits;
    });
  }
};

static void searches() {
  for (int trial = 0; trial < 3000; ++trial) {
    const int sizes[] = {1, 2, 63, 64, 65, 128, 4095, 4096, 4097, 20000};
    const int n = trial % 3 ? (int)pick(1, 300) : sizes[pick(0, 9)];
    std::vector<int64_t> f(n);
    const bool wild = trial % 5 == 4;
    int64_t at = pick(-5, 5);
    for (auto& v : f) v = wild ? pick(-9, 9) : (at += pick(0, 2));
    const int64_t x = pick(-8, wild ? 9 : f.back() + 3);
    const int got = HostSearch{}(n, x, [&](int i) { return f.at(i); });
    CHECK(got >= 0 && got < n, "a place in range");
    if (wild) continue;
    int want = 0;
    for (int i = 0; i < n; ++i) if (f[i] <= x) want = i;
    CHECK(got == want, "the last place at or below");
  }
}

struct Plan {
  std::vector<int32_t> table, lens, starts;
  RowsView r;
};

// kind 0: as a caller means it; 1: starts that do not decrease, all else senseless;
// 2: all of it senseless.
static Plan plan(int kind, int page_shift, int64_t pages, bool one) {
  Plan p;
  const int B = (int)(pick(0, 9) ? pick(1, 12) : pick(60, 200)), mp = (int)pick(0, 6), stride = mp + (int)pick(0, 3);
  p.table.resize((size_t)B * stride + 1);
  p.lens.resize(B);
  p.starts.resize(B + 1);
  const int32_t far[] = {INT_MAX, INT_MIN, INT_MAX - 1, -1, 1 << 30};
  for (auto& t : p.table) t = kind == 0 ? (int32_t)pick(0, pages - 1) : pick(0, 4) ? (int32_t)pick(-2, pages + 1) : far[pick(0, 4)];
  for (auto& l : p.lens)
    l = kind == 0 ? (int32_t)pick(0, (int64_t)mp << page_shift) : pick(0, 5) ? (int32_t)pick(-90, 600) : far[pick(0, 4)];
  p.starts[0] = kind == 0 ? 0 : (int32_t)pick(-9, 9);
  for (int b = 1; b <= B; ++b)
    p.starts[b] = kind == 2 ? (int32_t)pick(-9, 300) : p.starts[b - 1] + (int32_t)(pick(0, 4) ? pick(0, 9) : pick(0, 200));
  if (kind == 2 && pick(0, 2)) p.starts[pick(0, B)] = far[pick(0, 4)];
  const int64_t T = one ? B : kind == 0 ? p.starts[B] : pick(0, 400);
  p.r = RowsView{p.table.data(), stride, mp, p.lens.data(), one ? nullptr : p.starts.data(), B, T};
  return p;
}

static void stores() {
  for (int trial = 0; trial < 3000; ++trial) {
    const int kind = trial % 3, shift = (int)pick(4, 8), heads = (int)pick(1, 2), D = trial % 2 ? 64 : 100;
    const bool one = trial % 7 == 6;
    const int64_t pages = pick(1, 5);
    const CacheView c{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, pages, shift, heads, D, 32, (D + 31) / 32, cache_blocks(D), 1};
    const Plan p = plan(kind, shift, pages, one);
    const RowsView& r = p.r;
    if (r.rows == 0) continue;             // the entry points launch nothing
    const size_t units = ((size_t)pages * heads) << (shift - 4);
    std::vector<uint8_t> codes(units * 16 * c.row_bytes());
    std::vector<uint16_t> scales(units * 16 * c.G);
    std::vector<int> seen(r.rows);
    for (int64_t u = 0; u < store_units(r); ++u) {
      StoreBlock w;
      if (!find_store_block(r, (int)u, HostSearch{}, &w)) continue;
      CHECK(w.b >= 0 && w.b < r.batch, "a sequence of the batch");
      CHECK((w.base & 63) == 0, "whole steps");
      CHECK(w.rows == 0 || (w.first >= 0 && (int64_t)w.first + w.rows <= r.rows), "rows inside the call");
      for (int t = 0; t < 64; ++t) {
        const int64_t pos = w.base + t, at_row = pos - w.p0;
        const int64_t page = find_page(r, c, w.b, pos);
        CHECK(page >= -1 && page < pages, "a page of the cache");
        if (t % 16 == 0 && page >= 0)
          CHECK(find_page(r, c, w.b, pos + 15) == page, "a unit lies on one page");
        if (at_row < 0 || at_row >= w.rows) continue;
        const int64_t row = w.first + at_row;
        seen.at(row)++;
        if (kind != 2) {
          int b = -1;
          int64_t where = 0;
          CHECK(find_row(r, row, &b, &where) && b == w.b && where == pos, "the row at its sequence's position");
        }
        if (page < 0) continue;
        const int slot = (int)(pos & ((1 << shift) - 1)), ts = slot & 15, DB = c.row_bytes();
        for (int h = 0; h < heads; ++h) {
          // as the kernels go: from the unit of head 0, a page of units further for each head
          const int64_t unit = c.unit(page, 0, slot) + ((int64_t)h << (shift - 4));
          CHECK(unit == c.unit(page, h, slot), "a head's unit");
          codes.at(unit * 16 * DB + ts * DB + 3 * 4 * c.C + 4 * (c.C - 1) + 3) = 1;    // keys
          codes.at(unit * 16 * DB + (int64_t)(DB - 1) * 16 + ts) = 1;                  // values
          scales.at((unit * c.G + c.G - 1) * 16 + ts) = 1;
        }
      }
    }
    if (kind == 2) continue;
    for (int64_t t = 0; t < r.rows; ++t) {
      int b;
      int64_t pos;
      CHECK(seen[t] == (find_row(r, t, &b, &pos) ? 1 : 0), "every owned row once, no other");
    }
  }
}

// The attention kernel's shares, as its find_block cuts them.
static void shares() {
  for (int trial = 0; trial < 3000; ++trial) {
    const int kind = 1 + trial % 2, shift = (int)pick(4, 8), Ds[] = {64, 96, 128, 256}, D = Ds[pick(0, 3)];
    const Plan p = plan(kind, shift, 100, trial % 7 == 6);
    if (p.r.rows == 0) continue;
    AttentionArgs a{};
    const int groups[] = {32, 64, D}, group = groups[pick(0, 2)];
    a.c = CacheView{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 100, shift, (int)pick(1, 40), D, group, (D + group - 1) / group,
                    cache_blocks(D), (int)pick(0, 1)};
    a.r = p.r;
    a.r.max_pages = trial % 4 ? (int64_t)1 << 14 : p.r.max_pages;      // sizes only: the table is not read here
    a.ratio = (int)pick(1, trial % 3 ? 8 : 40);
    a.causal = (int)pick(0, 1);
    a.window = a.causal && pick(0, 1) ? pick(1, 700) : 0;
    Schedule s = plan_of(a.c, a.r, a.ratio);
    if (trial % 5 == 4) { s.units -= s.target * (s.crowded ? 2 : 1); s.target = s.crowded = s.planned = 0; }
    const int B = a.r.batch;
    std::vector<SequenceWork> w(B);
    float work = 0.0f, tiles = 0.0f;
    int most = 0;
    for (int b = 0; b < B; ++b) {
      w[b] = sequence_work(a, s.tile_rows, b);
      CHECK(w[b].rows == 0 || (w[b].first >= 0 && (int64_t)w[b].first + w[b].rows <= a.r.rows), "rows inside the call");
      CHECK(w[b].steps >= 1 && w[b].keys >= 0, "steps and keys");
      work += (float)w[b].tiles * (float)w[b].steps;
      tiles += (float)w[b].tiles;
      if (w[b].tiles > 0 && w[b].steps > most) most = w[b].steps;
    }
    std::vector<PlanEntry> before(B + 1);
    if (s.target > 0) {
      const int per = steps_per_block(s, work, tiles, most, [&](int x) {
        int sum = 0;
        for (const auto& v : w) sum += v.tiles > 0 ? (chunks_of(v.steps, x) - 1) * v.tiles : 0;
        return sum;
      });
      for (int b = 0; b < B; ++b) {
        const int chunks = w[b].tiles > 0 ? chunks_of(w[b].steps, per) : 0, mine = chunks * w[b].tiles;
        before[b + 1] = PlanEntry{before[b].blocks + mine, before[b].slots + (chunks > 1 ? mine : 0)};
      }
      CHECK(before[B].slots <= workspace_slots(s), "partial results inside the workspace");
    }
    for (int unit = 0; unit < s.units; ++unit) {
      int b, i, chunks;
      if (s.target > 0) {
        b = HostSearch{}(B, unit, [&](int x) { return (int64_t)before.at(x).blocks; });
        i = unit - before[b].blocks;
        if (i < 0 || i >= before[b + 1].blocks - before[b].blocks) continue;
        chunks = (before[b + 1].blocks - before[b].blocks) / w[b].tiles;
        CHECK(chunks == 1 || (before[b].slots + i >= 0 && before[b].slots + i < workspace_slots(s)), "a slot of the workspace");
      } else if (a.r.starts) {
        b = HostSearch{}(B, unit, [&](int x) { return tiles_before(a, s, x); });
        i = unit - (int)tiles_before(a, s, b);
        if (i < 0 || i >= w[b].tiles) continue;
        chunks = 1;
      } else {
        const int each = (a.ratio + s.tile_rows - 1) / s.tile_rows;
        b = unit / each;
        if (b >= B) continue;
        i = unit % each;
        if (i >= w[b].tiles) continue;
        chunks = 1;
      }
      const int chunk = i % chunks, tile = w[b].tiles - 1 - i / chunks, flats = w[b].rows * a.ratio;
      CHECK(tile >= 0 && tile * s.tile_rows < flats, "a tile with rows");
      int lo, hi, lo1, hi1, begin, end;
      visible(a, w[b], tile * s.tile_rows / a.ratio, &lo, &hi);
      const int last = ((tile + 1) * s.tile_rows < flats ? (tile + 1) * s.tile_rows : flats) - 1;
      visible(a, w[b], last / a.ratio, &lo1, &hi1);
      CHECK(w[b].first + last / a.ratio < a.r.rows, "its last row inside the call");
      chunk_steps(lo, hi1, chunk, chunks, &begin, &end);
      CHECK(lo >= 0 && hi1 <= w[b].keys && begin <= end && (begin == end || (begin >= 0 && (int64_t)(end - 1) * kStep < w[b].keys)),
            "steps inside the keys");
    }
  }
}

int main() {
  searches();
  stores();
  shares();
  if (failures) return 1;
  printf("all checks passed\n");
  return 0;
}
