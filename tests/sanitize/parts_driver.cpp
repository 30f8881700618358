// parts_driver.cpp -- whether a batch that shares its first tokens is computed in two parts
// and how these are cut (dequantizing_gemm_amd/csrc/cache_parts.h), under AddressSanitizer
// and UndefinedBehaviorSanitizer.
//
// With arguments (head_dim group affine heads batch rows ratio max_pages page from): the tile
// heights of both parts and the least number of shared tokens, or "apart".
// Without: over random sizes, that the workspace asked for a page table is enough for every
// shorter one, that what a plan asks for are forms that there are, launches that fit, and
// partial results that lie inside the workspace.
//
// Test infrastructure: built and run only by tests/test_sanitize_parts_cpu.py.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <random>

#include "../../dequantizing_gemm_amd/csrc/cache_parts.h"

static int failures = 0;
#define CHECK(cond, what)                                                      \
  do {                                                                         \
    if (!(cond) && ++failures < 30) fprintf(stderr, "FAIL line %d: %s\n", __LINE__, what); \
  } while (0)

using namespace int4dq;
static std::mt19937_64 rng(7);
static int64_t pick(int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); }
static int64_t spread(int64_t lo, int64_t hi) {      // over the logarithm
  int64_t x = pick(lo, hi);
  while (x > lo && pick(0, 3)) x = lo + (x - lo) / 2;
  return x;
}

static CacheView view(int D, int group, bool affine, int heads, int shift) {
  const int g = group < D ? group : D;
  return CacheView{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 1000, shift, heads, D, g, (D + g - 1) / g, cache_blocks(D), affine ? 1 : 0};
}

static void check_plan(const CacheView& c, const RowsView& r, int ratio, const Parts& p) {
  const int groups = c.C / scale_blocks(c);
  RowsView one = r;
  one.batch = 1;
  const struct { const Schedule& s; const RowsView& r; int64_t bytes; } parts[] = {{p.own, r, p.own_bytes}, {p.shared, one, p.shared_bytes}};
  for (const auto& x : parts) {
    const Schedule& s = x.s;
    CHECK(s.tile_rows == 16 || (s.tile_rows == 32 && max_tiles(c.C, groups, c.affine) == 2) ||
              (s.tile_rows == kWideRows && wide_tiles(c.C, groups, c.affine) > 0), "a form that there is");
    CHECK(s.target > 0 && s.partial && !s.last_round && workspace_slots(s) == s.units, "a slot for every block");
    CHECK(x.bytes >= workspace_bytes(s, c.heads, c.C, x.r.batch), "room for the part");
    CHECK((int64_t)s.units * c.heads < (1 << 24), "a launch of fewer than 2^32 threads");
    CHECK(s.planned == (x.r.batch > kScanBatch), "counted before where a wavefront does not hold the batch");
  }
  CHECK(p.own_bytes % 256 == 0, "the shared part's workspace is aligned");
  CHECK(p.from >= 1, "shared tokens, at least");
}

static void sweep() {
  for (int trial = 0; trial < 4000; ++trial) {
    const int groups[] = {32, 64, 128, 256};
    const int shift = (int)pick(4, trial % 5 == 0 ? 20 : 8);
    const CacheView c = view((int)(pick(0, 1) ? 32 * pick(2, 8) : pick(1, 256)), groups[pick(0, 3)], pick(0, 1), (int)spread(1, 64), shift);
    const int ratio = (int)spread(1, 16);
    const int batch = (int)spread(1, std::min<int64_t>(1 << 18, (1 << 20) / c.heads));
    const bool one = pick(0, 2) == 0;
    const int64_t rows = one ? batch : std::min<int64_t>(spread(1, 200000), (int64_t)(1 << 24) / (c.heads * ratio));
    if (rows * ratio * c.heads > (1 << 25)) continue;
    const int32_t starts = 0;
    RowsView r{nullptr, 0, 0, nullptr, one ? nullptr : &starts, batch, rows};
    const int64_t from[] = {-1, 0, 1, pick(1, 2000), pick(1, 40000), kLongTable - 1, kLongTable, kLongTable + 1, INT64_MAX};
    const int64_t f = from[pick(0, 8)];
    r.max_pages = pick(0, 3) ? std::max<int64_t>(0, (pick(0, 1) ? kLongTable : spread(1, 200000)) >> shift) + pick(0, 2) : INT32_MAX;
    const int64_t asked = parts_workspace(c, r, ratio, f);
    CHECK(asked >= 0, "a size");
    const int64_t limit = std::min<int64_t>(r.max_pages, ((kLongTable + 3000) >> shift) + 3);
    for (int64_t n = 0; n <= limit + 1; n = n < 40 || limit - n < 40 || std::abs((n << shift) - kLongTable) < 64 ? n + 1 : n + 1 + pick(0, 20)) {
      RowsView s = r;
      s.max_pages = n <= limit ? n : r.max_pages;
      Parts p;
      if (!plan_parts(c, s, ratio, f, &p)) continue;
      CHECK((s.max_pages << shift) >= p.from, "as many tokens as the table has");
      CHECK(p.bytes() <= asked, "enough for every shorter table");
      check_plan(c, s, ratio, p);
    }
    if (f < 0 && asked > 0) CHECK(sharing_pays(r, ratio) >= 1536, "shares where that was measured to pay");
  }
}

int main(int argc, char** argv) {
  if (argc == 11) {
    int64_t v[10];
    for (int i = 0; i < 10; ++i) v[i] = atoll(argv[i + 1]);
    int shift = 0;
    while ((1LL << shift) < v[8]) ++shift;
    const CacheView c = view((int)v[0], (int)v[1], v[2] != 0, (int)v[3], shift);
    const int32_t starts = 0;
    const RowsView r{nullptr, 0, v[7], nullptr, &starts, (int)v[4], v[5]};
    Parts p;
    if (!plan_parts(c, r, (int)v[6], v[9], &p)) printf("apart\n");
    else printf("%d %d %d\n", p.own.tile_rows, p.shared.tile_rows, p.from);
    return 0;
  }
  sweep();
  if (failures) return 1;
  printf("all checks passed\n");
  return 0;
}
