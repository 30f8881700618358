// step_driver.cpp -- the host side of a serving step over the 4-bit cache
// (include/int4dq_cache_step.h) under AddressSanitizer and UndefinedBehaviorSanitizer:
// the entry points' checks, with the kernel launchers replaced by stubs; the index
// arithmetic of the page kernels; and which keys the attention kernel's tiles take
// with first tokens that stay visible and in the two parts of a batch that shares
// tokens, on sound and on senseless plans: every key that a row sees in exactly one
// place, no other, and every partial result inside the workspace.
//
// Test infrastructure: built and run only by tests/test_sanitize_step_cpu.py.
// Exit status 0 when every check holds.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <random>
#include <vector>

#include "../../dequantizing_gemm_amd/csrc/cache.h"
#include "../../dequantizing_gemm_amd/csrc/cache_schedule.h"
#include "../../dequantizing_gemm_amd/csrc/cache_step.h"
#include "../../include/int4dq_cache_step.h"

static int failures = 0;
static int calls = 0, shared_calls = 0;
#define CHECK(cond, what)                                                                      \
  do {                                                                                         \
    if (!(cond)) {                                                                             \
      if (++failures < 30)                                                                     \
        fprintf(stderr, "FAIL line %d: %s (last error: \"%s\")\n", __LINE__, what, int4_last_error()); \
    }                                                                                          \
  } while (0)

namespace int4dq {
hipError_t launch_cache_release(const PagesArgs&, const uint8_t*, const int32_t*, hipStream_t) { ++calls; return hipSuccess; }
hipError_t launch_cache_extend(const PagesArgs&, const int32_t*, int32_t*, int64_t*, int64_t, hipStream_t) { ++calls; return hipSuccess; }
hipError_t launch_cache_append(const AppendArgs&, int, hipStream_t) { ++calls; return hipSuccess; }
hipError_t launch_cache_attention(const AttentionArgs&, void*, int64_t, hipStream_t) { ++calls; return hipSuccess; }
hipError_t launch_cache_attention_shared(const AttentionArgs&, int64_t, void*, int64_t, hipStream_t) { ++shared_calls; return hipSuccess; }
int64_t cache_attention_workspace(const CacheView&, const RowsView&, int) { return 512; }
int64_t cache_attention_shared_workspace(const CacheView&, const RowsView&, int, int64_t) { return 1024; }
}  // namespace int4dq
extern "C" const char* int4_last_error(void);

using namespace int4dq;
static std::mt19937_64 rng(1);
static int64_t pick(int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); }

static void pages() {
  for (int trial = 0; trial < 2000; ++trial) {
    PagesArgs a{};
    a.max_pages = pick(0, 20);
    a.page_shift = (int)pick(4, 20);
    a.pages = pick(0, 40);
    const int64_t length = pick(0, 3) ? pick(-100, 100000) : (pick(0, 1) ? INT32_MAX : INT32_MIN);
    const int64_t n = a.entries(length);
    CHECK(n >= 0 && n <= a.max_pages, "entries inside the table row");
    CHECK(n == a.max_pages || (n << a.page_shift) >= length, "entries for every token");
    CHECK(n == 0 || ((n - 1) << a.page_shift) < length, "no entry too many");
    const int64_t free = a.free_pages((int32_t)(pick(0, 1) ? pick(-5, 60) : (pick(0, 1) ? INT32_MAX : INT32_MIN)));
    CHECK(free >= 0 && free <= a.pages, "free pages inside their array");
    const int64_t page = pick(-3, 50), pos = pick(0, 1 << 21), slot = slot_of(pos, a.page_shift, page, a.pages);
    CHECK(slot == -1 ? page < 0 || page >= a.pages : slot >> a.page_shift == page && slot < (a.pages << a.page_shift), "slot on its page");
  }
}

// The keys that the tile of flat rows [flat0, flat0 + n) of a sequence (or of all, in
// the shared part) takes for each of its rows, counted, over all chunks.
// (of one of the heads: a row's heads may lie in two tiles).
static void count_tile(const AttentionArgs& a, const SequenceWork& w, int tile, int tile_rows, int chunks, int head,
                       std::vector<std::vector<int>>* seen) {
  const int flats = w.rows * a.ratio, flat0 = tile * tile_rows, flat1 = std::min(flats, flat0 + tile_rows);
  const int t0 = flat0 / a.ratio, t1 = (flat1 - 1) / a.ratio;
  int lo_first, hi_last, hi_first, lo_last;          // as the kernel's Span
  if (a.part == kSharedPart) {
    lo_first = INT32_MAX, hi_first = INT32_MAX, lo_last = 0, hi_last = 0;
    for (int t = t0; t <= t1; ++t) {
      int lo, hi;
      visible(a, w, t, &lo, &hi);
      if (hi > lo) lo_first = std::min(lo_first, lo);
      else if (sink_end(a) == 0) lo = hi = 0;
      hi_first = std::min(hi_first, hi);
      lo_last = std::max(lo_last, lo);
      hi_last = std::max(hi_last, hi);
    }
    if (lo_first > hi_last) lo_first = hi_last;
  } else {
    visible(a, w, t0, &lo_first, &hi_first);
    visible(a, w, t1, &lo_last, &hi_last);
  }
  const int first = first_key(a), sinks = sink_end(a);
  int last_step = -1, expected = 0;
  for (int chunk = 0; chunk < chunks; ++chunk) {
    const TileSteps<true> s = tile_steps<true>(a, lo_first, hi_last, chunk, chunks);
    CHECK(s.begin <= s.end, "places in order");
    if (chunk == 0) expected = s.begin;
    if (s.begin < s.end) CHECK(s.begin == expected, "chunks adjoin");
    if (s.begin < s.end) expected = s.end;
    for (int place = s.begin; place < s.end; ++place) {
      const int step = s.step_at(place);
      CHECK(step > last_step, "steps in order");
      last_step = step;
      CHECK(step >= 0 && step <= w.keys / kStep, "steps inside the sequence");
      const bool masked = step_masked(step, lo_last, hi_first);
      for (int f = flat0; f < flat1; ++f) {
        if (f % a.ratio != head) continue;
        int lo, hi;
        visible(a, w, f / a.ratio, &lo, &hi);
        for (int j = step * kStep; j < (step + 1) * kStep; ++j) {
          const bool sees = j < hi && (j >= lo || (j >= first && j < sinks));
          CHECK(sees || masked, "a hidden token in a step that hides none");
          if (sees) {
            const int row = w.first + f / a.ratio;
            CHECK(row < (int)seen->size() && j < (int)(*seen)[row].size(), "a key of the sequence");
            ++(*seen)[row][j];
          }
        }
      }
    }
  }
}

static void attention() {
  for (int trial = 0; trial < 1500; ++trial) {
    AttentionArgs a{};
    const int groups[] = {32, 64, 128}, Ds[] = {64, 128, 256}, ratios[] = {1, 2, 3, 4, 8};
    const int D = Ds[pick(0, 2)], group = std::min(D, groups[pick(0, 2)]);
    a.c = CacheView{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 1000, 4, (int)pick(1, 4), D, group, (D + group - 1) / group, cache_blocks(D), 0};
    a.ratio = ratios[pick(0, 4)];
    const int B = (int)pick(1, trial % 9 == 0 ? 80 : 8);
    const bool wild = trial % 4 == 3, one = trial % 4 == 2;
    const int64_t most = trial % 3 == 0 ? 1500 : 300;
    std::vector<int32_t> lens(B), starts(B + 1);
    for (int b = 0; b < B; ++b) {
      lens[b] = (int32_t)pick(wild ? -50 : 0, most);
      starts[b + 1] = starts[b] + (int32_t)(one ? 1 : pick(0, pick(0, 3) ? 3 : 70));
      if (!wild && !one) lens[b] = std::max(lens[b], starts[b + 1] - starts[b]);
      if (!wild && one) lens[b] = std::max(lens[b], 1);
    }
    if (wild) for (auto& s : starts) s += 3;
    a.r = RowsView{nullptr, 0, (most >> 4) + (wild ? -3 : 1), lens.data(), one ? nullptr : starts.data(), B,
                   one ? B : std::max<int64_t>(1, starts[B] + (wild ? pick(-3, 5) : 0))};
    a.causal = (int)pick(0, 3) > 0;
    a.window = a.causal && pick(0, 2) ? pick(1, pick(0, 1) ? 100 : 1200) : 0;
    a.sinks = pick(0, 2) ? pick(0, pick(0, 1) ? 10 : 400) : pick(0, 1) ? INT64_MAX : 0;
    const int32_t shared = (int32_t)(pick(0, 4) ? pick(0, most + 100) : pick(-100, 0));
    a.shared = &shared;
    a.least_shared = (int)pick(0, 1) * (int)pick(0, 500);
    // what each row sees, by the definition
    const int64_t cover = a.r.max_pages << 4;
    std::vector<std::vector<int>> want(a.r.rows), whole(a.r.rows), parts(a.r.rows);
    std::vector<int> owner(a.r.rows, -1);
    for (int t = 0; t < a.r.rows; ++t) {
      int b = -1;
      int64_t pos;
      if (!find_row(a.r, t, &b, &pos)) continue;
      owner[t] = b;
      const int n = (int)std::max<int64_t>(0, std::min<int64_t>(lens[b], cover));
      want[t].assign(n, 0);
      for (int j = 0; j < n; ++j)
        want[t][j] = (!a.causal || j <= pos) && (a.window == 0 || j > pos - a.window || j < a.sinks);
      whole[t].assign(n, 0);
      parts[t].assign(n, 0);
    }
    auto run = [&](AttentionArgs x, std::vector<std::vector<int>>* seen) {
      RowsView r = x.r;
      if (x.part == kSharedPart) {
        x.all = B;
        x.r.batch = r.batch = 1;
      }
      const int groups = x.c.C / scale_blocks(x.c), tall = 16 * max_tiles(x.c.C, groups, x.c.affine);
      const int heights[] = {tile_rows_of(x.c, r, x.ratio), 16, tall, wide_tiles(x.c.C, groups, x.c.affine) > 0 ? kWideRows : 16};
      Schedule s = plan_for(x.c, r, x.ratio, heights[pick(0, 3)], pick(0, 1) ? 8 : 16);
      s.partial = x.part != kWhole;
      // the cut: blocks inside the grid, partial results inside the workspace
      if (s.target > 0) {
        double work = 0, tiles = 0;
        int longest = 0;
        for (int b = 0; b < x.r.batch; ++b) {
          const SequenceWork w = sequence_work(x, s.tile_rows, b);
          work += (double)w.tiles * w.steps;
          tiles += w.tiles;
          if (w.tiles > 0) longest = std::max(longest, w.steps);
        }
        const int per = steps_per_block(s, (float)work, (float)tiles, longest, [&](int n) {
          int sum = 0;
          for (int b = 0; b < x.r.batch; ++b) {
            const SequenceWork w = sequence_work(x, s.tile_rows, b);
            if (w.tiles > 0) sum += (chunks_of(w.steps, n) - 1) * w.tiles;
          }
          return sum;
        });
        int64_t all = 0, slots = 0;
        for (int b = 0; b < x.r.batch; ++b) {
          const SequenceWork w = sequence_work(x, s.tile_rows, b);
          const int chunks = chunks_of(w.steps, per);
          all += (int64_t)w.tiles * chunks;
          if (chunks > 1 || leaves_parts(x, s)) slots += (int64_t)w.tiles * chunks;
        }
        CHECK(all <= s.units, "blocks inside the grid");
        CHECK(slots <= workspace_slots(s), "partial results inside the workspace");
      }
      if (s.target == 0) s.target = 1;
      int64_t blocks = 0;
      const int head = (int)pick(0, x.ratio - 1);
      for (int b = 0; b < x.r.batch; ++b) {
        const SequenceWork w = sequence_work(x, s.tile_rows, b);
        CHECK(w.rows == 0 || (w.first >= 0 && w.first + w.rows <= x.r.rows), "rows inside the call");
        const int chunks = chunks_of(w.steps, (int)pick(1, 20));
        for (int tile = 0; tile < w.tiles; ++tile) count_tile(x, w, tile, s.tile_rows, chunks, head, seen);
        blocks += (int64_t)w.tiles * chunks_of(w.steps, std::max(s.min_steps, w.steps));
      }
      CHECK(blocks <= s.units, "a block for every tile");
      if (s.partial) {
        CHECK(workspace_slots(s) == s.units, "a partial result for every block");
        void* const p = malloc((size_t)workspace_bytes(s, x.c.heads, x.c.C, x.r.batch));
        const Workspace ws = workspace_at(p, s, x.c.heads, x.c.C);
        ws.part[(int64_t)s.units * x.c.heads * partial_floats(s.tile_rows, x.c.C) - 1] = 1.0f;
        ws.record[s.units - 1].chunks = 1;
        *ws.used = 1;
        if (s.planned) ws.plan[x.r.batch].slots = 1;
        free(p);
      }
    };
    AttentionArgs x = a;
    run(x, &whole);
    x.part = kOwnPart;
    run(x, &parts);
    x.part = kSharedPart;
    // rows that no sequence owns lie between two sequences where starts decrease; here none do
    bool inside = true;
    const int s0 = a.r.starts ? starts[0] : 0, s1 = a.r.starts ? starts[B] : B;
    for (int t = std::max(0, s0); t < std::min<int64_t>(s1, a.r.rows); ++t) inside &= owner[t] >= 0;
    CHECK(inside, "owned rows are one run");
    run(x, &parts);
    for (int t = 0; t < a.r.rows; ++t) {
      CHECK(whole[t] == want[t], "the keys a row sees, each once");
      CHECK(parts[t] == want[t], "the keys a row sees, each once in one of the parts");
    }
  }
}

// Plans whose contents are of no sense: nothing out of range.
static void senseless() {
  for (int trial = 0; trial < 1500; ++trial) {
    AttentionArgs a{};
    a.c = CacheView{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 1000, 4, 1, 64, 64, 1, 2, 0};
    a.ratio = (int)pick(1, 5);
    const int B = (int)pick(1, 6);
    auto any = [&] { return (int32_t)(pick(0, 3) ? pick(-40, 400) : pick(0, 1) ? INT32_MAX - pick(0, 2) : INT32_MIN + pick(0, 2)); };
    std::vector<int32_t> lens(B), starts(B + 1);
    for (auto& x : lens) x = any();
    for (auto& x : starts) x = any();
    const int32_t shared = any();
    a.shared = &shared;
    a.r = RowsView{nullptr, 0, pick(0, 100), lens.data(), starts.data(), B, pick(1, 200)};
    a.causal = (int)pick(0, 1);
    a.window = a.causal ? pick(0, 300) : 0;
    a.sinks = pick(0, 1) ? pick(0, 300) : INT64_MAX;
    for (int part = kWhole; part <= kSharedPart; ++part) {
      AttentionArgs x = a;
      x.part = part;
      if (part == kSharedPart) x.all = B, x.r.batch = 1;
      for (int b = 0; b < x.r.batch; ++b) {
        const SequenceWork w = sequence_work(x, 16, b);
        CHECK(w.rows >= 0 && (w.rows == 0 || (w.first >= 0 && w.first + w.rows <= x.r.rows)), "rows inside the call");
        CHECK(w.steps >= 1 && w.keys >= 0 && w.keys <= (x.r.max_pages << 4), "keys inside the table");
        for (int t = 0; t < w.rows; t += 7) {
          int lo, hi;
          visible(x, w, t, &lo, &hi);
          CHECK(0 <= lo && lo <= hi && hi <= w.keys, "visible keys of the sequence");
          const TileSteps<true> s = tile_steps<true>(x, lo, hi, (int)pick(0, 3), 4);
          CHECK(s.begin <= s.end, "places in order");
          for (int place = s.begin; place < s.end; ++place)
            CHECK(s.step_at(place) >= 0 && s.step_at(place) <= w.keys / kStep, "steps inside the sequence");
        }
      }
    }
  }
}

static void entry_points() {
  alignas(256) static unsigned char arena[4096];
  int4_cache_t c{arena, (uint16_t*)arena, nullptr, arena, (uint16_t*)arena, nullptr, 4, 64, 2, 128, 64};
  int4_cache_rows_t r{(int32_t*)arena, 50, 50, (int32_t*)arena, (int32_t*)arena, 3, 7};
  int4_cache_pool_t pool{(int32_t*)arena, 50, 50, 3, 64, (int32_t*)arena, 9};
  int4_cache_transform_t t{(float*)arena, (float*)arena, 1e-6, (float*)arena, 128, 100, 128, 0};
  int32_t* const I = (int32_t*)arena;
  void* const P = arena;
  CHECK(int4_cache_release(&pool, I, arena, I, nullptr, I, I, nullptr) == INT4DQ_OK && calls == 1, "release");
  CHECK(int4_cache_extend(&pool, I, nullptr, I, I, I, (int64_t*)arena, 5, I, nullptr) == INT4DQ_OK && calls == 2, "extend");
  CHECK(int4_cache_append(&c, &r, &t, P, 512, 128, 4, P, 256, 128, P, 256, 128, 2, P, nullptr) == INT4DQ_OK && calls == 3, "append");
  auto attend = [&](int64_t sinks, const int32_t* shared, int64_t window, void* ws, int64_t bytes) {
    return int4_cache_attention_ex(&c, &r, P, 512, 128, 1, 4, 1.0f, 1, window, sinks, shared, -1, P, nullptr, ws, bytes, nullptr);
  };
  CHECK(attend(4, nullptr, 100, P, 256) == INT4DQ_OK && calls == 4 && shared_calls == 0, "sinks");
  CHECK(attend(0, I, 0, P, 256) == INT4DQ_OK && calls == 4 && shared_calls == 1, "shared");
  CHECK(attend(INT64_MAX, I, 5, nullptr, 0) == INT4DQ_OK && shared_calls == 2, "both, without a workspace");
  CHECK(attend(-1, nullptr, 100, P, 256) == INT4DQ_EINVAL && strstr(int4_last_error(), "sinks"), "sinks below 0");
  CHECK(attend(4, nullptr, -1, P, 256) == INT4DQ_EINVAL && strstr(int4_last_error(), "int4_cache_attention_ex"), "window");
  CHECK(attend(4, I, 9, arena + 16, 256) == INT4DQ_EINVAL && strstr(int4_last_error(), "aligned"), "workspace alignment");
  CHECK(attend(4, I, 9, nullptr, 256) == INT4DQ_EINVAL, "no workspace");
  CHECK(int4_cache_attention_ex_workspace_bytes(&c, &r, 4, 0, -1) == 512, "workspace");
  CHECK(int4_cache_attention_ex_workspace_bytes(&c, &r, 4, 1, -1) == 1024, "workspace of shared tokens");
  CHECK(int4_cache_attention_ex_workspace_bytes(&c, &r, 5, 1, -1) == -1, "workspace: q_heads");
  r.rows = 0;
  CHECK(int4_cache_attention_ex_workspace_bytes(&c, &r, 4, 1, -1) == 0, "no rows, no workspace");
  CHECK(attend(4, I, 9, P, 256) == INT4DQ_OK && calls == 4 && shared_calls == 2, "no rows");
}

// Only the last round's tiles cut: each tile in as many blocks as it has chunks, all of
// them in the grid, and the cut ones' partial results in the workspace.
static void last_round() {
  for (int trial = 0; trial < 3000; ++trial) {
    Schedule s{};
    s.tile_rows = kWideRows;
    s.target = (int)pick(1, 40);
    s.min_steps = pick(0, 1) ? 8 : 16;
    s.crowded = (int)pick(0, 1);
    const int tiles = (int)pick(0, 4 * s.target), most = (int)pick(0, 100);
    s.units = s.target * (s.crowded ? 2 : 1) + tiles + (int)pick(0, 3);
    cut_last_round(&s);
    const int chunks = last_round_chunks(s, tiles, most), left = tiles % s.target;
    CHECK(chunks >= 1 && (chunks == 1 || (chunks - 1) * s.min_steps < most) && left * chunks <= workspace_slots(s), "chunks of the last round");
    std::vector<std::vector<int>> seen(tiles);
    std::vector<int> slots(workspace_slots(s));
    for (int unit = 0; unit < s.units; ++unit) {
      const UnitShare x = last_round_share(s, tiles, chunks, unit);
      if (x.tile < 0 || x.tile >= tiles) continue;         // the kernel finds no sequence with it
      CHECK(x.chunk >= 0 && x.chunk < x.chunks && (x.chunks == 1 || x.chunks == chunks), "chunk");
      seen[x.tile].resize(x.chunks);
      ++seen[x.tile][x.chunk];
      if (x.chunks > 1) {
        CHECK(x.slot >= 0 && x.slot < left * chunks && slots[x.slot]++ == 0, "a slot of its own");
        CHECK(x.slot % x.chunks == x.chunk, "a tile's slots side by side");
      }
    }
    for (int t = 0; t < tiles; ++t) {
      CHECK((int)seen[t].size() == (t < tiles - left ? 1 : chunks), "all of a tile's chunks");
      for (const int n : seen[t]) CHECK(n == 1, "each chunk once");
    }
  }
}

int main() {
  entry_points();
  pages();
  last_round();
  attention();
  senseless();
  if (failures) return 1;
  printf("all checks passed\n");
  return 0;
}
