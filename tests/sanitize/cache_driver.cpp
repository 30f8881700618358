// cache_driver.cpp -- the host side of the 4-bit cache (include/int4dq_cache.h)
// under AddressSanitizer and UndefinedBehaviorSanitizer: every refusal of the
// entry points, with the kernel launchers replaced by stubs; and the index
// arithmetic that the kernels share with the host (cache.h, cache_schedule.h) on
// sound and on senseless plans: every address a row's codes and scales would be
// read from or written to lies inside the cache, every block and partial result
// inside the grid and the workspace, every key of every row in exactly one block.
//
// Test infrastructure: built and run only by tests/test_sanitize_cache_cpu.py.
// Exit status 0 when every check holds.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <random>
#include <vector>

#include "../../dequantizing_gemm_amd/csrc/cache.h"
#include "../../dequantizing_gemm_amd/csrc/cache_schedule.h"
#include "../../include/int4dq_cache.h"

static int failures = 0;
static int calls = 0;
static int64_t last_ws = -1;
static int last_wide = -1;
#define CHECK(cond, what)                                                                      \
  do {                                                                                         \
    if (!(cond)) {                                                                             \
      ++failures;                                                                              \
      fprintf(stderr, "FAIL line %d: %s (last error: \"%s\")\n", __LINE__, what, int4_last_error()); \
    }                                                                                          \
  } while (0)

namespace int4dq {
hipError_t launch_cache_write(const CacheView&, const RowsView&, const void*, int64_t, int64_t, const void*, int64_t,
                              int64_t, int, hipStream_t) { ++calls; return hipSuccess; }
hipError_t launch_cache_read(const CacheView&, const RowsView&, void*, void*, int, hipStream_t) { ++calls; return hipSuccess; }
hipError_t launch_cache_attention(const AttentionArgs& a, void*, int64_t bytes, hipStream_t) {
  ++calls;
  last_ws = bytes;
  last_wide = a.q_wide;
  return hipSuccess;
}
int64_t cache_attention_workspace(const CacheView& c, const RowsView& r, int ratio) {
  const Schedule s = plan_of(c, r, ratio);
  return s.target == 0 ? 0 : workspace_bytes(s, c.heads, c.C, r.batch);
}
}  // namespace int4dq
extern "C" const char* int4_last_error(void);

using namespace int4dq;
static std::mt19937_64 rng(1);
static int64_t pick(int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); }

// The exactly sized arrays of a cache; touching them checks an index.
struct Arrays {
  std::vector<uint8_t> kp, vp, kz, vz;
  std::vector<uint16_t> ks, vs;
  explicit Arrays(const CacheView& c) {
    const size_t units = (size_t)c.pages * c.heads << (c.page_shift - 4);
    kp.resize(units * 16 * c.row_bytes());
    vp.resize(kp.size());
    ks.resize(units * 16 * c.G);
    vs.resize(ks.size());
    kz.resize(ks.size());
    vz.resize(ks.size());
  }
};

static CacheView view(int D, int group, int heads, int shift, int pages) {
  if (group > D) group = D;
  return CacheView{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, pages, shift, heads, D, group,
                   (D + group - 1) / group, cache_blocks(D), (int)pick(0, 1)};
}

static void rows_and_pages() {
  for (int trial = 0; trial < 400; ++trial) {
    const int Ds[] = {1, 33, 64, 72, 80, 96, 128, 160, 192, 250, 256}, gs[] = {32, 64, 128, 256};
    const CacheView c = view(Ds[pick(0, 10)], gs[pick(0, 3)], (int)pick(1, 3), (int)pick(4, 7), (int)pick(1, 6));
    Arrays m(c);
    const int B = (int)pick(1, 9), mp = (int)pick(0, 4), stride = mp + (int)pick(0, 3);
    const bool wild = trial & 1;
    std::vector<int32_t> table(B * stride + 1), lens(B), starts(B + 1);
    for (auto& p : table) p = (int32_t)(wild ? pick(-3, 9) * (pick(0, 9) ? 1 : 300000000) : pick(0, c.pages - 1));
    for (auto& l : lens) l = (int32_t)(wild ? pick(0, 5) ? pick(-40, 400) : (pick(0, 1) ? INT32_MAX : INT32_MIN) : pick(0, (int64_t)mp << c.page_shift));
    for (int b = 1; b <= B; ++b) starts[b] = wild ? (int32_t)pick(-5, 60) : starts[b - 1] + (int32_t)pick(0, 20);
    if (wild && pick(0, 3) == 0) starts[pick(0, B)] = pick(0, 1) ? INT32_MAX : INT32_MIN;
    const bool one = trial % 5 == 0;
    const int64_t T = one ? B : pick(1, 70);
    const RowsView r{table.data(), stride, mp, lens.data(), one ? nullptr : starts.data(), B, T};
    for (int64_t t = 0; t < T; ++t) {
      int b = -1;
      int64_t pos = 0;
      if (!find_row(r, t, &b, &pos)) continue;
      CHECK(b >= 0 && b < B, "sequence inside the batch");
      if (!wild && !one) CHECK(starts[b] <= t && t < starts[b + 1], "the row's own sequence");
      const int64_t page = find_page(r, c, b, pos);
      if (page < 0) continue;
      CHECK(page < c.pages, "page inside the cache");
      const int slot = (int)(pos & ((1 << c.page_shift) - 1)), ts = slot & 15, DB = c.row_bytes();
      for (int h = 0; h < c.heads; ++h) {
        const int64_t u = c.unit(page, h, slot);
        m.kp.at(u * 16 * DB + ts * DB) = 1;
        m.kp.at(u * 16 * DB + ts * DB + 3 * 4 * c.C + 4 * (c.C - 1) + 3) = 1;
        m.vp.at(u * 16 * DB + ts) = 1;
        m.vp.at(u * 16 * DB + (int64_t)(4 * c.C - 1) * 64 + 48 + ts) = 1;
        m.ks.at((u * c.G) * 16 + ts) = 1;
        m.vz.at((u * c.G + c.G - 1) * 16 + ts) = 1;
      }
    }
  }
}

static void schedules() {
  for (int trial = 0; trial < 600; ++trial) {
    const int Ds[] = {64, 96, 128, 192, 256}, gs[] = {32, 64, 128, 256};
    AttentionArgs a{};
    a.c = view(Ds[pick(0, 4)], gs[pick(0, 3)], (int)pick(1, 12), (int)pick(4, 8), 1000);
    const int ratios[] = {1, 2, 3, 4, 7, 8, 16, 33};
    a.ratio = ratios[pick(0, 7)];
    const int B = (int)pick(1, trial % 7 == 0 ? 300 : 20);
    const bool wild = trial % 4 == 3, one = trial % 4 == 2;
    const int64_t most = trial % 3 == 0 ? 200000 : trial % 3 == 1 ? 3000 : 90;
    std::vector<int32_t> lens(B), starts(B + 1);
    for (int b = 0; b < B; ++b) {
      lens[b] = (int32_t)pick(wild ? -50 : 0, most);
      starts[b + 1] = starts[b] + (int32_t)(one ? 1 : pick(0, pick(0, 3) ? 3 : 400));
    }
    if (wild) for (auto& s : starts) s += 3;
    a.r = RowsView{nullptr, 0, (most >> a.c.page_shift) + (wild ? -1 : 1), lens.data(), one ? nullptr : starts.data(), B,
                   (int64_t)starts[B] + (wild ? pick(-3, 5) : 0)};
    if (a.r.max_pages < 0) a.r.max_pages = 0;
    if (a.r.rows < 1) a.r.rows = 1;
    if (one) a.r.rows = B;
    a.causal = (int)pick(0, 1);
    a.window = a.causal && pick(0, 1) ? pick(1, 5000) : 0;
    Schedule s = plan_of(a.c, a.r, a.ratio);
    CHECK(s.tile_rows == 16 || s.tile_rows == 32 || s.tile_rows == kWideRows, "tile height");
    CHECK(s.tile_rows != kWideRows || wide_tiles(a.c.C, a.c.C / scale_blocks(a.c), a.c.affine) > 0, "a form for prompts");
    CHECK(s.tile_rows == kWideRows || s.tile_rows <= 16 * max_tiles(a.c.C, a.c.C / scale_blocks(a.c), a.c.affine), "a tile height that has a form");
    CHECK(a.c.C % scale_blocks(a.c) == 0 && (a.c.G == 1 || a.c.group % (32 * scale_blocks(a.c)) == 0), "blocks to a scale");
    if (trial % 5 == 4) { s.units -= s.target * (s.crowded ? 2 : 1); s.target = s.crowded = s.planned = 0; }
    {
      void* const p = malloc((size_t)workspace_bytes(s, a.c.heads, a.c.C, B));
      const Workspace ws = workspace_at(p, s, a.c.heads, a.c.C);
      *ws.used = 1;
      if (s.planned) ws.plan[B].slots = 1;
      if (s.target > 0) {
        ws.record[0].chunk = ws.record[workspace_slots(s) - 1].chunks = 1;
        ws.part[workspace_slots(s) * (a.c.heads * partial_floats(s.tile_rows, a.c.C)) - 1] = 1.0f;
      }
      free(p);
    }
    if (a.r.starts)
      for (int b = 0; b < B; ++b)
        CHECK(tiles_before(a, s, b + 1) - tiles_before(a, s, b) >= sequence_work(a, s.tile_rows, b).tiles &&
                  tiles_before(a, s, b + 1) <= s.units, "a block for every tile");
    double all = 0, tiles = 0;
    int most_steps = 0;
    for (int b = 0; b < B; ++b) {
      const SequenceWork w = sequence_work(a, s.tile_rows, b);
      all += (double)w.tiles * w.steps;
      tiles += w.tiles;
      if (w.tiles > 0 && w.steps > most_steps) most_steps = w.steps;
    }
    for (const double off : {1.0 - 3e-5, 1.0, 1.0 + 3e-5}) {     // binary32 sums in some order
      if (s.target == 0 && off != 1.0) continue;
      auto added = [&](int x) {
        int sum = 0;
        for (int b = 0; b < B; ++b) {
          const SequenceWork w = sequence_work(a, s.tile_rows, b);
          if (w.tiles > 0) sum += (chunks_of(w.steps, x) - 1) * w.tiles;
        }
        return sum;
      };
      const int per = s.target == 0 ? INT32_MAX / 2 : steps_per_block(s, (float)(all * off), (float)tiles, most_steps, added);
      CHECK(per >= s.min_steps, "the least share");
      if (s.target > 0)
        CHECK(added(per) <= (tiles <= s.target ? s.target - (int)tiles : s.crowded ? 2 * s.target : s.target), "room for the cuts");
      int64_t blocks = 0, slots = 0, rows = 0;
      for (int b = 0; b < B; ++b) {
        const SequenceWork w = sequence_work(a, s.tile_rows, b);
        const int chunks = chunks_of(w.steps, per);
        blocks += (int64_t)w.tiles * chunks;
        CHECK(chunks >= 1 && (s.target > 0 || chunks == 1), "chunks");
        if (chunks > 1) slots += (int64_t)w.tiles * chunks;
        rows += w.rows;
        CHECK(w.rows == 0 || (w.first >= 0 && w.first + w.rows <= a.r.rows), "rows inside the call");
        CHECK((int64_t)w.tiles * s.tile_rows >= (int64_t)w.rows * a.ratio, "tiles cover the rows");
        const int flats = w.rows * a.ratio;
        for (int t = 0; t < w.tiles; t += 1 + w.tiles / 3) {
          int lo, hi, lo1, hi1, at = -1, begin, end;
          const int last = ((t + 1) * s.tile_rows < flats ? (t + 1) * s.tile_rows : flats) - 1;
          visible(a, w, t * s.tile_rows / a.ratio, &lo, &hi);
          visible(a, w, last / a.ratio, &lo1, &hi1);
          CHECK(lo >= 0 && lo <= hi && lo <= lo1 && hi <= hi1 && hi1 <= w.keys, "visible keys in order");
          for (int k = 0; k < chunks; ++k) {
            chunk_steps(lo, hi1, k, chunks, &begin, &end);
            CHECK(begin <= end, "chunk in order");
            if (begin < end) {
              CHECK(at < 0 ? begin == lo / kStep : begin == at, "chunks adjoin");
              at = end;
            }
          }
          if (hi1 > lo) CHECK(at == (hi1 - 1) / kStep + 1, "chunks reach the last key");
          else CHECK(at == -1, "no keys, no steps");
        }
      }
      CHECK(blocks <= s.units, "blocks inside the grid");
      CHECK(slots <= workspace_slots(s), "partial results inside the workspace");
    }
  }
}

// A sequence of 2^31 - 1 tokens: its last steps, and those that loads ask for ahead.
static void the_longest() {
  AttentionArgs a{};
  a.c = view(64, 64, 1, 4, 1);
  a.ratio = 1;
  a.causal = 1;
  const int32_t length = INT32_MAX, last = INT32_MAX / kStep;
  a.r = RowsView{nullptr, 1 << 27, 1 << 27, &length, nullptr, 1, 1};
  for (const int64_t window : {(int64_t)0, (int64_t)INT32_MAX - 1, (int64_t)INT32_MAX, (int64_t)1 << 40, (int64_t)100}) {
    a.window = window;
    const SequenceWork w = sequence_work(a, 16, 0);
    CHECK(w.keys == INT32_MAX && w.steps >= 1 && w.steps <= last + 1, "steps of the longest sequence");
    CHECK(window == 100 ? w.steps < 8 : w.steps == last + 1, "a window as long as the sequence");
    int lo, hi, begin, end;
    visible(a, w, 0, &lo, &hi);
    chunk_steps(lo, hi, 6, 7, &begin, &end);
    CHECK(end == last + 1 && hi == INT32_MAX, "its last chunk");
    CHECK(step_masked(last, lo, hi) && !step_masked(last - 1, lo - (window == 100 ? 200 : 0), hi), "the last step is masked");
  }
  for (int ahead = 0; ahead <= 8; ++ahead)
    for (int u = 0; u < 4; ++u)
      CHECK(unit_token(last + ahead, u) >> 4 == ((uint64_t)(last + ahead) * kStep + 16 * u) >> 4, "units ahead of the end");
}

static void refusals() {
  alignas(256) static unsigned char arena[4096];
  int4_cache_t c{arena, (uint16_t*)arena, nullptr, arena, (uint16_t*)arena, nullptr, 4, 64, 2, 128, 64};
  int4_cache_rows_t r{(int32_t*)arena, 50, 50, (int32_t*)arena, (int32_t*)arena, 3, 7};
  void* const P = arena;
  auto all = [&](const char* needle) {
    const int before = calls;
    const int rc[3] = {int4_cache_write(&c, &r, P, 256, 128, P, 256, 128, INT4DQ_ROWS_BF16, nullptr), 0, 0};
    CHECK(rc[0] == INT4DQ_EINVAL && strstr(int4_last_error(), needle) && strstr(int4_last_error(), "int4_cache_write"), needle);
    CHECK(int4_cache_read(&c, &r, P, P, INT4DQ_ROWS_F16, nullptr) == INT4DQ_EINVAL && strstr(int4_last_error(), needle), needle);
    CHECK(int4_cache_attention(&c, &r, P, 512, 128, INT4DQ_ROWS_F16, 4, 1.0f, 1, 0, P, nullptr, nullptr, 0, nullptr) ==
                  INT4DQ_EINVAL && strstr(int4_last_error(), needle), needle);
    CHECK(calls == before, "nothing launched");
  };
#define WITH(field, value, needle)           \
  do {                                       \
    const auto keep = field;                 \
    field = value;                           \
    all(needle);                             \
    field = keep;                            \
  } while (0)
  CHECK(int4_cache_write(&c, &r, P, 256, 128, P, 256, 128, INT4DQ_ROWS_BF16, nullptr) == INT4DQ_OK && calls == 1, "write");
  CHECK(int4_cache_read(&c, &r, P, P, INT4DQ_ROWS_F32, nullptr) == INT4DQ_OK && calls == 2, "read");
  auto attend = [&](const void* q, int64_t rs, int64_t hs, int dt, int64_t H, float scale, int causal, int64_t window,
                    void* out, void* ws, int64_t bytes) {
    return int4_cache_attention(&c, &r, q, rs, hs, dt, H, scale, causal, window, out, nullptr, ws, bytes, nullptr);
  };
  CHECK(attend(P, 512, 128, 1, 4, 1.0f, 1, 0, P, P, 256) == INT4DQ_OK && last_wide == 1 && last_ws == 256, "attention");
  CHECK(attend(arena + 2, 512, 128, 1, 4, 1.0f, 1, 0, P, P, 256) == INT4DQ_OK && last_wide == 0, "an odd address");
  CHECK(attend(P, 509, 128, 1, 4, 1.0f, 1, 0, P, P, 256) == INT4DQ_OK && last_wide == 0, "an odd stride");
  WITH(c.head_dim, 0, "head_dim"); WITH(c.head_dim, 257, "head_dim");
  WITH(c.group, 0, "group"); WITH(c.group, 48, "group"); WITH(c.group, 96, "group"); WITH(c.group, -1, "group");
  WITH(c.heads, 0, "heads"); WITH(c.heads, 65536, "heads");
  WITH(c.page_size, 8, "page_size"); WITH(c.page_size, 48, "page_size"); WITH(c.page_size, 1 << 21, "page_size"); WITH(c.page_size, 0, "page_size");
  WITH(c.pages, 0, "pages"); WITH(c.pages, INT64_MAX, "pages");
  WITH(c.k_packed, nullptr, "non-NULL"); WITH(c.v_scales, nullptr, "non-NULL");
  WITH(c.k_zeros, arena, "both"); WITH(c.v_zeros, arena, "both");
  WITH(c.v_packed, arena + 8, "aligned"); WITH(c.k_scales, (uint16_t*)(arena + 2), "aligned");
  WITH(r.batch, -1, "batch"); WITH(r.batch, INT64_MAX, "batch");
  WITH(r.rows, -1, "rows"); WITH(r.rows, INT64_MAX, "rows"); WITH(r.starts, nullptr, "one row a sequence");
  WITH(r.max_pages, -1, "max_pages"); WITH(r.table_stride, 4, "table_stride"); WITH(r.table_stride, INT64_MAX, "table_stride");
  WITH(r.lengths, nullptr, "lengths"); WITH(r.page_table, nullptr, "page_table");
  {
    const int before = calls;
    CHECK(int4_cache_write(nullptr, &r, P, 1, 1, P, 1, 1, 0, nullptr) == INT4DQ_EINVAL, "no cache");
    CHECK(int4_cache_write(&c, nullptr, P, 1, 1, P, 1, 1, 0, nullptr) == INT4DQ_EINVAL, "no rows");
    CHECK(int4_cache_write(&c, &r, P, 1, 1, P, 1, 1, 3, nullptr) == INT4DQ_EINVAL, "dtype");
    CHECK(int4_cache_write(&c, &r, nullptr, 1, 1, P, 1, 1, 0, nullptr) == INT4DQ_EINVAL, "no k");
    CHECK(int4_cache_write(&c, &r, P, INT64_MAX, 1, P, 1, 1, 0, nullptr) == INT4DQ_EINVAL, "stride");
    CHECK(int4_cache_write(&c, &r, P, 1, 1, P, 1, INT64_MIN, 0, nullptr) == INT4DQ_EINVAL, "stride");
    CHECK(int4_cache_read(&c, &r, P, nullptr, 0, nullptr) == INT4DQ_EINVAL, "no v");
    CHECK(int4_cache_read(&c, &r, P, P, -1, nullptr) == INT4DQ_EINVAL, "dtype");
    CHECK(attend(P, 1, 1, 0, 4, 1.0f, 1, 0, P, nullptr, 0) == INT4DQ_EINVAL, "binary32 queries");
    CHECK(attend(P, 1, 1, 1, 3, 1.0f, 1, 0, P, nullptr, 0) == INT4DQ_EINVAL, "q_heads");
    CHECK(attend(P, 1, 1, 1, 65536, 1.0f, 1, 0, P, nullptr, 0) == INT4DQ_EINVAL, "q_heads");
    CHECK(attend(P, 1, 1, 1, 4, 0.0f, 1, 0, P, nullptr, 0) == INT4DQ_EINVAL, "scale 0");
    CHECK(attend(P, 1, 1, 1, 4, -1.0f, 1, 0, P, nullptr, 0) == INT4DQ_EINVAL, "scale below 0");
    CHECK(attend(P, 1, 1, 1, 4, __builtin_nanf(""), 1, 0, P, nullptr, 0) == INT4DQ_EINVAL, "scale NaN");
    CHECK(attend(P, 1, 1, 1, 4, __builtin_inff(), 1, 0, P, nullptr, 0) == INT4DQ_EINVAL, "scale infinite");
    CHECK(attend(P, 1, 1, 1, 4, 1.0f, 1, -1, P, nullptr, 0) == INT4DQ_EINVAL, "window");
    CHECK(attend(P, 1, 1, 1, 4, 1.0f, 0, 5, P, nullptr, 0) == INT4DQ_EINVAL, "window without causal");
    CHECK(attend(P, 1, INT64_MAX, 1, 4, 1.0f, 1, 0, P, nullptr, 0) == INT4DQ_EINVAL, "stride");
    CHECK(attend(P, 1, 1, 1, 4, 1.0f, 1, 0, P, nullptr, 256) == INT4DQ_EINVAL, "no workspace");
    CHECK(attend(P, 1, 1, 1, 4, 1.0f, 1, 0, P, P, -1) == INT4DQ_EINVAL, "workspace bytes");
    CHECK(attend(P, 1, 1, 1, 4, 1.0f, 1, 0, P, arena + 16, 256) == INT4DQ_EINVAL, "workspace alignment");
    CHECK(attend(nullptr, 1, 1, 1, 4, 1.0f, 1, 0, P, nullptr, 0) == INT4DQ_EINVAL, "no q");
    CHECK(attend(P, 1, 1, 1, 4, 1.0f, 1, 0, nullptr, nullptr, 0) == INT4DQ_EINVAL, "no out");
    CHECK(calls == before, "nothing launched");
    // no rows, no sequences: nothing to do, no pointer needed
    int4_cache_rows_t none = r;
    none.rows = 0;
    CHECK(int4_cache_write(&c, &none, nullptr, 1, 1, nullptr, 1, 1, 0, nullptr) == INT4DQ_OK, "no rows to write");
    CHECK(int4_cache_read(&c, &none, nullptr, nullptr, 0, nullptr) == INT4DQ_OK, "no rows to read");
    none.batch = 0;
    none.lengths = nullptr;
    CHECK(int4_cache_attention(&c, &none, nullptr, 1, 1, 1, 4, 1.0f, 1, 0, nullptr, nullptr, nullptr, 0, nullptr) ==
              INT4DQ_OK, "no sequences");
    CHECK(calls == before, "nothing launched");
    CHECK(int4_cache_attention_workspace_bytes(&c, &none, 4) == 0, "no sequences, no workspace");
    CHECK(int4_cache_attention_workspace_bytes(&c, &r, 4) > 0, "workspace");
    CHECK(int4_cache_attention_workspace_bytes(&c, &r, 5) == -1, "workspace: q_heads");
    CHECK(int4_cache_attention_workspace_bytes(nullptr, &r, 4) == -1, "workspace: no cache");
    r.rows = 1 << 26;
    CHECK(attend(P, 1, 1, 1, 64, 1.0f, 1, 0, P, nullptr, 0) == INT4DQ_EINVAL, "rows * q_heads");
  }
  CHECK(int4_cache_row_bytes(0) == -1 && int4_cache_row_bytes(257) == -1, "row bytes");
  CHECK(int4_cache_row_bytes(1) == 32 && int4_cache_row_bytes(65) == 48 && int4_cache_row_bytes(128) == 64 &&
            int4_cache_row_bytes(129) == 96 && int4_cache_row_bytes(193) == 128, "row bytes");
}

int main() {
  refusals();
  rows_and_pages();
  schedules();
  the_longest();
  if (failures) return 1;
  printf("all checks passed\n");
  return 0;
}
