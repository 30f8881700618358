// cache.h -- what the key/value cache's kernels and entry points share: the
// cache and row descriptors in kernel form, and where a row's codes lie. The
// index arithmetic is host and device code, so that it is also checked on a
// machine without a GPU.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace int4dq {

constexpr int kMaxHeadDim = 256;

// Blocks of 32 channels that hold head_dim channels: the code rows are padded
// to one of five widths, so that five forms of the attention kernel cover all.
__host__ __device__ inline int cache_blocks(int64_t head_dim) {
  const int c = (int)((head_dim + 31) / 32);
  return c <= 2 ? 2 : c == 5 ? 6 : c == 7 ? 8 : c;
}

struct CacheView {
  uint8_t* k_packed;
  uint16_t* k_scales;
  uint8_t* k_zeros;
  uint8_t* v_packed;
  uint16_t* v_scales;
  uint8_t* v_zeros;
  int64_t pages;
  int page_shift;   // log2 of the tokens on a page
  int heads, D, group, G, C;
  int affine;       // whether there are zero points (known also where the pointers are not given)

  // Index of the 16-token unit that holds `slot` of `page`, counted over the
  // whole cache: its codes start at unit * 16 * DB bytes (keys and values) and
  // its scales and zero points at unit * 16 * G.
  __host__ __device__ int64_t unit(int64_t page, int head, int slot) const {
    return ((page * heads + head) << (page_shift - 4)) + (slot >> 4);
  }
  __host__ __device__ int row_bytes() const { return 16 * C; }
};

struct RowsView {
  const int32_t* table;
  int64_t table_stride;
  int64_t max_pages;
  const int32_t* lengths;
  const int32_t* starts;   // nullptr: one row a sequence
  int batch;
  int64_t rows;

  __host__ __device__ int64_t start(int b) const { return starts ? starts[b] : b; }
};

// Sequence and position of row t: false if no sequence owns it. For any
// contents of starts the sequence found is inside the batch. This is the row
// layout's definition one row at a time, for checks on the host of what the write
// and read kernels' blocks take (StoreBlock).
__host__ __device__ inline bool find_row(const RowsView& r, int64_t t, int* seq, int64_t* pos) {
  int b = (int)t;
  if (r.starts) {
    int lo = 0, hi = r.batch;              // the last b with starts[b] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (r.starts[mid] <= t) lo = mid; else hi = mid;
    }
    b = lo;
    if (r.starts[b] > t || r.starts[b + 1] <= t) return false;
  } else if (t >= r.batch) {
    return false;
  }
  *seq = b;
  *pos = (int64_t)r.lengths[b] - (r.start(b + 1) - t);
  return true;
}

// Page of position pos of sequence b, or -1 where it has none.
__host__ __device__ inline int64_t find_page(const RowsView& r, const CacheView& c, int b, int64_t pos) {
  if (pos < 0 || (pos >> c.page_shift) >= r.max_pages) return -1;
  const int64_t page = r.table[b * r.table_stride + (pos >> c.page_shift)];
  return page >= 0 && page < c.pages ? page : -1;
}

// ---------------------------------------------------------------- blocks of the write and read kernels

// 64 positions from `base` of sequence b; its rows start at position p0 with row
// `first` of the call, `rows` of them: slot t of the block is row first + base + t - p0
// where that is one of them.
struct StoreBlock {
  int b, first, rows;
  int64_t p0, base;
};

__host__ __device__ inline StoreBlock store_rows(const RowsView& r, int b) {
  const int s0 = r.starts ? r.starts[b] : b, s1 = r.starts ? r.starts[b + 1] : b + 1;
  StoreBlock x;
  x.b = b;
  x.first = s0 > 0 ? s0 : 0;
  const int last = s1 < r.rows ? s1 : (int)r.rows;
  x.rows = last > x.first ? last - x.first : 0;
  x.p0 = (int64_t)r.lengths[b] - s1 + x.first;
  x.base = x.p0 & ~(int64_t)63;         // positions below 0 among them
  return x;
}

// Before sequence b come at most this many steps (n rows touch at most n / 64 + 2),
// a number that needs no other sequence's length; the grid (store_units) has them all.
__host__ __device__ inline int64_t steps_before(const RowsView& r, int b) {
  const int64_t x = r.starts[b];
  return (x < 0 ? 0 : x < r.rows ? x : r.rows) / 64 + 2 * (int64_t)b;
}
__host__ __device__ inline int64_t store_units(const RowsView& r) {
  return r.starts ? r.rows / 64 + 2 * (int64_t)r.batch : r.batch;
}

// Block `unit` of the grid: false if it has no rows. search(n, x, f): the last i in
// [0, n) with f(i) <= x (lanes.h).
template <typename S>
__host__ __device__ inline bool find_store_block(const RowsView& r, int unit, S search, StoreBlock* out) {
  if (!r.starts) {
    *out = store_rows(r, unit);
    return true;
  }
  const int b = search(r.batch, unit, [&](int i) { return steps_before(r, i); });
  *out = store_rows(r, b);
  out->base += (unit - steps_before(r, b)) * 64;
  return out->base >= out->p0 - 63 && out->base < out->p0 + out->rows;
}

// ---------------------------------------------------------------- attention

// Arguments of the attention kernels.
struct AttentionArgs {
  CacheView c;
  RowsView r;
  const void* q;
  int64_t q_row_stride, q_head_stride;
  int bf16;                 // q and out: 1 bfloat16, 0 binary16
  int q_wide;               // every 8 channels of q lie 16-byte aligned and head_dim is a multiple of 8
  int ratio;                // query heads per key/value head
  float scale_part;         // scale * log2 e = scale_part * 2^scale_exp, the part in [0.5, 1]
  int scale_exp;
  int causal;
  int64_t window;           // 0: none
  void* out;
  float* lse;               // or nullptr
};

hipError_t launch_cache_write(const CacheView& c, const RowsView& r, const void* k, int64_t k_row_stride,
                              int64_t k_head_stride, const void* v, int64_t v_row_stride,
                              int64_t v_head_stride, int dtype, hipStream_t stream);
hipError_t launch_cache_read(const CacheView& c, const RowsView& r, void* k, void* v, int dtype,
                             hipStream_t stream);
hipError_t launch_cache_attention(const AttentionArgs& a, void* workspace, int64_t workspace_bytes,
                                  hipStream_t stream);
// Reads sizes of the views only, and whether starts is nullptr.
int64_t cache_attention_workspace(const CacheView& c, const RowsView& r, int ratio);

}  // namespace int4dq
