// cache_step.h -- kernel arguments and launchers of a serving step's operators
// over the 4-bit cache (include/int4dq_cache_step.h).
#pragma once

#include "cache.h"

namespace int4dq {

// ---------------------------------------------------------------- pages

struct PagesArgs {
  int32_t* table;            // [batch, max_pages]
  int64_t table_stride, max_pages;
  int batch;
  int page_shift;            // log2 of the tokens on a page
  const int32_t* lengths;
  int32_t* free;             // [pages]
  int64_t pages;
  const int32_t* count;      // [2], of which the first is read
  int32_t* new_lengths;      // may be lengths
  int32_t* new_count;        // may be count

  // Table entries that a sequence of `length` tokens takes: as many as it has pages for.
  __host__ __device__ int64_t entries(int64_t length) const {
    const int64_t n = length > 0 ? (length + ((int64_t)1 << page_shift) - 1) >> page_shift : 0;
    return n < max_pages ? n : max_pages;
  }
  // Free pages, of which count may say anything.
  __host__ __device__ int64_t free_pages(int32_t said) const {
    return said < 0 ? 0 : said < pages ? said : pages;
  }
};

// Slot of position pos, given the entry of its page: -1 where there is none.
__host__ __device__ inline int64_t slot_of(int64_t pos, int page_shift, int64_t page, int64_t pages) {
  return page >= 0 && page < pages ? (page << page_shift) + (pos & (((int64_t)1 << page_shift) - 1)) : -1;
}

hipError_t launch_cache_release(const PagesArgs& a, const uint8_t* done, const int32_t* shared, hipStream_t stream);
// starts: [batch + 1]; slots: [rows] or nullptr; added: [batch] or nullptr (one token each).
hipError_t launch_cache_extend(const PagesArgs& a, const int32_t* added, int32_t* starts, int64_t* slots, int64_t rows,
                               hipStream_t stream);

// ---------------------------------------------------------------- norms, rotation, write

struct AppendArgs {
  CacheView c;
  RowsView r;
  const void *q, *k, *v;
  int64_t q_row_stride, q_head_stride, k_row_stride, k_head_stride, v_row_stride, v_head_stride;
  void* out;                 // dense [rows, q_heads, head_dim]
  int q_heads;
  const float *q_norm, *k_norm;          // [head_dim] or nullptr
  double eps;
  const float* rope;         // cosines, then sines, of each position; or nullptr
  int64_t rope_stride, positions;
  int half;                  // half of the rotated channels
  int interleaved;
};

hipError_t launch_cache_append(const AppendArgs& a, int dtype, hipStream_t stream);

// ---------------------------------------------------------------- attention over shared tokens

// Attention of a batch whose sequences begin with the same a.shared tokens, computed
// once from `from` of them on (below 0: where that pays); each sequence for itself below,
// and where the workspace is too small.
hipError_t launch_cache_attention_shared(const AttentionArgs& a, int64_t from, void* workspace, int64_t workspace_bytes,
                                         hipStream_t stream);
// 0: a call of these sizes does not share.
int64_t cache_attention_shared_workspace(const CacheView& c, const RowsView& r, int ratio, int64_t from);

}  // namespace int4dq
