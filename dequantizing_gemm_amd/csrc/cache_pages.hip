// cache_pages.hip -- the page table of a serving batch, kept on the GPU: pages for
// new tokens and the slots of the new rows, pages of ended sequences back to the
// free ones (include/int4dq_cache_step.h).
//
// Mathematics: exclusive sums over the batch of new tokens (starts) and of the
// pages they need; the i-th page of sequence b is the free page
// count - 1 - (pages needed before b) - i, whatever else runs.
//
// Work. One block of 1024 threads, a thread a sequence for the sums and then a thread a
// page: the sums need each other, and a step's work is small. Bound by latency: 128
// sequences of one new token 5.2 us, 9 ended ones' 282 pages given back 3.9 us, 72447 new
// tokens of 46 sequences, 4534 pages, 7.7 us and their slots, on the whole GPU, 3.6 us;
// 8000 sequences of one new token 25 us.
#include "cache_step.h"
#include "lanes.h"

namespace int4dq {

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / kWave;

// Inclusive sum over the wavefront's lanes of 0 <= v < 2^42: two sums of 32 bits.
__device__ __forceinline__ int64_t lane_scan_wide(int64_t v) {
  const uint32_t low = lane_scan((uint32_t)v & 0xFFFFu), high = lane_scan((uint32_t)(v >> 16));
  return ((int64_t)high << 16) + low;
}

// Sums over the block's threads of 0 <= v <= 2^31.
struct BlockScan {
  int64_t wave[2][kWaves];               // two buffers: one barrier a scan
};
__device__ __forceinline__ void block_scan(BlockScan& s, int turn, int64_t v, int64_t* before, int64_t* all) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int64_t upto = lane_scan_wide(v);
  if (lane == kWave - 1) s.wave[turn][wave] = upto;
  __syncthreads();
  int64_t sum = 0, mine = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    mine = i == wave ? sum : mine;
    sum += s.wave[turn][i];
  }
  *before = mine + upto - v;
  *all = sum;
}

// The last i in [0, n) with f[i] <= x, where f does not decrease and f[0] <= x.
__device__ __forceinline__ int last_upto(const int64_t* f, int n, int64_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (f[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int32_t clamp32(int64_t v) { return v < INT32_MAX ? (int32_t)v : INT32_MAX; }

// One block: the sequences by 1024, then the entries that these give back by 1024, in order.
__global__ __launch_bounds__(kThreads) void cache_release_kernel(PagesArgs a, const uint8_t* done, const int32_t* shared) {
  __shared__ BlockScan scan;
  __shared__ int64_t first[kThreads];
  __shared__ int kept[2][kWaves];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  int64_t left = a.free_pages(a.count[0]);
  const int64_t skip = shared && *shared > 0 ? *shared >> a.page_shift : 0;
  int turn = 0, half = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kThreads, turn ^= 1) {
    const int b = b0 + tid;
    int64_t mine = 0;
    if (b < a.batch) {
      const int32_t length = a.lengths[b];
      const bool ended = done[b] != 0;
      if (ended) mine = a.entries(length) - skip;
      if (mine < 0) mine = 0;
      a.new_lengths[b] = ended ? 0 : length;
    }
    int64_t before, all;
    block_scan(scan, turn, mine, &before, &all);
    first[tid] = before;
    __syncthreads();
    for (int64_t e0 = 0; e0 < all; e0 += kThreads, half ^= 1) {
      const int64_t e = e0 + tid;
      int64_t page = -1;
      if (e < all) {
        const int s = last_upto(first, kThreads, e);
        page = a.table[(int64_t)(b0 + s) * a.table_stride + skip + (e - first[s])];
      }
      const bool keep = page >= 0 && page < a.pages;
      const uint64_t bits = __ballot(keep);
      if (lane == 0) kept[half][wave] = __builtin_popcountll(bits);
      __syncthreads();
      int64_t at = left;
      int sum = 0;
      for (int i = 0; i < kWaves; ++i) {
        at += i < wave ? kept[half][i] : 0;
        sum += kept[half][i];
      }
      at += __builtin_popcountll(bits & (((uint64_t)1 << lane) - 1));
      if (keep && at < a.pages) a.free[at] = (int32_t)page;
      left = left + sum < a.pages ? left + sum : a.pages;
    }
    __syncthreads();                     // before `first` is written again, and for the count
  }
  if (tid == 0) {
    a.new_count[0] = (int32_t)left;
    a.new_count[1] = 0;
  }
}

// One block: the sequences by 1024; their pages, and (few rows) their rows' slots.
// SLOTS: whether it writes those too.
template <bool SLOTS>
__global__ __launch_bounds__(kThreads) void cache_extend_kernel(PagesArgs a, const int32_t* added, int32_t* starts,
                                                                int64_t* slots, int64_t rows) {
  __shared__ BlockScan scan_rows, scan_pages;
  __shared__ int64_t first_page[kThreads], first_row[kThreads];
  __shared__ int64_t first_pos[kThreads], held_of[kThreads];
  const int tid = threadIdx.x;
  const int64_t left = a.free_pages(a.count[0]);
  int64_t row0 = 0, page0 = 0;           // rows and pages of the sequences before these
  int turn = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kThreads, turn ^= 1) {
    const int b = b0 + tid;
    int64_t length = 0, more = 0;
    if (b < a.batch) {
      length = a.lengths[b];
      more = added ? added[b] : 1;
      if (length < 0) length = 0;
      if (more < 0) more = 0;
    }
    const int64_t total = clamp32(length + more), held = a.entries(length), need = a.entries(total) - held;
    int64_t rows_before, rows_all, before, all;
    block_scan(scan_rows, turn, more, &rows_before, &rows_all);
    block_scan(scan_pages, turn, need, &before, &all);
    if (b < a.batch) {
      a.new_lengths[b] = (int32_t)total;
      starts[b] = clamp32(row0 + rows_before);
    }
    first_page[tid] = before;
    first_row[tid] = rows_before;
    first_pos[tid] = total - more;       // length, but where the sequence ends at 2^31 - 1
    held_of[tid] = held;
    __syncthreads();
    for (int64_t i = tid; i < all; i += kThreads) {
      const int s = last_upto(first_page, kThreads, i);
      const int64_t at = left - 1 - page0 - i;
      a.table[(int64_t)(b0 + s) * a.table_stride + held_of[s] + (i - first_page[s])] = at >= 0 ? a.free[at] : -1;
    }
    __syncthreads();                     // pages before their slots
    if constexpr (SLOTS) {
      const int64_t end = row0 + rows_all < rows ? rows_all : rows - row0;
      for (int64_t i = tid; i < end; i += kThreads) {
        const int s = last_upto(first_row, kThreads, i);
        const int64_t pos = first_pos[s] + (i - first_row[s]), index = pos >> a.page_shift;
        const int64_t page = index < a.max_pages ? a.table[(int64_t)(b0 + s) * a.table_stride + index] : -1;
        slots[row0 + i] = slot_of(pos, a.page_shift, page, a.pages);
      }
    }
    row0 += rows_all;
    page0 += all;
    __syncthreads();                     // before the arrays are written again
  }
  if constexpr (SLOTS)
    for (int64_t t = row0 + tid; t < rows; t += kThreads) slots[t] = -1;
  if (tid == 0) {
    starts[a.batch] = clamp32(row0);
    a.new_count[0] = (int32_t)(left > page0 ? left - page0 : 0);
    a.new_count[1] = clamp32(page0 > left ? page0 - left : 0);
  }
}

// A thread a row; lengths and starts are the new ones. (The new tokens are read themselves only
// where starts do not tell them: their array may be that of the lengths, which are new by now.)
__global__ __launch_bounds__(256) void cache_slots_kernel(PagesArgs a, const int32_t* added, const int32_t* starts,
                                                          int64_t* slots, int64_t rows) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= rows) return;
  int lo = 0, hi = a.batch;              // the last sequence that starts at or before t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= t) lo = mid; else hi = mid;
  }
  int64_t slot = -1;
  if (t < starts[a.batch]) {
    const int64_t more = starts[lo + 1] < INT32_MAX || !added ? starts[lo + 1] - starts[lo] : added[lo];
    const int64_t pos = a.new_lengths[lo] - more + (t - starts[lo]), index = pos >> a.page_shift;
    if (pos >= 0 && index < a.max_pages)
      slot = slot_of(pos, a.page_shift, a.table[(int64_t)lo * a.table_stride + index], a.pages);
  }
  slots[t] = slot;
}

// From more rows than this, their slots are written by a kernel of their own, on the
// whole GPU, instead of by the one block that takes the pages, which takes a microsecond
// for 1024 of them (16 sequences: 1008 rows 6.8 us, 2016 7.8, 2064 8.1, 64512 10.8).
constexpr int64_t kRowsOfOneBlock = 2048;

}  // namespace

hipError_t launch_cache_release(const PagesArgs& a, const uint8_t* done, const int32_t* shared, hipStream_t stream) {
  hipLaunchKernelGGL(cache_release_kernel, dim3(1), dim3(kThreads), 0, stream, a, done, shared);
  return hipGetLastError();
}

hipError_t launch_cache_extend(const PagesArgs& a, const int32_t* added, int32_t* starts, int64_t* slots, int64_t rows,
                               hipStream_t stream) {
  const bool apart = slots && rows > kRowsOfOneBlock;
  if (slots && !apart)
    hipLaunchKernelGGL(cache_extend_kernel<true>, dim3(1), dim3(kThreads), 0, stream, a, added, starts, slots, rows);
  else
    hipLaunchKernelGGL(cache_extend_kernel<false>, dim3(1), dim3(kThreads), 0, stream, a, added, starts, slots, rows);
  if (apart)
    hipLaunchKernelGGL(cache_slots_kernel, dim3((unsigned)((rows + 255) / 256)), dim3(256), 0, stream, a, added, starts,
                       slots, rows);
  return hipGetLastError();
}

}  // namespace int4dq
