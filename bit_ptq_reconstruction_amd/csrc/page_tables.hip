// page_tables.hip -- pages, places and slots of the tokens that join each sequence.
//
//   need_b = ceil((len_b + n_b) / P) - ceil(len_b / P),   pages free[count - 1 - sum of needs before - j],  j < need_b
//
// A few dozen bytes a sequence and 16 a token, so the time is that of the launch and of the chain lengths -> sums -> pages:
// a sum over the sequences gives the rows, a second one (of those that fit) the pages, and each row finds its sequence by
// bisection of the first sum in LDS.
//
// Few rows: one block does everything.  Many: blocks take slices of the rows and each works the sums out by itself (8 bytes a
// sequence).  The first one also writes the sequences' state; where that lies in the inputs' place (lengths, count), which the
// other blocks read, a second launch of one block does.
//
// 24 sequences of one new token take 4.3 us, of which a launch is 2.5; 300 with prompts of up to 1374 tokens (176433 rows of 16
// bytes) 6.9, in place 11.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qv_runs_internal.h"

namespace qv {

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int64_t kRefused = INT64_MIN;  // in the place of a sequence's pages

struct Args {
  const int32_t *runs, *lens, *free_pages, *free_count;
  int32_t *table, *starts, *lens_out, *free_left, *seq, *index, *status;
  int64_t* slots;
  int64_t num_free, ld_table;
  uint32_t B, T, page_size, capacity;
  uint32_t slice;   // rows of a block
  int32_t rows, state;  // whether this launch writes the rows, and its first block the sequences' state
};

// Sums of numbers >= 0 that stay at the largest one.
__device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) {
  const uint32_t s = a + b;
  return s < a ? 0xFFFFFFFFu : s;
}

// Sum over the threads before this one of the block, and of all of them; `totals` is for this call alone until the next barrier
// but one.
__device__ __forceinline__ uint32_t sum_before(uint32_t x, uint32_t (&totals)[kWaves], uint32_t* all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t upto = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t y = (uint32_t)__shfl_up((int)upto, d);
    if (lane >= d) upto = add(upto, y);
  }
  if (lane == 63) totals[wave] = upto;
  const uint32_t in_wave = (uint32_t)__shfl_up((int)upto, 1);
  __syncthreads();
  uint32_t before = lane ? in_wave : 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const uint32_t t = totals[w];
    if (w < wave) before = add(before, t);
    sum = add(sum, t);
  }
  *all = sum;
  return before;
}

__device__ __forceinline__ int32_t cut(uint32_t x) { return x > 0x7FFFFFFFu ? 0x7FFFFFFF : (int32_t)x; }

__global__ __launch_bounds__(kThreads) void tables_kernel(Args a) {
  __shared__ uint32_t row_totals[kWaves], page_totals[kWaves];
  __shared__ uint32_t starts[kThreads + 1];  // of this chunk's sequences
  __shared__ uint32_t len[kThreads];         // before
  __shared__ int64_t from[kThreads];         // page e >= ceil(len / P) of the sequence is free_pages[from - e]
  const uint32_t P = a.page_size;
  const int32_t counted = *a.free_count;
  const int64_t count = counted < 0 ? 0 : (counted > a.num_free ? a.num_free : counted);
  const uint32_t first_row = blockIdx.x * a.slice, last_row = first_row + a.slice < a.T ? first_row + a.slice : a.T;
  uint32_t rows = 0, asked = 0;  // of the chunks before
  __shared__ uint32_t granted;
  if (threadIdx.x == 0) granted = 0;
  const bool state = a.state && blockIdx.x == 0;

  for (uint32_t chunk = 0; chunk == 0 || chunk < a.B; chunk += kThreads) {
    const uint32_t b = chunk + threadIdx.x;
    const bool live = b < a.B;
    const int32_t n_ = live ? a.runs[b] : 0, len_ = live ? a.lens[b] : 0;
    const uint32_t n = n_ < 0 ? 0 : n_, l = len_ < 0 ? 0 : len_;
    uint32_t all_rows, all_pages;
    const uint32_t at = add(rows, sum_before(n, row_totals, &all_rows)), end = add(at, n);
    const uint32_t held = (l + P - 1) / P;
    uint32_t need = (l + n) / P + ((l + n) % P ? 1 : 0);
    need = need > held ? need - held : 0;
    int why = n > a.capacity || l > a.capacity - n ? QV_RUN_NO_ROOM : (n && end > a.T ? QV_RUN_NO_ROWS : QV_RUN_OK);
    if (why) need = 0;
    const uint32_t before = add(asked, sum_before(need, page_totals, &all_pages));
    if (need && (int64_t)before + need > count) why = QV_RUN_NO_PAGES;
    starts[threadIdx.x] = at;
    if (threadIdx.x == kThreads - 1) starts[kThreads] = end;
    len[threadIdx.x] = l;
    from[threadIdx.x] = why ? kRefused : count - 1 - before + held;
    if (state && live) {
      a.starts[b] = cut(at);
      if (b == a.B - 1) a.starts[a.B] = cut(end);
      a.lens_out[b] = (int32_t)(why ? l : l + n);
      a.status[b] = why;
      if (!why && need) atomicAdd(&granted, need);
    }
    __syncthreads();
    if (a.rows) {
      // The rows of this chunk's sequences that lie in the block's slice, and with the last chunk those behind all of them.
      const bool last = a.B - chunk <= kThreads;
      const uint32_t to = last ? last_row : (starts[kThreads] < last_row ? starts[kThreads] : last_row);
      for (uint32_t t = (starts[0] > first_row ? starts[0] : first_row) + threadIdx.x; t < to; t += kThreads) {
        int32_t seq = -1, index = -1;
        int64_t slot = -1;
        if (t < starts[kThreads]) {
          uint32_t low = 0, high = kThreads;  // starts[low] <= t < starts[high]
#pragma unroll
          for (int i = 0; i < 10; ++i) {
            const uint32_t mid = (low + high) / 2;
            const bool up = starts[mid] <= t;
            low = up ? mid : low;
            high = up ? high : mid;
          }
          if (from[low] != kRefused) {
            seq = (int32_t)(chunk + low);
            const uint32_t place = len[low] + (t - starts[low]), entry = place / P, in_page = place - entry * P;
            index = (int32_t)place;
            int32_t* const held_at = a.table + (int64_t)seq * a.ld_table + entry;
            const bool fresh = entry >= (len[low] + P - 1) / P;
            const int32_t page = fresh ? a.free_pages[from[low] - entry] : *held_at;
            if (fresh && in_page == 0) *held_at = page;
            slot = page < 0 ? -1 : (int64_t)page * P + in_page;
          }
        }
        a.seq[t] = seq;
        a.index[t] = index;
        a.slots[t] = slot;
      }
      __syncthreads();
    }
    rows = add(rows, all_rows);
    asked = add(asked, all_pages);
  }
  if (state) {
    __syncthreads();
    if (threadIdx.x == 0) {
      *a.free_left = (int32_t)(count - granted);
      if (a.B == 0) a.starts[0] = 0;
    }
  }
}

}  // namespace

hipError_t launch_page_tables(const TablesArgs& in, hipStream_t st) {
  Args a = {};
  a.runs = in.runs;
  a.lens = in.lens;
  a.free_pages = in.free_pages;
  a.free_count = in.free_count;
  a.table = in.page_table;
  a.starts = in.starts;
  a.lens_out = in.lens_out;
  a.free_left = in.free_left;
  a.seq = in.token_seq;
  a.index = in.token_index;
  a.status = in.status;
  a.slots = in.slots;
  a.num_free = in.num_free;
  a.ld_table = in.ld_table;
  a.B = (uint32_t)in.B;
  a.T = (uint32_t)in.T;
  a.page_size = (uint32_t)in.page_size;
  a.capacity = (uint32_t)(in.max_pages * in.page_size);
  a.slice = a.T;
  a.rows = a.state = 1;
  if (in.T > 2 * kThreads) {
    const uint32_t blocks = in.T > 1024 * kThreads ? 1024 : (uint32_t)((in.T + kThreads - 1) / kThreads);
    a.slice = (uint32_t)((in.T + blocks - 1) / blocks);
    a.state = in.lens_out != in.lens && in.free_left != in.free_count;
    tables_kernel<<<blocks, kThreads, 0, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.state) return e;
    a.rows = 0;
    a.state = 1;
  }
  tables_kernel<<<1, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace qv
