// A step of a batch over the paged cache, made on the GPU from the requests'
// lengths: pages for the new tokens off the free list, the block table's new
// entries, the rows' starts, and every row's position and slot (plan); and the
// pages of tokens that are not kept back to the list (trim).
//
//   old_b = ceil(have_b / ps), need_b = ceil((have_b + new_b) / ps) - old_b,
//   upto_b = need_0 + .. + need_b;   b is served where need_b = 0 or upto_b <= count.
// The list is a stack: page k of the step (k counts the served sequences' new
// pages, in order) is free[count - 1 - k].  Trim puts page k of those that go back,
// counted the same way, to free[count + back - 1 - k], so that a trim back to the
// lengths before a plan undoes it.
//
// Bound by latency: a few dozen bytes per sequence and eight per row, behind a
// chain of lengths, prefix sums, look-up and page id.  So one cluster does it in
// one launch: every CTA makes the prefix sums itself, in shared memory, the CTAs
// deal the rows and the pages among themselves, and a cluster barrier stands
// between everyone's reads of the lengths and the list's count and their update.
// No atomic decides anything: the same call gives the same pages.
//   A step of 64 sequences and 80 rows, plan and trim: 7.2 us as two nodes of a graph;
// five prompts of 64961 rows: 10.4 us (0.5 MB of positions and slots by 8 CTAs).
#pragma once

#include <cstdint>

#include "paged.cuh"
#include "ptx.cuh"

namespace cpattn {

constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxCtas = 8;

struct PagedPlanParams {
  PagedPool pool;         // its table is written
  int* table;
  const int* cache_lens;  // [num_seqs]; < 0: an empty place
  const int* new_lens;    // plan
  const int* keep;        // trim
  int* free_pages;        // [num_pages]
  int* free_count;        // [1]
  int* lens;              // plan: written; trim: read
  int* row_starts;        // [num_seqs + 1]
  int* positions;         // [rows]
  int* slots;
  int* status;
  int num_seqs, rows;
};

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive;" ::: "memory");
}
__device__ __forceinline__ void cluster_await() {
  asm volatile("barrier.cluster.wait;" ::: "memory");
}

// Inclusive sums over the block of two 64-bit values per thread.  `carry`: 64
// values of shared memory, free to be reused after the next barrier.
__device__ __forceinline__ void block_sums(long long& a, long long& b, long long* carry) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xFFFFFFFFu, a, o), y = __shfl_up_sync(0xFFFFFFFFu, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    carry[warp] = a;
    carry[32 + warp] = b;
  }
  __syncthreads();
  long long x = lane < kPlanThreads / 32 ? carry[lane] : 0;
  long long y = lane < kPlanThreads / 32 ? carry[32 + lane] : 0;
  x = lane < warp ? x : 0;
  y = lane < warp ? y : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    y += __shfl_xor_sync(0xFFFFFFFFu, y, o);
  }
  a += x;
  b += y;
}

// The b < n whose slice [ends[b - 1], ends[b]) holds i (ends[n - 1] > i).
__device__ __forceinline__ int slice_of(const int* ends, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > i) hi = mid; else lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ long long pages_of(const PagedPool& c, long long tokens) {
  return (tokens + (1 << c.page_shift) - 1) >> c.page_shift;
}

__device__ __forceinline__ int clip(long long x) { return static_cast<int>(min(x, 0x7FFFFFFFLL)); }

__device__ __forceinline__ int listed_pages(const PagedPlanParams& p) {
  return max(0, min(load_now(p.free_count), p.pool.num_pages));
}

// Shared memory: for each sequence the end of its rows, the end of its new pages
// and the tokens it has (its sign bit: not served).
__global__ void __launch_bounds__(kPlanThreads)
    paged_plan_kernel(const __grid_constant__ PagedPlanParams p) {
  extern __shared__ int sm[];
  __shared__ long long carry[64];
  __shared__ int sh_taken;
  int* row_end = sm;
  int* page_end = row_end + p.num_seqs;
  int* held = page_end + p.num_seqs;
  const int tid = threadIdx.x, ctas = gridDim.x;
  griddep_launch_dependents();
  griddep_wait();
  const PagedPool& c = p.pool;
  const int count = listed_pages(p);
  const int per = (p.num_seqs + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(p.num_seqs, tid * per), b1 = min(p.num_seqs, b0 + per);
  bool trouble = load_now(p.free_count) != count;
  struct Seq {
    long long rows, need;
    int have;
    bool here;
  };
  // (rows first: the prefix sums of the rows do not depend on what is served.)
  auto seq = [&](int b) {
    Seq s;
    s.have = load_now(p.cache_lens + b);
    s.rows = s.have < 0 ? 0 : max(load_now(p.new_lens + b), 0);
    const long long total = pages_of(c, static_cast<long long>(s.have) + s.rows);
    s.here = s.have >= 0 && total <= c.max_pages;
    s.need = s.here ? total - pages_of(c, s.have) : 0;
    return s;
  };
  long long rows = 0, need = 0;
  for (int b = b0; b < b1; ++b) {
    const Seq s = seq(b);
    rows += s.rows;
    need += s.need;
  }
  const long long rows_own = rows, need_own = need;
  if (tid == 0) sh_taken = 0;
  block_sums(rows, need, carry);
  rows -= rows_own;
  need -= need_own;
  int taken = 0;
  for (int b = b0; b < b1; ++b) {
    const Seq s = seq(b);
    rows += s.rows;
    need += s.need;
    // A sequence whose rows pass the call's is not served either.
    const bool in = s.here && (s.need == 0 || need <= count) && (s.rows == 0 || rows <= p.rows);
    if (in && s.need > 0) taken = static_cast<int>(need);
    trouble |= s.have >= 0 && !in;
    row_end[b] = clip(rows);
    page_end[b] = clip(need);
    held[b] = in ? s.have : (s.have | static_cast<int>(0x80000000u));
  }
  if (taken > 0) atomicMax(&sh_taken, taken);
  cluster_arrive();  // this CTA has read the lengths and the count
  __syncthreads();
  taken = sh_taken;
  if (trouble && blockIdx.x == 0 && p.status != nullptr) atomicCAS(p.status, kStatusOk, kStatusPage);
  const int first = blockIdx.x * kPlanThreads + tid, step = ctas * kPlanThreads;
  const int total = p.num_seqs > 0 ? row_end[p.num_seqs - 1] : 0;
  // Rows before the table's new entries: nobody reads one of those.
  for (int r = first; r < p.rows; r += step) {
    int pos = -1, slot = -1;
    if (r < total) {
      const int b = slice_of(row_end, p.num_seqs, r);
      const int have = held[b];
      if (have >= 0) {
        pos = have + r - (b > 0 ? row_end[b - 1] : 0);
        const int col = pos >> c.page_shift, old = static_cast<int>(pages_of(c, have));
        const int page = load_now(col < old ? p.table + b * c.table_stride + col
                                            : p.free_pages + count - 1 -
                                                  ((b > 0 ? page_end[b - 1] : 0) + col - old));
        if (static_cast<unsigned>(page) < static_cast<unsigned>(c.num_pages))
          slot = (page << c.page_shift) | (pos & ((1 << c.page_shift) - 1));
        else if (p.status != nullptr)
          atomicCAS(p.status, kStatusOk, kStatusPage);
      }
    }
    p.positions[r] = pos;
    p.slots[r] = slot;
  }
  for (int k = first; k < taken; k += step) {
    const int b = slice_of(page_end, p.num_seqs, k);
    const int col = static_cast<int>(pages_of(c, held[b])) + k - (b > 0 ? page_end[b - 1] : 0);
    p.table[b * c.table_stride + col] = load_now(p.free_pages + count - 1 - k);
  }
  cluster_await();
  if (blockIdx.x != 0) return;
  for (int b = tid; b < p.num_seqs; b += kPlanThreads) {
    const int have = held[b], n = row_end[b] - (b > 0 ? row_end[b - 1] : 0);
    const int own = load_now(p.cache_lens + b);  // (lens may be the same array)
    p.lens[b] = have >= 0 ? have + n : own;
    p.row_starts[b + 1] = row_end[b];
  }
  if (tid == 0) {
    p.row_starts[0] = 0;
    *p.free_count = count - taken;
  }
}

__global__ void __launch_bounds__(kPlanThreads)
    paged_trim_kernel(const __grid_constant__ PagedPlanParams p) {
  extern __shared__ int sm[];
  __shared__ long long carry[64];
  int* page_end = sm;
  int* kept = page_end + p.num_seqs;
  const int tid = threadIdx.x, ctas = gridDim.x;
  griddep_launch_dependents();
  griddep_wait();
  const PagedPool& c = p.pool;
  const int count = listed_pages(p);
  const int per = (p.num_seqs + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(p.num_seqs, tid * per), b1 = min(p.num_seqs, b0 + per);
  bool trouble = load_now(p.free_count) != count;
  auto back_of = [&](int b, int* first) {
    const int n = load_now(p.lens + b), keep = load_now(p.keep + b);
    *first = 0;
    if (keep < 0 || keep >= n) return 0LL;
    const long long all = pages_of(c, n), left = pages_of(c, keep);
    *first = static_cast<int>(left);
    if (all > c.max_pages) trouble = true;
    return max(0LL, min(all, static_cast<long long>(c.max_pages)) - left);
  };
  long long back = 0, none = 0;
  int f;
  for (int b = b0; b < b1; ++b) back += back_of(b, &f);
  const long long own = back;
  block_sums(back, none, carry);
  back -= own;
  for (int b = b0; b < b1; ++b) {
    back += back_of(b, &f);
    page_end[b] = clip(back);
    kept[b] = f;
  }
  cluster_arrive();
  __syncthreads();
  int total = p.num_seqs > 0 ? page_end[p.num_seqs - 1] : 0;
  // More pages than the pool has: some of them twice.  None goes back then.
  if (static_cast<long long>(count) + total > c.num_pages) {
    trouble = true;
    total = 0;
  }
  if (trouble && blockIdx.x == 0 && p.status != nullptr) atomicCAS(p.status, kStatusOk, kStatusPage);
  const int first = blockIdx.x * kPlanThreads + tid, step = ctas * kPlanThreads;
  for (int k = first; k < total; k += step) {
    const int b = slice_of(page_end, p.num_seqs, k);
    const int col = kept[b] + k - (b > 0 ? page_end[b - 1] : 0);
    const int page = load_now(p.table + b * c.table_stride + col);
    p.free_pages[count + total - 1 - k] = page;
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(c.num_pages) && p.status != nullptr)
      atomicCAS(p.status, kStatusOk, kStatusPage);
  }
  cluster_await();
  if (blockIdx.x == 0 && tid == 0) *p.free_count = count + total;
}

}  // namespace cpattn
