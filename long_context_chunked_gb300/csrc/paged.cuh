// The paged KV cache: writing new tokens into pages (as bf16, or quantised to
// e4m3) and reading pages back into the striped cache of the chunked prefill.
// The attention over the pages is in paged_decode.cuh.
//
// A page holds page_size consecutive tokens of one sequence for every kv
// head: pages[page][kv head][slot][HD], so the rows of one (page, kv head)
// are contiguous.  Token t of sequence b sits in page table[b][t / page_size]
// at slot t mod page_size.  Lengths and the table are read on the device, so
// a captured step can be replayed after they changed; the kernels therefore
// check every page id and length themselves: what lies outside is skipped and
// reported through the status word (kStatusPage).
//
// e4m3 pages carry one fp32 scale per (token, kv head) and for K and V each:
//   s = max(amax, 2^-110) / 448,  x8 = e4m3(x * (448 / amax)),  x ~ s * x8,
// so that a token can be appended without touching the page's earlier ones.
// The scale is one factor of a whole row: the attention multiplies it into a
// logit (K) or a probability (V), never into the row's HD values.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <type_traits>

#include "ptx.cuh"
#include "walk.cuh"

namespace cpattn {

// Every load of the paged kernels from memory that a kernel ahead of them on the
// stream may write (pages, tables, lengths, rows): an ordinary one.  They are
// programmatic dependents, which may start while that kernel still writes, and
// the non-coherent __ldg is for what nobody writes while the grid runs.
template <class T>
__device__ __forceinline__ T load_now(const T* p) {
  return *p;
}

struct PagedPool {
  void* k;           // bf16 or e4m3 [num_pages][NKV][page_size][HD]
  void* v;
  float* k_scales;   // e4m3: [num_pages][NKV][page_size]
  float* v_scales;
  const int* table;  // [num_seqs][table_stride], the first max_pages columns used
  long long table_stride;
  int num_pages, max_pages, page_shift, nkv;
};

// Page holding tokens [idx * page_size, ...) of sequence b, or -1 (reported).
__device__ __forceinline__ int page_id(const PagedPool& c, int b, int idx, int* status) {
  int id = -1;
  if (idx < c.max_pages) {
    id = load_now(c.table + b * c.table_stride + idx);
    if (id >= c.num_pages) id = -1;
  }
  if (id < 0) {
    id = -1;
    if (status != nullptr) atomicCAS(status, kStatusOk, kStatusPage);
  }
  return id;
}

// Row of (page, kv head, slot) in the pool's [num_pages * NKV * page_size, HD].
__device__ __forceinline__ long long pool_row(const PagedPool& c, int page, int g, int slot) {
  return ((static_cast<long long>(page) * c.nkv + g) << c.page_shift) + slot;
}

// ----------------------------------------------------------- conversions
constexpr float kE4m3Max = 448.f;
constexpr float kTinyAmax = 7.703719777548943e-34f;  // 2^-110: keeps 448 / amax finite

// Two fp32 values as e4m3 (round to nearest even, saturating), lo in the low byte.
__device__ __forceinline__ uint16_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 values as fp16 (exact), the low byte in the lower half.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return r;
}

// Largest magnitude of eight bf16 values, as bf16 bits: for sign-less bf16
// the order of the bit patterns is the order of the values, with infinities
// and NaNs on top.
__device__ __forceinline__ uint32_t amax_bits(uint4 x) {
  const uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                              __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
  return max(m & 0xFFFFu, m >> 16);
}

// ------------------------------------------------------------------ write
struct PagedWriteParams {
  PagedPool pool;
  const uint4* k_new;     // bf16 [rows][NKV][HD]
  const uint4* v_new;
  const int* cache_lens;  // [num_seqs]; < 0: the sequence is skipped
  const int* row_starts;  // [num_seqs + 1], or null: row b belongs to sequence b
  int* status;
  int num_seqs, rows;
  int heads_per_item;     // kv heads one warp takes of its rows
};

// The last sequence that starts at or before row `row`, 0 if none does.  Whole
// warp, one coalesced load per factor of 32 in the number of sequences.
__device__ __forceinline__ int write_seq(const PagedWriteParams& p, int row, int lane) {
  int lo = 0, n = p.num_seqs;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lane * step;
    const uint32_t m =
        __ballot_sync(0xFFFFFFFFu, at < n && load_now(p.row_starts + lo + min(at, n - 1)) <= row);
    const int k = m == 0u ? 0 : 31 - __clz(static_cast<int>(m));
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// Place of row `row` of the call in the pool: (page << 8) | slot, or -1: nobody's
// (before the first sequence or behind the last one), a skipped sequence's, or
// no page for it.  b: a sequence that starts at or before the row's own.
__device__ __forceinline__ long long write_place(const PagedWriteParams& p, int row, int b) {
  if (row >= p.rows) return -1;
  int i = 0;
  if (p.row_starts != nullptr) {
    int begin = load_now(p.row_starts + b), end = load_now(p.row_starts + b + 1);
    while (row >= end && b + 1 < p.num_seqs) {
      ++b;
      begin = end;
      end = load_now(p.row_starts + b + 1);
    }
    if (row < begin || row >= end) return -1;
    i = row - begin;
  }
  const int have = load_now(p.cache_lens + b);
  if (have < 0) return -1;
  const long long t = static_cast<long long>(have) + i;
  const int page =
      page_id(p.pool, b, static_cast<int>(min(t >> p.pool.page_shift, 0x7FFFFFFFLL)), p.status);
  return page < 0 ? -1 : (static_cast<long long>(page) << 8) | (t & ((1 << p.pool.page_shift) - 1));
}

// One warp per (ROWS rows, group of kv heads).  A row's 16-byte vectors: at
// HD = 128 the lower half-warp holds K and the upper one V, at HD = 256 the
// whole warp holds K, then V.  HBM-bound copy: 2 bytes read and 1 (e4m3) or 2
// written per value.  What bounds it is how much of it is in flight, so a warp
// loads the rows of its first head before it looks for their places (some
// dependent loads, lane r for row r), and every head's ROWS rows together.
// ROWS = 1 spreads few rows over more warps.
//   64961 prompt tokens of 2 heads of 256 to bf16 pages: 41.8 us for 266 MB,
// 6.4 TB/s.  To e4m3 pages a head's rows are quantised before the next head's are
// loaded: 17421 tokens of 4 heads of 128 take 14.0 us for 54 MB, 3.9 TB/s, and
// 40000 tokens of 2 heads of 256 37.7 us for 124 MB, 3.3 TB/s (108 registers, so
// two blocks per SM).  A decode step of 7 tokens: 2.3 us as a node of a graph.
template <int HD, bool Q8, int ROWS>
__global__ void __launch_bounds__(256)
    paged_write_kernel(const __grid_constant__ PagedWriteParams p) {
  constexpr int VECS = HD / 8;        // 16-byte vectors per row
  constexpr int LOADS = HD / 128;     // loads of a row: K and V together, or one after the other
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int nkv = p.pool.nkv;
  const int groups = (nkv + p.heads_per_item - 1) / p.heads_per_item;
  const long long items = static_cast<long long>((p.rows + ROWS - 1) / ROWS) * groups;
  const long long warps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
  const bool k_lane = lane < 16;
  const int vec = LOADS == 1 ? lane & 15 : lane;
  for (long long it = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
       it < items; it += warps) {
    const int row0 = static_cast<int>(it / groups) * ROWS;
    const int g0 = static_cast<int>(it % groups) * p.heads_per_item;
    const int g1 = min(nkv, g0 + p.heads_per_item);
    uint4 x[ROWS][LOADS];
    auto load = [&](int g) {
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
          const int row = min(row0 + r, p.rows - 1);
          const bool is_k = LOADS == 1 ? k_lane : l == 0;
          x[r][l] = load_now((is_k ? p.k_new : p.v_new) +
                             (static_cast<long long>(row) * nkv + g) * VECS + vec);
        }
    };
    load(g0);
    const int seq = p.row_starts != nullptr ? write_seq(p, row0, lane) : 0;
    const int row = row0 + lane;
    const long long mine =
        lane < ROWS ? write_place(p, row, p.row_starts != nullptr ? seq : row) : -1;
    long long place[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) place[r] = __shfl_sync(0xFFFFFFFFu, mine, r);
    for (int g = g0; g < g1; ++g) {
      if (g > g0) load(g);
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
          const bool is_k = LOADS == 1 ? k_lane : l == 0;
          const long long dst = pool_row(p.pool, static_cast<int>(place[r] >> 8), g,
                                         static_cast<int>(place[r] & 255));
          void* pool = is_k ? p.pool.k : p.pool.v;
          if constexpr (Q8) {
            uint32_t m = amax_bits(x[r][l]);
#pragma unroll
            for (int o = VECS / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            // A row with an infinity or a NaN has no scale: all of it reads back as NaN.
            float amax = __uint_as_float(m << 16);
            amax = m >= 0x7F80u ? __uint_as_float(0x7FC00000u) : fmaxf(amax, kTinyAmax);
            const float inv = kE4m3Max / amax;
            const uint32_t w[4] = {x[r][l].x, x[r][l].y, x[r][l].z, x[r][l].w};
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              h[j] = pack_e4m3x2(__uint_as_float(w[j] << 16) * inv,
                                 __uint_as_float(w[j] & 0xFFFF0000u) * inv);
            if (place[r] >= 0) {
              reinterpret_cast<uint2*>(pool)[dst * VECS + vec] =
                  make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
              if (vec == 0) (is_k ? p.pool.k_scales : p.pool.v_scales)[dst] = amax / kE4m3Max;
            }
          } else {
            if (place[r] >= 0) reinterpret_cast<uint4*>(pool)[dst * VECS + vec] = x[r][l];
          }
        }
      }
    }
  }
}

// ------------------------------------------------------------------- read
struct PagedReadParams {
  PagedPool pool;
  const int* first;  // [num_seqs] first token read, or null: 0
  const int* lens;   // [num_seqs] tokens [first, lens) are read; lens <= first: none
  uint4* k_cache;    // bf16 [num_seqs][NKV][P][S][HD]
  uint4* v_cache;    // bf16 or fp16
  int* status;
  int num_seqs, P, S, v_f16;
  int heads_per_item;
};

// Exclusive prefix sums of count(b), b < n, into prefix[0..n] (shared memory),
// by the whole block of 256 threads.
template <class Count>
__device__ __forceinline__ void block_prefix(int n, int* prefix, Count count) {
  __shared__ int warp_sum[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (n + 255) / 256;
  const int b0 = min(n, tid * per), b1 = min(n, b0 + per);
  int sum = 0;
  for (int b = b0; b < b1; ++b) sum += count(b);
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < warp; ++w) base += warp_sum[w];
  int at = base + inc - sum;
  for (int b = b0; b < b1; ++b) {
    prefix[b] = at;
    at += count(b);
  }
  if (b1 == n && (b0 < n || tid == 0)) prefix[n] = at;
  __syncthreads();
}

// Eight values of a pool row, e4m3 or bf16, and the same in the cache's type
// (f16: fp16, else bf16).
__device__ __forceinline__ void load_vec(uint2& x, const void* pool, long long at) {
  x = load_now(reinterpret_cast<const uint2*>(pool) + at);
}
__device__ __forceinline__ void load_vec(uint4& x, const void* pool, long long at) {
  x = load_now(reinterpret_cast<const uint4*>(pool) + at);
}
__device__ __forceinline__ uint4 widen_vec(uint2 x, float s, bool f16, bool* overflow) {
  const uint32_t w[2] = {x.x, x.y};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t h = e4m3x2_to_f16x2(static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1))));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    if (f16) {
      o[j] = pack_f16x2(f.x * s, f.y * s);
      if ((o[j] & 0x7C00u) == 0x7C00u || (o[j] & 0x7C000000u) == 0x7C000000u) *overflow = true;
    } else {
      o[j] = pack_bf16x2(f.x * s, f.y * s);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ uint4 widen_vec(uint4 x, float, bool f16, bool* overflow) {
  return f16 ? bf16x8_to_f16x8(x, overflow) : x;
}

// One warp per (RUN consecutive tokens, group of kv heads), lanes as in the
// write; a run starts at a multiple of RUN, so it lies in one page and one
// look-up serves it.  HBM-bound copy; the loads of a run's rows go out together
// (one row at a time: 80 us where four took 60.5, the first case below).
//   86970 tokens of 4 heads of 128 from bf16 pages: 58.9 us for 356 MB,
// 6.0 TB/s.  28672 tokens of 2 heads of 256 from e4m3 pages of 16: 18.9 us for
// 89 MB, 4.7 TB/s, the launch and the prefix sums of every block among them.
constexpr int kReadRun = 4;

template <int HD, bool Q8>
__global__ void __launch_bounds__(256)
    paged_read_kernel(const __grid_constant__ PagedReadParams p) {
  constexpr int VECS = HD / 8;
  constexpr int LOADS = HD / 128;
  constexpr int RUN = kReadRun;
  extern __shared__ int prefix[];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int nkv = p.pool.nkv;
  // Tokens that both the striped cache and the table's row can hold.
  const long long room = min(static_cast<long long>(p.P) * p.S,
                             static_cast<long long>(p.pool.max_pages) << p.pool.page_shift);
  auto start = [&](int b) { return p.first != nullptr ? max(load_now(p.first + b), 0) : 0; };
  auto stop = [&](int b) {
    return static_cast<int>(min(static_cast<long long>(load_now(p.lens + b)), room));
  };
  block_prefix(p.num_seqs, prefix, [&](int b) {  // runs of each sequence
    if (p.lens[b] > room && p.status != nullptr) atomicCAS(p.status, kStatusOk, kStatusPage);
    const int s = start(b), e = stop(b);
    return e > s ? (e + RUN - 1) / RUN - s / RUN : 0;
  });
  const int total = prefix[p.num_seqs];
  const int groups = (nkv + p.heads_per_item - 1) / p.heads_per_item;
  const long long items = static_cast<long long>(total) * groups;
  const long long warps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
  const bool k_lane = lane < 16;
  const int vec = LOADS == 1 ? lane & 15 : lane;
  for (long long it = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
       it < items; it += warps) {
    const int run = static_cast<int>(it / groups);
    const int g0 = static_cast<int>(it % groups) * p.heads_per_item;
    int lo = 0, hi = p.num_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= run) lo = mid; else hi = mid - 1;
    }
    const int t_first = start(lo), t_stop = stop(lo);
    const int t0 = (t_first / RUN + run - prefix[lo]) * RUN;
    const int page = page_id(p.pool, lo, t0 >> p.pool.page_shift, p.status);
    if (page < 0) continue;
    const int slot0 = t0 & ((1 << p.pool.page_shift) - 1);
    // Places of the run's tokens in a (sequence, kv head)'s [P * S] rows; -1: not read.
    long long row[RUN];
#pragma unroll
    for (int r = 0; r < RUN; ++r) {
      const int t = t0 + r;
      row[r] = t >= t_first && t < t_stop ? static_cast<long long>(t % p.P) * p.S + t / p.P : -1;
    }
    const int g1 = min(nkv, g0 + p.heads_per_item);
    for (int g = g0; g < g1; ++g) {
      const long long src = pool_row(p.pool, page, g, slot0);
      const long long dst = (static_cast<long long>(lo) * nkv + g) * p.P * p.S;
      typename std::conditional<Q8, uint2, uint4>::type x[RUN][LOADS];
      float sc[RUN][LOADS];
#pragma unroll
      for (int r = 0; r < RUN; ++r)
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
          const bool is_k = LOADS == 1 ? k_lane : l == 0;
          load_vec(x[r][l], is_k ? p.pool.k : p.pool.v, (src + r) * VECS + vec);
          if (Q8) sc[r][l] = load_now((is_k ? p.pool.k_scales : p.pool.v_scales) + src + r);
        }
#pragma unroll
      for (int r = 0; r < RUN; ++r)
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
          const bool is_k = LOADS == 1 ? k_lane : l == 0;
          if (row[r] < 0) continue;
          bool overflow = false;
          const uint4 y = widen_vec(x[r][l], sc[r][l], !is_k && p.v_f16 != 0, &overflow);
          if (overflow && p.status != nullptr) atomicCAS(p.status, kStatusOk, kStatusRange);
          (is_k ? p.k_cache : p.v_cache)[(dst + row[r]) * VECS + vec] = y;
        }
    }
  }
}

}  // namespace cpattn
