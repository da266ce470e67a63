// The paged KV cache: writing new tokens into pages (as bf16, or quantised to
// e4m3 or e2m1) and reading pages back into the striped cache of the chunked
// prefill.
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
//
// e2m1 pages hold 4-bit values (magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6), two to a
// byte, and scales of two levels for each (token, kv head), K and V each:
//   s = 2^(floor(log2 amax) - 9), amax at least 2^-117,
//   r_g = e4m3(amax_g / (6 s)) of each group g of 32 values, at most 176,
//   x4 = e2m1((x / s) / r_g), 0 where r_g = 0,   x ~ s r_g x4.
// s is a power of two so that every one of these roundings is decided exactly in
// fp32 for a bf16 x: x / s is exact, and a quotient of two numbers this short is
// either a border between two codes or further from it than fp32 rounds.  amax / s
// is 512 to 1024 and e4m3's least normal value 2^-6: so r_g has e4m3's precision for
// groups down to 2^-12.4 of the row's largest value (2^-13.4 at best), fewer bits
// below, and is 0 from 2^-16.4 (2^-17.4) on.  A row's scales are one record of
// 4 + HD / 32 bytes, s as fp32 and then the r_g, so that one copy brings them.
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

// Page formats, as CPATTN_PAGES_*.
constexpr int kBf16 = 0, kE4m3 = 1, kE2m1 = 4;

constexpr int kGroup4 = 32;  // values of an e2m1 row that share an r_g
__host__ __device__ constexpr int record_bytes(int hd) { return 4 + hd / kGroup4; }
// Bytes of a row's values.
__host__ __device__ constexpr int row_bytes(int hd, int fmt) {
  return fmt == kBf16 ? 2 * hd : (fmt == kE4m3 ? hd : hd / 2);
}

struct PagedPool {
  void* k;           // bf16, e4m3 or e2m1 [num_pages][NKV][page_size][HD]
  void* v;
  float* k_scales;   // e4m3: [num_pages][NKV][page_size]; e2m1: records, as many
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

// Eight fp32 values as e2m1 (round to nearest even, saturating), the first in the
// lowest bits; and eight values as fp16 pairs (exact).
__device__ __forceinline__ uint32_t pack_e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}
__device__ __forceinline__ void e2m1x8_to_f16x8(uint32_t x, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(x));
}

// Products and sums of pairs of fp32 values, each rounded as by itself.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair_of(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split(f32x2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void mul_pair(float& a, float& b, f32x2 f) {  // (a, b) *= f
  const float2 r = split(mul2(pair_of(a, b), f));
  a = r.x;
  b = r.y;
}
__device__ __forceinline__ void add_pair(float& a, float& b, f32x2 x) {  // (a, b) += x
  const float2 r = split(add2(pair_of(a, b), x));
  a = r.x;
  b = r.y;
}
// (a, b) = (x, y) f + z
__device__ __forceinline__ void fma_pair(float x, float y, f32x2 f, f32x2 z, float& a, float& b) {
  const float2 r = split(fma2(pair_of(x, y), f, z));
  a = r.x;
  b = r.y;
}
__device__ __forceinline__ f32x2 bf16x2_to_f32x2(uint32_t x) {
  return pair_of(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
}

// Largest magnitude of eight bf16 values, as bf16 bits: for sign-less bf16
// the order of the bit patterns is the order of the values, with infinities
// and NaNs on top.
__device__ __forceinline__ uint32_t amax_bits(uint4 x) {
  const uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                              __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
  return max(m & 0xFFFFu, m >> 16);
}

__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// A row of HD values in HD / 8 neighbouring lanes, eight each: what the page
// stores for it.  In two steps, so that several rows' arithmetic can be in
// flight before the first of them is stored.  mag: the bits of the lane's largest
// magnitude.  Rows that hold an infinity or a NaN have a NaN scale and read back
// as NaN.  All lanes of the warp call `quantise`.
template <int FMT>
struct PackedRow;
template <>
struct PackedRow<kBf16> {
  uint4 x;
};
template <>
struct PackedRow<kE4m3> {
  uint2 x;
  float s;
};
template <>
struct PackedRow<kE2m1> {
  uint32_t x;  // the first value in the lowest bits
  float s;
  uint32_t r;  // the r_g of four groups, from this lane's on
};

// (As paged_write_kernel has it for itself, whose 14 us for 17421 rows of 4 heads of 128
// this form made 19; both have to store the same bits.)
template <int HD>
__device__ __forceinline__ void quantise(const float (&x)[8], uint32_t mag, PackedRow<kE4m3>& y) {
#pragma unroll
  for (int o = HD / 16; o > 0; o >>= 1) mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, o));
  const float amax = mag >= 0x7F800000u ? __uint_as_float(0x7FC00000u)
                                        : fmaxf(__uint_as_float(mag), kTinyAmax);
  const float inv = kE4m3Max / amax;
  uint32_t h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) h[j] = pack_e4m3x2(x[2 * j] * inv, x[2 * j + 1] * inv);
  y.x = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  y.s = amax / kE4m3Max;
}

// e2m1.  The quotients amax_g / s / 6 and x / s / r_g are made of products with the
// divisor's reciprocal: by Markstein's theorem (IBM J. Res. Dev. 34, 1990), with f
// the reciprocal of d rounded to nearest and q = a f rounded, the remainder a - q d
// is exact in one fused step, and q + (a - q d) f rounds to a / d correctly.
struct Scales4 {
  float s;            // of the row
  uint32_t r;         // of the lane's group
  f32x2 inv_s, f, d;  // 1 / s, 1 / r_g (0 where r_g is), -r_g
};
// mag: the bits of the group's largest magnitude, row: of the row's.
__device__ __forceinline__ Scales4 scales4(uint32_t mag, uint32_t row) {
  const bool fine = row < 0x7F800000u;
  const uint32_t e = fine ? max(row >> 23, 10u) : 10u;      // exponent field of amax
  const float inv_s = __uint_as_float((263u - e) << 23);    // 2^(9 - k), k = e - 127
  const float a = __uint_as_float(mag) * inv_s, a6 = a * (1.f / 6.f);
  Scales4 y;
  y.r = pack_e4m3x2(fmaf(fmaf(-a6, 6.f, a), 1.f / 6.f, a6), 0.f) & 0xFFu;
  if (!fine) y.r = 0u;
  // 1 / r_g to nearest: one of Newton's steps from the approximation, whose error it
  // squares; r_g has 4 bits, so no quotient is that close to two floats' middle.
  const float rf = f16x2_to_f32x2(e4m3x2_to_f16x2(static_cast<uint16_t>(y.r))).x;
  float f;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(f) : "f"(rf));
  f = fmaf(fmaf(-rf, f, 1.f), f, f);
  if (y.r == 0u) f = 0.f;
  y.s = fine ? __uint_as_float((e - 9u) << 23) : __uint_as_float(0x7FC00000u);
  y.inv_s = pair_of(inv_s, inv_s);
  y.f = pair_of(f, f);
  y.d = pair_of(-rf, -rf);
  return y;
}
__device__ __forceinline__ float2 quotients4(f32x2 x, const Scales4& c) {
  const f32x2 v = mul2(x, c.inv_s), p = mul2(v, c.f);
  return split(fma2(fma2(p, c.d, v), c.f, p));
}

template <int HD>
__device__ __forceinline__ void quantise(const float (&x)[8], uint32_t mag, PackedRow<kE2m1>& y) {
  mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, 1));
  mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, 2));
  uint32_t row = mag;
#pragma unroll
  for (int o = HD / 16; o >= 4; o >>= 1) row = max(row, __shfl_xor_sync(0xFFFFFFFFu, row, o));
  const Scales4 c = scales4(mag, row);
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 z = quotients4(pair_of(x[j], x[j + 1]), c);
    q[j] = z.x;
    q[j + 1] = z.y;
  }
  y.x = c.r != 0u ? pack_e2m1x8(q) : 0u;
  y.s = c.s;
  // The record's words: four r_g each.
  uint32_t r = c.r;
  r |= __shfl_down_sync(0xFFFFFFFFu, r, 4) << 8;
  r |= __shfl_down_sync(0xFFFFFFFFu, r, 8) << 16;
  y.r = r;
}

// To row `dst` of the pool, lane `vec` of the row's HD / 8.
template <int HD>
__device__ __forceinline__ void store_row(const PagedPool& c, bool is_k, long long dst, int vec,
                                          const PackedRow<kBf16>& y) {
  reinterpret_cast<uint4*>(is_k ? c.k : c.v)[dst * (HD / 8) + vec] = y.x;
}
template <int HD>
__device__ __forceinline__ void store_row(const PagedPool& c, bool is_k, long long dst, int vec,
                                          const PackedRow<kE4m3>& y) {
  reinterpret_cast<uint2*>(is_k ? c.k : c.v)[dst * (HD / 8) + vec] = y.x;
  if (vec == 0) (is_k ? c.k_scales : c.v_scales)[dst] = y.s;
}
template <int HD>
__device__ __forceinline__ void store_row(const PagedPool& c, bool is_k, long long dst, int vec,
                                          const PackedRow<kE2m1>& y) {
  reinterpret_cast<uint32_t*>(is_k ? c.k : c.v)[dst * (HD / 8) + vec] = y.x;
  uint32_t* rec =
      reinterpret_cast<uint32_t*>(is_k ? c.k_scales : c.v_scales) + dst * (record_bytes(HD) / 4);
  if (vec == 0) rec[0] = __float_as_uint(y.s);
  if ((vec & 15) == 0) rec[1 + vec / 16] = y.r;
}
__device__ __forceinline__ void bf16x8_to_f32x8(uint4 x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = __uint_as_float(w[j] << 16);
    f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}

// ------------------------------------------------------------------ write
struct PagedWriteParams {
  PagedPool pool;
  const uint4* k_new;     // bf16 [rows][NKV][HD]
  const uint4* v_new;
  const int* cache_lens;  // [num_seqs]; < 0: the sequence is skipped
  const int* row_starts;  // [num_seqs + 1], or null: row b belongs to sequence b
  const int* lens;        // [num_seqs] tokens from here on are left out, or null
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
// (before the first sequence or behind the last one), a skipped sequence's, one
// from its length on, or no page for it.  b: a sequence that starts at or before the row's own.
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
  const int len = p.lens != nullptr ? load_now(p.lens + b) : 0x7FFFFFFF;
  const long long t = static_cast<long long>(have) + i;
  if (have < 0 || (t >= len && p.lens != nullptr)) return -1;
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
// 40000 tokens of 2 heads of 256 37.3 us for 124 MB, 3.3 TB/s (96 registers, so
// two blocks per SM).  A decode step of 7 tokens: 2.3 us as a node of a graph.
template <int HD, int ROWS, int FMT>
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
          if constexpr (FMT == kE4m3) {
            uint32_t m = amax_bits(x[r][l]);
#pragma unroll
            for (int o = VECS / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            // A row with an infinity or a NaN has no scale: all of it reads back as NaN.
            // (The same bits as `quantise` makes.)
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

// The write to e2m1 pages.  The arithmetic of 8 values is 33 instructions, but that
// of their row's and group's scales, their place and their record some 80 for a
// lane that has no more than 8 of them.  So a lane takes 16, half a group: a row
// lies in HD / 16 lanes, and a warp has a row's K and V side by side, at HD = 128
// two rows' (write4_at_once).  As many blocks as the SMs hold (write4_blocks) go
// through the rows, and load the next ones before they quantise these: many rows by
// two, few at HD = 256 by one.
//   28672 tokens of 2 heads of 256: 17.6 us for 75 MB, 4.2 TB/s; 17421 tokens of 4
// heads of 128: 12.8 us for 46 MB, 3.6 TB/s (8 values a lane: 22.8 and 15.7; blocks
// in waves, as above: 19.6 and 13.1; four rows of 256 with two blocks per SM: 17.5).
// Bound by instructions and by the look-ups, three dependent loads for two rows.
__host__ __device__ constexpr int write4_at_once(int hd) { return 256 / hd; }
__host__ __device__ constexpr int write4_blocks(int hd, int rows) { return hd * rows > 256 ? 3 : 4; }
template <int HD, int ROWS>
__global__ void __launch_bounds__(256, write4_blocks(HD, ROWS))
    paged_write4_kernel(const __grid_constant__ PagedWriteParams p) {
  constexpr int LANES = HD / 16, AT_ONCE = write4_at_once(HD), STEPS = ROWS / AT_ONCE;
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, l = lane % LANES;
  const bool is_k = (lane / LANES & 1) == 0;
  const int own = lane / (2 * LANES);  // row of a step's
  const int nkv = p.pool.nkv;
  const int groups = (nkv + p.heads_per_item - 1) / p.heads_per_item;
  const long long items = static_cast<long long>((p.rows + ROWS - 1) / ROWS) * groups;
  const long long warps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
  const uint4* from = is_k ? p.k_new : p.v_new;
  uint2* codes = static_cast<uint2*>(is_k ? p.pool.k : p.pool.v);
  uint32_t* records = reinterpret_cast<uint32_t*>(is_k ? p.pool.k_scales : p.pool.v_scales);
  uint4 x[STEPS][2], y[STEPS][2];
  auto load = [&](int row0, int g) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int row = min(row0 + i * AT_ONCE + own, p.rows - 1);
      const uint4* src = from + (static_cast<long long>(row) * nkv + g) * (HD / 8) + 2 * l;
      y[i][0] = load_now(src);
      y[i][1] = load_now(src + 1);
    }
  };
  long long it = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (it >= items) return;
  int row0 = static_cast<int>(it / groups) * ROWS, g0 = static_cast<int>(it % groups) * p.heads_per_item;
  load(row0, g0);
  while (true) {
    const int g1 = min(nkv, g0 + p.heads_per_item);
    const int seq = p.row_starts != nullptr ? write_seq(p, row0, lane) : 0;
    const int row = row0 + lane;
    const long long mine =
        lane < ROWS ? write_place(p, row, p.row_starts != nullptr ? seq : row) : -1;
    long long place[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) place[i] = __shfl_sync(0xFFFFFFFFu, mine, i * AT_ONCE + own);
    it += warps;
    for (int g = g0; g < g1; ++g) {
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        x[i][0] = y[i][0];
        x[i][1] = y[i][1];
      }
      if (g + 1 < g1) {
        load(row0, g + 1);
      } else if (it < items) {
        row0 = static_cast<int>(it / groups) * ROWS;
        g0 = static_cast<int>(it % groups) * p.heads_per_item;
        load(row0, g0);
      }
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const uint32_t w[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w,
                               x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
        uint32_t mag = max(amax_bits(x[i][0]), amax_bits(x[i][1])) << 16;
        mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, 1));
        uint32_t all = mag;
#pragma unroll
        for (int o = LANES / 2; o >= 2; o >>= 1) all = max(all, __shfl_xor_sync(0xFFFFFFFFu, all, o));
        const Scales4 c = scales4(mag, all);
        float q[2][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 v = quotients4(bf16x2_to_f32x2(w[j]), c);
          q[j >> 2][2 * (j & 3)] = v.x;
          q[j >> 2][2 * (j & 3) + 1] = v.y;
        }
        const bool some = c.r != 0u;
        const uint2 z = make_uint2(some ? pack_e2m1x8(q[0]) : 0u, some ? pack_e2m1x8(q[1]) : 0u);
        uint32_t r = c.r;
        r |= __shfl_down_sync(0xFFFFFFFFu, r, 2) << 8;
        r |= __shfl_down_sync(0xFFFFFFFFu, r, 4) << 16;
        if (place[i] < 0) continue;
        const long long dst =
            pool_row(p.pool, static_cast<int>(place[i] >> 8), g, static_cast<int>(place[i] & 255));
        codes[dst * LANES + l] = z;
        uint32_t* rec = records + dst * (record_bytes(HD) / 4);
        if (l == 0) rec[0] = __float_as_uint(c.s);
        if ((l & 7) == 0) rec[1 + l / 8] = r;
      }
    }
    if (it >= items) break;
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
__device__ __forceinline__ void load_vec(uint32_t& x, const void* pool, long long at) {
  x = load_now(reinterpret_cast<const uint32_t*>(pool) + at);
}
// (s: e2m1: s r_g.  A row of ordinary magnitudes comes back exactly: s r_g x4 has
// at most 6 significant bits.)
__device__ __forceinline__ uint4 widen_vec(uint32_t x, float s, bool f16, bool* overflow) {
  uint32_t h[4], o[4];
  e2m1x8_to_f16x8(x, h);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = f16x2_to_f32x2(h[j]);
    if (f16) {
      o[j] = pack_f16x2(f.x * s, f.y * s);
      if ((o[j] & 0x7C00u) == 0x7C00u || (o[j] & 0x7C000000u) == 0x7C000000u) *overflow = true;
    } else {
      o[j] = pack_bf16x2(f.x * s, f.y * s);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
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
// From e2m1 pages: the same 28672 tokens 17.7 us for 75 MB, 17421 of 4 heads of 128
// 14.5 us for 46 MB: as many rows, look-ups and blocks for half the bytes (runs of 8 or
// 16 tokens, and grids of resident blocks only, were no faster; 16 values a lane with
// stores of 32 bytes took half the instructions and 19.1 and 15.0 us).
constexpr int kReadRun = 4;

template <int HD, int FMT>
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
      typename std::conditional<FMT == kBf16, uint4,
                                typename std::conditional<FMT == kE4m3, uint2, uint32_t>::type>::type
          x[RUN][LOADS];
      float sc[RUN][LOADS];
#pragma unroll
      for (int r = 0; r < RUN; ++r)
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
          const bool is_k = LOADS == 1 ? k_lane : l == 0;
          load_vec(x[r][l], is_k ? p.pool.k : p.pool.v, (src + r) * VECS + vec);
          const float* scales = is_k ? p.pool.k_scales : p.pool.v_scales;
          if (FMT == kE4m3) sc[r][l] = load_now(scales + src + r);
          if (FMT == kE2m1) {
            const float* rec = scales + (src + r) * (record_bytes(HD) / 4);
            const uint8_t rg = load_now(reinterpret_cast<const uint8_t*>(rec) + 4 + vec / (kGroup4 / 8));
            sc[r][l] = load_now(rec) * f16x2_to_f32x2(e4m3x2_to_f16x2(rg)).x;
          }
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
