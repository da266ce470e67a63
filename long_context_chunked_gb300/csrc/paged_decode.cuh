// Decode attention over the paged KV cache: one new token per sequence,
//   O[b, h] = sum_t p_t v_t / l,  p_t = 2^(x_t - m),  x_t = scale log2(e) <q, k_t>,
//   m >= max_t x_t - 8,  l = sum_t p_t,  LSE = (m + log2 l) ln 2
// over the cached tokens of kv head g = h / G.
//
// HBM-bound: a cached row is read once and used for the G q heads of its kv head,
// 4 HD G flops per 4 HD bytes (bf16), far below what even the legacy tensor path
// delivers per byte.  (Of more than 16 heads every further block of 16 copies
// the rows again, mostly from L2: 8 x 32768 bf16 tokens of 32 heads on one kv
// head of 128 move 171 MB of DRAM for 134 MB, 41.0 us; of 16 heads 32.6 us.)  So
// the kernel is built around an unbroken stream of TMA copies, and computes with
// mma.sync, transposed:
// S^T = K Q^T and O^T += V^T P^T put the cached rows on M = 16 and the q heads
// on N = 8, so a group of up to 8 heads pays for 8.  tcgen05's M = 128 would
// leave most of its rows empty, or need e4m3 V converted to fp16 through
// shared memory, while here that conversion sits in registers between
// ldmatrix and mma.
//
// Work split.  The cache is cut into tiles of WT tokens of one row = (sequence,
// kv head, block of up to 16 q heads).  All tiles of all rows form one list
// (sequence-major, then kv head), and each WORKER of the grid takes an equal,
// contiguous slice of it, whatever the lengths are: one long sequence and many
// ragged ones are balanced alike, and nothing depends on lengths the host does
// not know.  A worker works alone: it issues its own TMA copies into its own
// ring of slots (K and V tiles alternate, the next copy goes out as soon as a
// slot is read), holds Q, m, l and O (all HD columns) in registers, and turns
// the accumulators of K Q^T into the operand of V^T P^T there (movmatrix).  A
// row inside its slice it finishes by itself.  At most its first and its last
// row are shared with other workers; their (m, l, O) go to the workspace as
// pieces, which a second kernel joins in list order, so that results do not
// depend on timing:
//   m = max m_i,  O = sum 2^(m_i - m) O_i / sum 2^(m_i - m) l_i.
// A CTA whose whole slice lies in one row deals its tiles to the workers in
// turn, sums their O in shared memory, in worker order, and leaves one piece:
// neighbouring tiles read at the same time keep DRAM 15 % faster than 8 streams
// per SM.  So where there are few rows and every one is worth a CTA or more,
// the CTAs are dealt to the rows first (each row a whole number of them).
//
// A worker is one warp, and a row up to 16 q heads of a kv head: its O then
// takes up to HD / 2 registers, and 8 warps fit an SM.  (Two warps of 8
// heads on the same slots convert everything twice: 1x128k e4m3 took 40 us
// where one warp of 16 heads took 28, both without the join.)
//
// e4m3 (Q8): K and V are converted to fp16 (exact) in registers; mma.sync on
// e4m3 operands takes the same conversions and adds fp32 additions (measured
// by instruction counters).  Q is fp16, scaled by a power of two per head so
// that its largest element is in [1, 2): elements below 2^-14 of it lose bits,
// at most 2^-25 of the largest.  A K row's scale multiplies its logit.  A V
// row's scale multiplies its probability: P is stored as p_t s_t 2^7 / W,
// rounded once to fp16.  W is a power of two, at most twice the largest product
// p_t s_t that the head has met in the slice (or 2^-100), and no product passes
// 448 W.  So a scale counts as far as its token's probability goes: below a
// reference that is at least every scale, one V row of 1e10 at a logit of -50
// left nothing of rows of 1.  fp16 holds 11 bits of products down to 2^-21 W,
// fewer below, and none below 2^-32 W.  (Against one reference per warp, which
// was wrong: 1x128k 37.8 -> 38.9 us, 64 ragged 59.0 -> 58.3.  The largest product
// found by a bound from p and s apart, and then once more token by token: 39.2.)
// bf16: P is carried as a bf16 hi + lo pair against bf16 V.  hi is cut, not
// rounded, and lo takes 2^-22 p besides (far below its own rounding, 2^-16 p), so
// that both are positive wherever p is: an infinite v_t stays infinite, where a lo
// of 0 or below would make NaN of it.
//
// m and W are references, not exact maxima: they are raised only when a logit
// exceeds m by 8, so p stays below 2^8, or a P would pass 57344, which after a
// row's first tile hardly happens.  O is in units of W / 2^7.
//
// Measured (both launches): 8 x 32768 tokens, bf16, 32 q heads on 2 kv heads of
// 256: 97 us for 537 MB (5.5 TB/s, 82 % of a copy's rate); 64 ragged sequences
// of 1 to 8191 tokens, e4m3, 32 on 4 of 128: 58.1 us for 275 MB (4.7 TB/s,
// 70 %), 16 on 2 of 256: 59.3 us; 1 x 126977, e4m3, 32 on 2 of 256: 38.9 us for
// 132 MB (3.4 TB/s, 50 %), 8 on 2 of 256: 33.9 us; 1 x 500, bf16, 8 on 2 of 128:
// 8.0 us where the table's row names 768 tokens at most, 9.3 us where it has
// room for more, so that the join has to be launched.  What lies between them
// and the copy's rate: about 7 us until the first tile is in (lengths, page
// ids, tile: three round trips, one after the other), 4 to 5 us of join, and
// CTAs that end apart (9 or 10 to a row of the first case).  While tiles flow,
// bf16 is bound by DRAM, and e4m3 by the latency of conversions and products
// in 8 warps (a quarter of the issue slots is used).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "paged.cuh"
#include "ptx.cuh"

namespace cpattn {

constexpr float kRaise = 8.f;                    // m is raised when a logit exceeds it by this
constexpr float kPScale = 128.f;                 // Q8: P is stored times 2^7 / W
constexpr float kMinW = 7.888609052210118e-31f;  // 2^-100: kPScale / W stays finite
constexpr float kMaxW = 8.507059173023462e+37f;  // 2^126, far above the largest scale of 2^119
constexpr float kPMax = 57344.f;                 // Q8: W is raised where a P would pass this
constexpr float kAboveOne = 1.00000023841857910f;  // 1 + 2^-22 (bf16: P's lo)
constexpr int kDecMaxHeads = 16;                 // of a row
constexpr int kDecStages = 8;                    // tiles whose absent pages a worker remembers

// NB: blocks of 8 q heads of a row (1: groups of up to 8 heads; 2: the rest).
// NW workers per CTA with NSLOT slots of SLOT bytes each, 192 KB in all; WT
// tokens per tile.  8 KB slots and 8 workers: more and smaller ones pay the
// fixed cost of a tile more often (64 ragged at HD = 128: 16 workers with 4 KB
// slots 80 us, 12 68 us, 8 with 8 KB 66 us; later, 12 workers with two slots of
// 8 KB 60.7 us, 8 with three 58.0), and at HD = 256 12 workers spill besides
// (e4m3, NB = 1, four slots of 4 KB: 1x126977 36.6 us, 33.9 by 8; 64 ragged of 8
// heads per kv head 64.5 and 59.3).
template <int HD, bool Q8, int NB>
struct DecodeLayout {
  static constexpr int ESZ = Q8 ? 1 : 2;
  static constexpr int NW = 8;
  static constexpr int THREADS = 32 * NW;
  static constexpr int SLOT = 8192;
  static constexpr int NSLOT = 196608 / (NW * SLOT);
  static constexpr int WT = SLOT / (HD * ESZ);
  static constexpr int WT_SHIFT = WT == 16 ? 4 : (WT == 32 ? 5 : 6);
  // Beginning and ending a row costs a worker about as much as 40 KB of tiles;
  // the list counts them before the row's first tile (64 ragged sequences,
  // tiles of 16 KB: 70 us without, 62.9 with one, 59.3 with two, 58.9 with three).
  static constexpr int ROW = 40960 / (2 * SLOT);
  static constexpr int BOXW = 128 / ESZ;         // values per 128-byte box row
  static constexpr int NBOX = HD / BOXW;         // column blocks of a tile
  static constexpr int MT = WT / 16;             // m-tiles of K Q^T
  static constexpr int MO = HD / 16;             // m-tiles of V^T P^T
  static constexpr int HEADS = 8 * NB;
  // Where O leaves no registers for Q, Q is read from shared memory: once for
  // the CTA if it is uniform, else each worker has its own in the place of its
  // third slot.
  static constexpr bool Q_SMEM = HD * NB == 512;
  static constexpr int Q_BYTES = HEADS * HD * 2;
  static constexpr int C_STRIDE = HD + 8;        // floats of a head's O where workers sum theirs
  static constexpr int OFF_SCALE = NW * NSLOT * SLOT;
  static constexpr int OFF_Q = OFF_SCALE + (Q8 ? NW * NSLOT * WT * 4 : 0);
  static constexpr int OFF_QEXP = OFF_Q + (Q_SMEM ? Q_BYTES : 0);  // [NW][HEADS] 2^e of each Q row
  static constexpr int OFF_ENDS = OFF_QEXP + (Q_SMEM ? NW * HEADS * 4 : 0);  // [THREADS] 64-bit
  static constexpr int OFF_ML = OFF_ENDS + THREADS * 8;  // [NW][HEADS] (m, l)
  static constexpr int OFF_BAR = OFF_ML + NW * HEADS * 8;
  static constexpr int OFF_BAD = OFF_BAR + NW * NSLOT * 8;  // [NW][kDecStages] absent boxes of a tile
  static constexpr int OFF_MISC = OFF_BAD + NW * kDecStages * 4;  // spots, scan, abort flag
  static constexpr int SMEM_BYTES = OFF_MISC + NW * 16 + THREADS / 32 * 8 + 16;
  static_assert(HEADS * C_STRIDE * 4 <= NSLOT * SLOT, "a worker's O fits its slots");
  static_assert(!Q_SMEM || (NSLOT == 3 && Q_BYTES <= SLOT && OFF_Q % 512 == 0),
                "a worker's Q fits a slot, and chunks can be XORed into a row's address");
  static_assert(OFF_BAR % 8 == 0 && OFF_MISC % 16 == 0 && OFF_SCALE % 128 == 0 && OFF_Q % 16 == 0 && OFF_ENDS % 8 == 0,
                "shared memory alignment");
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(NSLOT / 2 + 3 <= kDecStages, "tiles between their look-up and their use");
};

// A row in several pieces, by their places in the workspace, in list order:
// head0, then the first places of the workers head_w + 1 .. (n_head in all),
// those of the CTAs mid_cta .. (n_mid) and of the workers tail_w .. (n_tail).
// n_head + n_mid + n_tail == 0: not in pieces.
struct DecodeCut {
  int b, rr, head0, head_w, n_head, mid_cta, n_mid, tail_w, n_tail, pad[3];
};

constexpr int kBriefRounds = 3;  // rounds of tiles that a CTA alone does for a short row

struct PagedDecodeParams {
  CUtensorMap tm_k;  // [pool rows][HD], box BOXW x 1 x min(page_size, WT)
  CUtensorMap tm_v;
  PagedPool pool;
  const int* lens;            // [num_seqs]; <= 0: no tokens
  const __nv_bfloat16* q;     // [num_seqs][NQ][HD]
  __nv_bfloat16* out;
  float* lse;                 // or null
  float* ws_o;                // [2 * workers][8 NB][HD] O of a worker's first / last row
  float2* ws_ml;              // [2 * workers][8 NB] its m and l
  // The cut row that begins in a worker's slice; by row, where there are no
  // more rows than CTAs, else by worker.
  DecodeCut* ws_cut;          // [workers]
  int* status;
  uint32_t* bar_counts;       // barrier-count build: by CTA and worker, else unused
  unsigned long long timeout_ns;
  int pool_rows;              // num_pages * NKV * page_size
  int debug_flags;
  int by_row;                 // ws_cut is indexed by row
  int workers;                // per CTA
  int piece_rows;             // 8 NB
  int num_ctas;               // CTAs of the decode kernel
  int num_seqs, nq, group, hblocks;  // hblocks: blocks of 8 NB q heads per kv head
  float scale_log2;
};

enum : int { kSiteDecFull = 9 };  // after the prefill's sites
// Barrier-count build, by worker: copies sent (row kCountRowArrive) and copies
// seen to have landed, which have to be as many.
constexpr int kCountRowLanded = 1;

// ------------------------------------------------------------------ mma.sync
// c (16 x 8) = (ZERO ? 0 : c) + A (16 x 16) B (16 x 8).
template <bool F16, bool ZERO = false>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (F16 && ZERO)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  else if constexpr (ZERO)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  else if constexpr (F16)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit values, two neighbouring columns per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Asynchronous copy of 16 bytes, and an arrival on `bar` once this thread's
// copies so far have landed.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src))
               : "memory");
}
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// The power of two at or above x, 2^-126 <= x <= 2^127, and 1 / x of a power of
// two x, 2^-126 <= x <= 2^126: W's arithmetic, exact.
__device__ __forceinline__ float pow2_above(float x) {
  return __uint_as_float((__float_as_uint(x) + 0x7FFFFFu) & 0x7F800000u);
}
__device__ __forceinline__ float pow2_inverse(float x) {
  return __uint_as_float(0x7F000000u - __float_as_uint(x));
}

// Four e4m3 values as two fp16 pairs (exact).
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t x, uint32_t* lo, uint32_t* hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(*lo), "=r"(*hi)
      : "r"(x));
}

// Shared address of 16-byte chunk `chunk` of row `row` in the column block at
// `base` (rows of 128 bytes, as a 128-byte-swizzled TMA box stores them).
__device__ __forceinline__ uint32_t sw128(uint32_t base, int row, int chunk) {
  return base + row * 128 + ((chunk ^ (row & 7)) << 4);
}

// ------------------------------------------------------------- the slices
// Tokens of sequence b, cut to what its table row can name.
__device__ __forceinline__ int decode_len(const PagedDecodeParams& p, int b) {
  const long long room = static_cast<long long>(p.pool.max_pages) << p.pool.page_shift;
  return static_cast<int>(max(0LL, min(static_cast<long long>(load_now(p.lens + b)), room)));
}

// Tiles of n tokens (unsigned: n may end less than a tile below 2^31).
template <int WT>
__device__ __forceinline__ int tile_count(int n) {
  return static_cast<int>((static_cast<uint32_t>(n) + WT - 1) / WT);
}

// Units of the list that a row of sequence b takes.
template <int WT, int ROW>
__device__ __forceinline__ int row_units(const PagedDecodeParams& p, int b) {
  const int n = decode_len(p, b);
  return n > 0 ? tile_count<WT>(n) + ROW : 0;
}

// Quotients of tile counts, which hardly ever pass 32 bits: a 64-bit division
// takes far longer than a 32-bit one, and every warp waits for a few of these.
__device__ __forceinline__ long long div_count(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// Slices: worker w of the `active` ones that share the list takes the tiles
// [start(w), start(w + 1)), q of them and one more for w < r; tile i belongs to
// worker owner(i).
struct DecodeSlices {
  long long total, q;
  int active, r;

  __device__ __forceinline__ void init(long long total_, long long workers) {
    total = total_;
    active = static_cast<int>(min(total, workers));
    q = active > 0 ? div_count(total, active) : 0;
    r = static_cast<int>(total - q * active);
  }
  __device__ __forceinline__ long long start(int w) const { return q * w + min(w, r); }
  __device__ __forceinline__ int owner(long long i) const {
    const long long big = (q + 1) * r;  // tiles of the slices with q + 1
    return static_cast<int>(i < big ? div_count(i, q + 1) : r + div_count(i - big, q));
  }
};

// A worker's way through its slice [s, s1) of the list, one row segment (`units`
// of the list) at a time: tiles tile0, tile0 + step, .. (`tiles` of them) of row rr = kv head
// * hblocks + head block of sequence b.  tiles == 0: the slice is done.
struct DecodeWalk {
  long long s, s1;
  int b, rr, tile0, tiles, units, step, nt, n;

  // To the segment that begins at unit u of row (b, rr), or behind it to the
  // first one with tiles.
  template <int WT, int ROW>
  __device__ __forceinline__ void enter(const PagedDecodeParams& p, int rows_per_seq, int u) {
    n = decode_len(p, b);
    nt = tile_count<WT>(n);
    while (true) {
      units = static_cast<int>(min(static_cast<long long>(nt + ROW - u), s1 - s));
      tile0 = max(u - ROW, 0);
      tiles = max(u + units - ROW, 0) - tile0;
      if (tiles > 0 || s + units >= s1) return;
      s += units;
      u = 0;
      step_row<WT, ROW>(p, rows_per_seq);
    }
  }
  template <int WT, int ROW>
  __device__ __forceinline__ void step_row(const PagedDecodeParams& p, int rows_per_seq) {
    if (++rr < rows_per_seq) return;
    rr = 0;
    do {
      n = decode_len(p, ++b);
    } while (n == 0);
    nt = tile_count<WT>(n);
  }
  template <int WT, int ROW>
  __device__ __forceinline__ void next(const PagedDecodeParams& p, int rows_per_seq) {
    s += units;
    tiles = 0;
    if (s >= s1) return;
    step_row<WT, ROW>(p, rows_per_seq);
    enter<WT, ROW>(p, rows_per_seq, 0);
  }
};

// Whole block: the slices, and where each worker's one begins: spot[w] =
// (b, rr, tile0); or, where the CTAs are dealt to the rows, this CTA's row and
// share: spot[0] = (b, rr, its number among the row's CTAs, their number),
// and true is returned.  `ends` (shared memory): per thread, the list index
// behind its sequences.
//   Few short rows (no more rows than CTAs, none of more than three tiles per
// worker) take a CTA each: nothing is left to join (1x500: 10.9 us joined from
// two CTAs per row).
//   Dealt to the rows: row r takes the CTAs round(P_r n / total) ..
// round(P_r+1 n / total) - 1 of n, P the tiles of the rows before it, if that
// leaves every row a CTA and no CTA more than 1.2 times the mean.
template <int WT, int ROW, int NW>
__device__ __forceinline__ bool decode_slices(const PagedDecodeParams& p, int rows_per_seq,
                                              long long* warp_sum, long long* ends, int4* spot,
                                              DecodeSlices* out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.num_seqs + 32 * NW - 1) / (32 * NW);
  const int b0 = min(p.num_seqs, tid * per), b1 = min(p.num_seqs, b0 + per);
  const long long room = static_cast<long long>(p.pool.max_pages) << p.pool.page_shift;
  long long sum = 0;
  bool brief = p.by_row != 0;
  for (int b = b0; b < b1; ++b) {
    sum += row_units<WT, ROW>(p, b);
    brief = brief && decode_len(p, b) <= kBriefRounds * NW * WT;
    if (p.lens[b] > room && blockIdx.x == 0 && p.status != nullptr)
      atomicCAS(p.status, kStatusOk, kStatusPage);
  }
  long long inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_sum[warp] = inc;
  if (__syncthreads_and(brief)) {
    const int b = static_cast<int>(blockIdx.x) / rows_per_seq;
    if (tid == 0)
      spot[0] = make_int4(b, static_cast<int>(blockIdx.x) % rows_per_seq, 0,
                          b < p.num_seqs && decode_len(p, b) > 0 ? 1 : 0);
    out->init(0, 0);
    __syncthreads();
    return true;
  }
  long long base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) base += warp_sum[w];
    total += warp_sum[w];
  }
  ends[tid] = (base + inc) * rows_per_seq;
  out->init(total * rows_per_seq, static_cast<long long>(gridDim.x) * NW);
  bool dealt = p.by_row != 0;  // (one thread per sequence then)
  if (p.by_row) {
    const long long all = out->total;
    const int n = static_cast<int>(min(div_count(all + NW - 1, NW), static_cast<long long>(gridDim.x)));
    const long long before = (base + inc - sum) * rows_per_seq;
    int a = sum > 0 ? static_cast<int>(div_count(2 * before * n + all, 2 * all)) : 0;
    for (int rr = 0; rr < rows_per_seq && sum > 0; ++rr) {
      const int e = static_cast<int>(div_count(2 * (before + (rr + 1) * sum) * n + all, 2 * all));
      dealt = dealt && e > a && 5 * sum * n <= 6 * all * (e - a);
      if (a <= static_cast<int>(blockIdx.x) && static_cast<int>(blockIdx.x) < e)
        spot[0] = make_int4(tid, rr, static_cast<int>(blockIdx.x) - a, e - a);
      a = e;
    }
    if (tid == 0 && static_cast<int>(blockIdx.x) >= n) spot[0] = make_int4(0, 0, 0, 0);
  }
  if (__syncthreads_and(dealt)) return true;
  // Each worker looks for its slice's first tile: the first
  // thread whose sequences end behind it, then among that thread's sequences.
  const int worker = blockIdx.x * NW + warp;
  if (worker < out->active) {
    const long long s0 = out->start(worker);
    int t = 0;
    for (int k = 0; k < NW; ++k) {
      const uint32_t behind = __ballot_sync(0xFFFFFFFFu, ends[32 * k + lane] > s0);
      if (behind != 0u) {
        t = 32 * k + __ffs(static_cast<int>(behind)) - 1;
        break;
      }
    }
    long long a = t > 0 ? ends[t - 1] : 0;
    for (int b = t * per; b < p.num_seqs; ++b) {
      const int nt = row_units<WT, ROW>(p, b);
      const long long n = static_cast<long long>(nt) * rows_per_seq;
      if (s0 < a + n) {
        const int rr = static_cast<int>(div_count(s0 - a, nt));
        if (lane == 0)
          spot[warp] = make_int4(b, rr, static_cast<int>(s0 - a - static_cast<long long>(rr) * nt), 0);
        break;
      }
      a += n;
    }
  }
  __syncthreads();
  return false;
}

// ------------------------------------------------------------------ kernel
template <int HD, bool Q8, int NB>
__global__ void __launch_bounds__(DecodeLayout<HD, Q8, NB>::THREADS, 1)
    paged_decode_kernel(const __grid_constant__ PagedDecodeParams p) {
  using Ly = DecodeLayout<HD, Q8, NB>;
  constexpr int WT = Ly::WT, ROW = Ly::ROW, MT = Ly::MT, MO = Ly::MO, NSLOT = Ly::NSLOT, NW = Ly::NW;
  constexpr int HEADS = Ly::HEADS;
  // Where Q is in shared memory, K Q^T can be a loop that holds the code of KU
  // steps.  With e4m3's conversions a whole tile's code is more than the
  // instruction cache feeds without pauses (1x128k: 38.7 us unrolled, 37.4 by
  // twos, 38.6 by ones with the loop over V's halves rolled up too); with bf16
  // it is not (8x32k: 96.5 us unrolled, 99 by twos).
  constexpr bool ROLL = Ly::Q_SMEM && Q8;
  constexpr int KU = ROLL ? 2 : HD / 16;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, wk = tid >> 5;  // wk: worker of the CTA
  griddep_launch_dependents();
  // Swizzled copies need a 1024-byte aligned base (which the launch gives).
  if ((sbase & 1023u) != 0) {
    griddep_wait();
    if (tid == 0 && p.status != nullptr) atomicCAS(p.status, kStatusOk, kStatusLayout);
    // Nothing to join (by row: no more rows than CTAs).
    if (p.by_row ? tid == 0 : lane == 0)
      p.ws_cut[p.by_row ? blockIdx.x : blockIdx.x * NW + wk] = DecodeCut{};
    return;
  }
  const uint32_t full0 = sbase + Ly::OFF_BAR + wk * (8 * NSLOT);
  int4* spots = reinterpret_cast<int4*>(smem + Ly::OFF_MISC);
  volatile int* abort_flag =
      reinterpret_cast<volatile int*>(smem + Ly::OFF_MISC + NW * 16 + Ly::THREADS / 4);
  if (lane == 0) {
    for (int s = 0; s < NSLOT; ++s) {
      mbar_init(full0 + 8 * s, Q8 ? 1 + WT / 4 : 1);  // (Q8: the copies of the scales arrive too)
    }
    if (wk == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  if (tid == 0) {
    prefetch_tmap(&p.tm_k);
    prefetch_tmap(&p.tm_v);
  }
  // Launched as a programmatic dependent of whatever is ahead on the stream:
  // nothing above reads or writes global memory that another kernel does.
  griddep_wait();
  const int rows_per_seq = p.pool.nkv * p.hblocks;
  const int worker = blockIdx.x * NW + wk;
  DecodeSlices sl_;
  const bool dealt = decode_slices<WT, ROW, NW>(p, rows_per_seq,
                            reinterpret_cast<long long*>(smem + Ly::OFF_MISC + NW * 16),
                            reinterpret_cast<long long*>(smem + Ly::OFF_ENDS), spots, &sl_);
  const DecodeSlices slices = sl_;
  const int cta_w0 = static_cast<int>(blockIdx.x) * NW;
  const BoundedWait wait{abort_flag, p.status, p.timeout_ns, nullptr, 0u, 0};

  DecodeWalk at;
  at.s = at.s1 = 0;
  at.b = at.rr = at.tile0 = at.tiles = at.units = at.nt = at.n = 0;
  at.step = 1;
  // `uniform`: the CTA's whole slice, tiles [cta_t0, cta_t1) of its row, lies
  // in one row; the workers take its tiles in turn.
  bool uniform = dealt;
  int cta_t0 = 0, cta_t1 = 0;
  if (dealt) {
    const int4 mine = spots[0];
    at.b = mine.x;
    at.rr = mine.y;
    if (mine.w > 0) {
      at.n = decode_len(p, at.b);
      at.nt = tile_count<WT>(at.n);
      cta_t0 = static_cast<int>(div_count(static_cast<long long>(at.nt) * mine.z, mine.w));
      cta_t1 = static_cast<int>(div_count(static_cast<long long>(at.nt) * (mine.z + 1), mine.w));
    }
  } else {
    if (worker < slices.active) {
      at.s = slices.start(worker);
      at.s1 = slices.start(worker + 1);
      at.b = spots[wk].x;
      at.rr = spots[wk].y;
      at.template enter<WT, ROW>(p, rows_per_seq, spots[wk].z);
    }
    if (cta_w0 + NW <= slices.active) {
      const long long cta_units = slices.start(cta_w0 + NW) - slices.start(cta_w0);
      const int4 first = spots[0];
      if (first.z + cta_units <= row_units<WT, ROW>(p, first.x)) {
        uniform = true;
        at.b = first.x;
        at.rr = first.y;
        at.n = decode_len(p, at.b);
        at.nt = tile_count<WT>(at.n);
        cta_t0 = max(first.z - ROW, 0);
        cta_t1 = max(static_cast<int>(first.z + cta_units) - ROW, 0);
      }
    }
  }
  const int nslot = Ly::Q_SMEM && !uniform ? NSLOT - 1 : NSLOT;  // (see Q_SMEM)
  const uint32_t ring = sbase + wk * (nslot * Ly::SLOT);
  if (uniform) {
    at.s = at.s1 = at.units = 0;  // (one segment)
    at.tile0 = cta_t0 + wk;
    at.step = NW;
    at.tiles = max(0, (cta_t1 - at.tile0 + NW - 1) / NW);
  }

  // ------------------------------------------- the worker's stream of copies
  // Copy u of the worker is K (u even) or V (u odd) of its tile u / 2, in slot
  // u % nslot.  A slot should be refilled the moment it has been read, so what
  // the next copy needs is in registers by then: `cur` is the tile whose V goes
  // out next, `next` the one whose K does, and `raw` the page ids of the tile
  // behind it, loaded but not looked at.
  const int ps = 1 << p.pool.page_shift;
  const int box = min(ps, WT), box_shift = min(p.pool.page_shift, Ly::WT_SHIFT);
  const int boxes = WT >> box_shift;
  volatile uint32_t* my_bad =
      reinterpret_cast<volatile uint32_t*>(smem + Ly::OFF_BAD) + wk * kDecStages;
  DecodeWalk ahead = at;  // the tile whose page ids are loaded next
  int aj = 0;             // its index in ahead's segment
  // Lane i: first token of box i (-1: none), its page id, and the kv head.
  int raw_t = -1, raw_id = 0, raw_g = 0;
  bool raw_any = false, next_any = false;
  int next_row = 0, cur_row = 0;      // lane i: pool row of box i
  int next_scale = 0, cur_scale = 0;  // Q8: lane i: pool row of tokens 4 i .., or -1
  int resolved = 0, issued = 0, slot_out = 0;
  auto load_raw = [&]() {
    raw_any = ahead.tiles > 0;
    raw_t = -1;
    if (!raw_any) return;
    const int t = (ahead.tile0 + aj * ahead.step) * WT + (lane << box_shift);
    raw_g = ahead.rr / p.hblocks;
    if (lane < boxes && t < ahead.n) {
      raw_t = t;
      raw_id = load_now(p.pool.table + ahead.b * p.pool.table_stride + (t >> p.pool.page_shift));
    }
    if (++aj >= ahead.tiles) {
      ahead.template next<WT, ROW>(p, rows_per_seq);
      aj = 0;
    }
  };
  // raw becomes next.  A box's row is where it starts, or p.pool_rows (out of
  // range: TMA fills zeros) when it lies behind the last token or its page is
  // absent.
  auto resolve = [&]() {
    next_any = raw_any;
    bool bad = false;
    next_row = p.pool_rows;
    if (raw_t >= 0) {
      bad = static_cast<unsigned>(raw_id) >= static_cast<unsigned>(p.pool.num_pages);
      if (!bad) next_row = static_cast<int>(pool_row(p.pool, raw_id, raw_g, raw_t & (ps - 1)));
    }
    const uint32_t badm = __ballot_sync(0xFFFFFFFFu, bad);
    if (bad && p.status != nullptr) atomicCAS(p.status, kStatusOk, kStatusPage);
    if (lane == 0) my_bad[resolved & (kDecStages - 1)] = badm;
    ++resolved;
    if (Q8) {
      const int tok = 4 * lane;
      const int row = __shfl_sync(0xFFFFFFFFu, next_row, (tok & (WT - 1)) >> box_shift);
      next_scale = tok < WT && row < p.pool_rows ? row + (tok & (box - 1)) : -1;
    }
  };
  auto send = [&](const CUtensorMap* m, const float* scales, int row, int scale_row) {
    const uint32_t bar = full0 + 8 * slot_out, dst = ring + slot_out * Ly::SLOT;
    if (lane == 0) {
      count_arrive(p.bar_counts, 1u, wk, 1);
      mbar_arrive_expect_tx(bar, Ly::SLOT);
#pragma unroll
      for (int c = 0; c < Ly::NBOX; ++c) tma_load_3d(dst + c * (WT * 128), m, bar, c * Ly::BOXW, 0, row);
    }
    if (boxes > 1) {
      if (lane > 0 && lane < boxes) {
#pragma unroll
        for (int c = 0; c < Ly::NBOX; ++c)
          tma_load_3d(dst + c * (WT * 128) + (lane << box_shift) * 128, m, bar, c * Ly::BOXW, 0, row);
      }
    }
    if (Q8 && lane < WT / 4) {  // four tokens' scales (a page holds 16 or more)
      if (scale_row >= 0)
        copy16_async(sbase + Ly::OFF_SCALE + (wk * NSLOT + slot_out) * (WT * 4) + 16 * lane,
                     scales + scale_row);
      copies_arrive(bar);
    }
    if (++slot_out == nslot) slot_out = 0;
    ++issued;
  };
  auto advance = [&]() {
    cur_row = next_row;
    cur_scale = next_scale;
    resolve();
    load_raw();
  };
  // The next copy, if there is one: called nslot times at first, then once for
  // every slot read.
  auto issue = [&]() {
    if (issued & 1) {
      send(&p.tm_v, p.pool.v_scales, cur_row, cur_scale);
    } else if (next_any) {
      send(&p.tm_k, p.pool.k_scales, next_row, next_scale);
      advance();
    }
  };
  load_raw();
  {
    // (The second tile's page ids are on their way before the first's are
    // looked at.)
    const int t0 = raw_t, id0 = raw_id, g0 = raw_g;
    const bool any0 = raw_any;
    load_raw();
    const int t1 = raw_t, id1 = raw_id, g1 = raw_g;
    const bool any1 = raw_any;
    raw_t = t0, raw_id = id0, raw_g = g0, raw_any = any0;
    resolve();
    raw_t = t1, raw_id = id1, raw_g = g1, raw_any = any1;
  }
  if ((p.debug_flags & kDebugDropArrive) && blockIdx.x == 0 && wk == 0 && next_any) {
    // Fault injection: the worker's first copy is never sent.
    slot_out = 1;
    issued = 1;
    advance();
  }
#pragma unroll 1
  for (int i = 0; i < nslot; ++i)
    if (issued == i) issue();

  // Sequences without tokens: zeros, and an LSE of -infinity.
  for (int b = blockIdx.x; b < p.num_seqs; b += gridDim.x) {
    if (decode_len(p, b) > 0) continue;
    uint4* o = reinterpret_cast<uint4*>(p.out + static_cast<long long>(b) * p.nq * HD);
    for (int i = tid; i < p.nq * (HD / 8); i += Ly::THREADS) o[i] = make_uint4(0u, 0u, 0u, 0u);
    if (p.lse != nullptr)
      for (int h = tid; h < p.nq; h += Ly::THREADS)
        p.lse[static_cast<long long>(b) * p.nq + h] = -INFINITY;
    if (p.by_row)
      for (int r = tid; r < rows_per_seq; r += Ly::THREADS) p.ws_cut[b * rows_per_seq + r] = DecodeCut{};
  }
  if (!p.by_row && lane == 0) p.ws_cut[worker] = DecodeCut{};

  // Accumulator fragments (16 x 8): rows r0 and r0 + 8 (tokens or columns of
  // V), columns 2 quad and 2 quad + 1 (q heads of the block).
  const int quad = lane & 3, r0 = lane >> 2, r8 = lane & 7, oct = lane >> 3;
  int slot = 0, used = 0;  // the next slot to read, and copies read so far
  uint32_t phase = 0;
  // A warp whose wait expired, or that another warp's expired wait ends, is
  // through with its tiles (ok = false): it lets its copies in flight land,
  // still says where its rows' pieces are and meets every barrier, and the
  // status word tells the host.
  bool ok = true;
  auto await = [&]() {  // whether the copy in `slot` has landed, alike in the warp
    bool in = mbar_try_wait(full0 + 8 * slot, phase);
    if (!in) in = wait(full0 + 8 * slot, phase, kSiteDecFull);
    ok = __all_sync(0xFFFFFFFFu, in);
    __syncwarp();
    if (ok) count_wait(p.bar_counts, kCountRowLanded, wk);
    return ok;
  };
  // The slot has been read by every lane.  __syncwarp, and not the vote, orders
  // the lanes' reads (and clears) of it before the copies that a few of them
  // send into it, and of Q before the next row's.
  auto release = [&]() {
    __syncwarp();
    if (++slot == nslot) {
      slot = 0;
      phase ^= 1u;
    }
    ++used;
    issue();
  };
  // Copies used .. issued - 1 are in flight: they land before the ring is used
  // for something else and before the CTA exits.
  auto drain = [&]() {
    for (; used < issued; ++used) {
      if (mbar_wait_drain(full0 + 8 * slot, phase, 200ull * 1000 * 1000))
        count_wait(p.bar_counts, kCountRowLanded, wk);
      if (++slot == nslot) {
        slot = 0;
        phase ^= 1u;
      }
    }
    __syncwarp();
  };

  // (A worker without tiles still takes part in its CTA's sum.)
  for (bool once = uniform && cta_t1 > cta_t0; at.tiles > 0 || once;
       once = false, at.template next<WT, ROW>(p, rows_per_seq)) {
    const int g = at.rr / p.hblocks;
    const int h0 = g * p.group + (at.rr % p.hblocks) * HEADS;  // the row's first q head
    const int heads = min(HEADS, (g + 1) * p.group - h0);

    // B fragments of Q^T, 16 dims a step.  bf16: as it is, dims 16 ks + 2 quad +
    // {0, 1} and + 8 of head r0 of each block.  Q8: fp16, scaled by a power of
    // two, dims 16 ks + 4 quad + {0 .. 3}, the order in which the e4m3 K
    // fragments come out of ldmatrix.
    // For the largest magnitude `big` of a head (bf16 bits): e, the exponent of
    // the head's largest value (zeros and subnormals: -126), down = 2^-e, and
    // 2^e, which gives it back to the logits; 2^-127, 2^-128 and 2^128 are made
    // in two steps.
    auto scaling = [](uint32_t big, float* down, float* up) {
      const int e = max(static_cast<int>(big >> 7), 1) - 127;
      const int e1 = min(e, 126), e2 = e - e1;
      *down = __int_as_float((127 - e1) << 23) * (e2 == 0 ? 1.f : (e2 == 1 ? 0.5f : 0.25f));
      *up = __int_as_float((127 + e1) << 23) * (e2 == 0 ? 1.f : (e2 == 1 ? 2.f : 4.f));
    };
    uint32_t q[Ly::Q_SMEM ? 1 : HD / 16][2 * NB];
    float qexp[NB];
    // Q_SMEM: rows of HD 16-bit values, 16-byte chunks swizzled by the row.
    const uint32_t q_at = uniform ? Ly::OFF_Q : NW * (NSLOT - 1) * Ly::SLOT + wk * Ly::Q_BYTES;
    if constexpr (Ly::Q_SMEM) {
      float* exps = reinterpret_cast<float*>(smem + Ly::OFF_QEXP) + (uniform ? 0 : wk * HEADS);
      for (int r = uniform ? wk : 0; r < HEADS; r += uniform ? NW : 1) {
        const uint2* src = reinterpret_cast<const uint2*>(
            p.q + (static_cast<long long>(at.b) * p.nq + (r < heads ? h0 + r : h0)) * HD);
        uint2 w[HD / 128];
        uint32_t big = 0;
#pragma unroll
        for (int i = 0; i < HD / 128; ++i) {
          w[i] = r < heads ? load_now(src + 32 * i + lane) : make_uint2(0u, 0u);
          big = __vmaxu2(big, __vmaxu2(w[i].x & 0x7FFF7FFFu, w[i].y & 0x7FFF7FFFu));
        }
        if constexpr (Q8) {
          big = __reduce_max_sync(0xFFFFFFFFu, max(big & 0xFFFFu, big >> 16));
          float down, up;
          scaling(big, &down, &up);
          if (lane == 0) exps[r] = up;
#pragma unroll
          for (int i = 0; i < HD / 128; ++i) {
            w[i].x = pack_f16x2(__uint_as_float(w[i].x << 16) * down,
                                __uint_as_float(w[i].x & 0xFFFF0000u) * down);
            w[i].y = pack_f16x2(__uint_as_float(w[i].y << 16) * down,
                                __uint_as_float(w[i].y & 0xFFFF0000u) * down);
          }
        }
#pragma unroll
        for (int i = 0; i < HD / 128; ++i) {
          // Dims 4 k .. 4 k + 3, k = 32 i + lane: 8 bytes.  Q8: dims 4 a + 2 c of
          // a 16-block go to position 2 a + 8 c.
          const int k = 32 * i + lane;
          const int c0 = Q8 ? 2 * (k >> 2) : k >> 1;
          uint8_t* row = smem + q_at + r * (2 * HD);
          if constexpr (Q8) {
            *reinterpret_cast<uint32_t*>(row + ((c0 ^ (r & 7)) << 4) + (k & 3) * 4) = w[i].x;
            *reinterpret_cast<uint32_t*>(row + (((c0 + 1) ^ (r & 7)) << 4) + (k & 3) * 4) = w[i].y;
          } else {
            *reinterpret_cast<uint2*>(row + ((c0 ^ (r & 7)) << 4) + (k & 1) * 8) = w[i];
          }
        }
      }
      if (uniform)
        __syncthreads();
      else
        __syncwarp();
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) qexp[nb] = Q8 ? exps[8 * nb + r0] : 1.f;
    } else {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const bool here = 8 * nb + r0 < heads;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(
            p.q + (static_cast<long long>(at.b) * p.nq + (here ? h0 + 8 * nb + r0 : h0)) * HD);
        uint32_t big = 0;
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          uint2 w;
          if constexpr (Q8) {
            w = load_now(reinterpret_cast<const uint2*>(src) + 4 * ks + quad);
          } else {
            w.x = load_now(src + 8 * ks + quad);
            w.y = load_now(src + 8 * ks + 4 + quad);
          }
          if (!here) w = make_uint2(0u, 0u);
          q[ks][2 * nb] = w.x;
          q[ks][2 * nb + 1] = w.y;
          if (Q8) big = __vmaxu2(big, __vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu));
        }
        qexp[nb] = 1.f;
        if constexpr (Q8) {
          big = max(big & 0xFFFFu, big >> 16);
          big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
          big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
          float down;
          scaling(big, &down, &qexp[nb]);
#pragma unroll
          for (int ks = 0; ks < HD / 16; ++ks)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t w = q[ks][2 * nb + j];
              q[ks][2 * nb + j] = pack_f16x2(__uint_as_float(w << 16) * down,
                                             __uint_as_float(w & 0xFFFF0000u) * down);
            }
        }
      }
    }
    const uint32_t q_row = sbase + q_at + ((NB == 2 ? (oct >> 1) * 8 : 0) + r8) * (2 * HD) +
                           (((oct & 1) ^ r8) << 4);
    auto q_frag = [&](int ks, uint32_t (&f)[4]) {  // [nb][b0, b1]
      if constexpr (Ly::Q_SMEM) {
        ldsm4(f, q_row ^ (ks << 5));
      } else {
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) f[i] = q[ks][i];
      }
    };
    float sl[NB][2], m[NB][2], l[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // of head 2 quad + j (never 0: -infinity times it has to stay -infinity)
        const float qe = __shfl_sync(0xFFFFFFFFu, qexp[nb], 4 * (2 * quad + j));
        sl[nb][j] = fmaxf(p.scale_log2 * qe, 1.17549435e-38f);
        m[nb][j] = -INFINITY;
        l[nb][j] = 0.f;
      }
    float ps[NB][2];  // Q8: 2^7 / W
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) ps[nb][0] = ps[nb][1] = kPScale / kMinW;
    float o[MO][NB][4];
#pragma unroll
    for (int i = 0; i < MO; ++i)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][nb][j] = 0.f;

    for (int v = 0; ok && v < at.tiles; ++v) {
      const int valid = min(WT, at.n - (at.tile0 + v * at.step) * WT);  // tokens of the tile

      // ---- S^T = K Q^T
      if (!await()) break;
      const uint32_t bad = my_bad[(used >> 1) & (kDecStages - 1)];
      const bool partial = valid < WT || bad != 0u;
      const uint32_t kb = ring + slot * Ly::SLOT;
      float c[MT][NB][4];
      if constexpr (ROLL) {
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 4; ++j) c[t][nb][j] = 0.f;
      }
      const uint32_t k_at = sw128(kb, (oct & 1) * 8 + r8, oct >> 1);  // (chunks are XORed in)
      if constexpr (Q8) {
#pragma unroll KU
        for (int ks = 0; ks < HD / 16; ks += 2) {  // 32 dims: chunks ks and ks + 1
          uint32_t qa[4], qb[4];
          q_frag(ks, qa);
          q_frag(ks + 1, qb);
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            uint32_t kr[4], a[4];  // token half, then chunk, by lane octet
            ldsm4(kr, (k_at ^ ((ks & 7) << 4)) + (ks >> 3) * (WT * 128) + t * 2048);
            e4m3x4_to_f16x4(kr[0], &a[0], &a[2]);
            e4m3x4_to_f16x4(kr[1], &a[1], &a[3]);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              if (ks == 0 && !ROLL)
                mma16816<true, true>(c[t][nb], a, qa[2 * nb], qa[2 * nb + 1]);
              else
                mma16816<true>(c[t][nb], a, qa[2 * nb], qa[2 * nb + 1]);
            }
            e4m3x4_to_f16x4(kr[2], &a[0], &a[2]);
            e4m3x4_to_f16x4(kr[3], &a[1], &a[3]);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma16816<true>(c[t][nb], a, qb[2 * nb], qb[2 * nb + 1]);
          }
        }
      } else {
#pragma unroll KU
        for (int ks = 0; ks < HD / 16; ++ks) {  // 16 dims: chunks 2 ks and 2 ks + 1
          uint32_t qf[4];
          q_frag(ks, qf);
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            uint32_t a[4];
            ldsm4(a, (k_at ^ ((2 * ks & 7) << 4)) + (ks >> 2) * (WT * 128) + t * 2048);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              if (ks == 0 && !ROLL)
                mma16816<false, true>(c[t][nb], a, qf[2 * nb], qf[2 * nb + 1]);
              else
                mma16816<false>(c[t][nb], a, qf[2 * nb], qf[2 * nb + 1]);
            }
          }
        }
      }
      // c becomes <q, k> times the token's scale; what is no token is -infinity,
      // by value.  The logits (log2 units) are c sl, taken with m below.
      const float* ksc = reinterpret_cast<const float*>(
          smem + Ly::OFF_SCALE + (wk * NSLOT + slot) * (WT * 4));
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float ks = Q8 ? ksc[16 * t + 8 * i + r0] : 1.f;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (Q8) c[t][nb][2 * i + j] *= ks;
        }
      bool seen[MT][2];
      if (partial) {
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int tok = 16 * t + 8 * i + r0;
            seen[t][i] = tok < valid && !((bad >> (tok >> box_shift)) & 1u);
            if (!seen[t][i]) {
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) c[t][nb][2 * i] = c[t][nb][2 * i + 1] = -INFINITY;
            }
          }
      }
      float mx[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          mx[nb][j] = fmaxf(c[0][nb][j], c[0][nb][2 + j]);
#pragma unroll
          for (int t = 1; t < MT; ++t)
            mx[nb][j] = fmaxf(mx[nb][j], fmaxf(c[t][nb][j], c[t][nb][2 + j]));
          mx[nb][j] *= sl[nb][j];  // sl > 0
        }
      release();

      // ---- m
      if (!await()) break;
      const uint32_t vb = ring + slot * Ly::SLOT;
      float vs[MT][2];
      if constexpr (Q8) {
        const float* vsc = reinterpret_cast<const float*>(
            smem + Ly::OFF_SCALE + (wk * NSLOT + slot) * (WT * 4));
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            vs[t][i] = vsc[16 * t + 8 * i + r0];
            if (partial && !seen[t][i]) vs[t][i] = 0.f;
          }
      }
      float a[NB][2];  // 2^(m before - m)
      bool raise = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          a[nb][j] = 1.f;
          raise |= mx[nb][j] > m[nb][j] + kRaise;
        }
      raise = __any_sync(0xFFFFFFFFu, raise);
      if (raise) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x = mx[nb][j];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
            const float mn = fmaxf(m[nb][j], x);
            if (m[nb][j] != mn) a[nb][j] = ex2_approx(m[nb][j] - mn);
            m[nb][j] = mn;
            l[nb][j] *= a[nb][j];
            if constexpr (!Q8) {
#pragma unroll
              for (int i = 0; i < MO; ++i) {
                o[i][nb][j] *= a[nb][j];
                o[i][nb][2 + j] *= a[nb][j];
              }
            }
          }
      }

      // ---- p (Q8: times the V row's scale), and l
      float wx[NB][2];  // Q8: the lane's largest product
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        wx[nb][0] = wx[nb][1] = 0.f;
        const float m0 = m[nb][0] == -INFINITY ? 0.f : m[nb][0];
        const float m1 = m[nb][1] == -INFINITY ? 0.f : m[nb][1];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float& e0 = c[t][nb][2 * i];
            float& e1 = c[t][nb][2 * i + 1];
            e0 = ex2_approx(fmaf(e0, sl[nb][0], -m0));
            e1 = ex2_approx(fmaf(e1, sl[nb][1], -m1));
            l[nb][0] += e0;
            l[nb][1] += e1;
            if constexpr (Q8) {
              e0 *= vs[t][i];
              e1 *= vs[t][i];
              wx[nb][0] = fmaxf(wx[nb][0], fabsf(e0));
              wx[nb][1] = fmaxf(wx[nb][1], fabsf(e1));
            }
          }
      }
      if constexpr (Q8) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 2; ++j) raise |= wx[nb][j] * ps[nb][j] > kPMax;
        if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float w = wx[nb][j];
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) w = fmaxf(w, __shfl_xor_sync(0xFFFFFFFFu, w, d));
              // W falls with p where m has risen, or rises to the tile's largest product.
              const float was = kPScale * pow2_inverse(ps[nb][j]) * a[nb][j];
              const float inv = pow2_inverse(pow2_above(fminf(fmaxf(fmaxf(was, w), kMinW), kMaxW)));
              const float as = was * inv;
              ps[nb][j] = kPScale * inv;
#pragma unroll
              for (int i = 0; i < MO; ++i) {
                o[i][nb][j] *= as;
                o[i][nb][2 + j] *= as;
              }
            }
        }
      }

      // ---- P, transposed into the B operand of V^T P^T (16 tokens per step)
      uint32_t ph[MT][NB][2], pl[Q8 ? 1 : MT][NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float e0 = c[t][nb][2 * i], e1 = c[t][nb][2 * i + 1];
            if constexpr (Q8) {
              ph[t][nb][i] = transpose8(pack_f16x2(e0 * ps[nb][0], e1 * ps[nb][1]));
            } else {
              // hi: the upper 16 bits; lo: the rest, and 2^-22 of the whole (kAboveOne).
              const uint32_t b0 = __float_as_uint(e0), b1 = __float_as_uint(e1);
              ph[t][nb][i] = transpose8(__byte_perm(b0, b1, 0x7632));
              pl[t][nb][i] =
                  transpose8(pack_bf16x2(fmaf(e0, kAboveOne, -__uint_as_float(b0 & 0xFFFF0000u)),
                                         fmaf(e1, kAboveOne, -__uint_as_float(b1 & 0xFFFF0000u))));
            }
          }

      // ---- O^T += V^T P^T
      if (valid < WT) {
        // Slots behind the last token may hold anything; 0 * NaN must not
        // reach O.
        constexpr int CH = HD * Ly::ESZ / 16;
        for (int i = lane; i < (WT - valid) * CH; i += 32) {
          const int ch = i % CH;
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                           sw128(vb + (ch >> 3) * (WT * 128), valid + i / CH, ch & 7)),
                       "r"(0)
                       : "memory");
        }
        __syncwarp();
      }
#pragma unroll
      for (int k = 0; k < MT; ++k) {
        if constexpr (Q8) {
#pragma unroll
          for (int ch = 0; ch < MO; ch += 2) {  // two 16-byte chunks: 32 columns
            uint32_t vr[4];  // token half, then chunk, by lane octet
            ldsm4_t(vr, sw128(vb + (ch >> 3) * (WT * 128), k * 16 + (oct & 1) * 8 + r8,
                              (ch & 7) + (oct >> 1)));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              // Each register holds two tokens x two columns; regrouped, the
              // lower half is the even column's (rows 0-7 of the m-tile), the
              // upper the odd one's (rows 8-15).
              uint32_t a[4];
              e4m3x4_to_f16x4(__byte_perm(vr[2 * j], 0u, 0x3120), &a[0], &a[1]);
              e4m3x4_to_f16x4(__byte_perm(vr[2 * j + 1], 0u, 0x3120), &a[2], &a[3]);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma16816<true>(o[ch + j][nb], a, ph[k][nb][0], ph[k][nb][1]);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < MO; ++i) {  // 16 columns: chunks 2 i and 2 i + 1
            uint32_t a[4];  // chunk, then token half, by lane octet
            ldsm4_t(a, sw128(vb + (i >> 2) * (WT * 128), k * 16 + (oct >> 1) * 8 + r8,
                             (2 * i & 7) + (oct & 1)));
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              mma16816<false>(o[i][nb], a, ph[k][nb][0], ph[k][nb][1]);
              mma16816<false>(o[i][nb], a, pl[k][nb][0], pl[k][nb][1]);
            }
          }
        }
      }
      // Cleared slots: these writes come before the copy that reuses the slot.
      if (valid < WT) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      release();
    }

    if (!ok) drain();

    // ---- the end of the row, or of this warp's part of it
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nb][j] += __shfl_xor_sync(0xFFFFFFFFu, l[nb][j], d);
    // Whether the row begins and ends here, and whether it is the CTA's alone.
    const bool begins = uniform ? cta_t0 == 0 && wk == 0 : at.tile0 == 0;
    const bool ends = !uniform && at.tile0 + at.tiles == at.nt;
    const bool cta_whole = uniform && cta_t0 == 0 && cta_t1 == at.nt;
    if (begins && lane == 0) {
      // The worker in whose slice a row begins says where its pieces are.
      DecodeCut d = {};
      d.b = at.b;
      d.rr = at.rr;
      if (dealt) {
        if (!cta_whole) {
          d.mid_cta = blockIdx.x;
          d.n_mid = spots[0].w;
        }
      } else if (!(ends || cta_whole)) {
        // List index behind the row's last tile.
        const long long end =
            uniform ? slices.start(cta_w0) - spots[0].z + ROW + at.nt
                    : at.s + at.units + (at.nt - at.tiles);
        const int last = slices.owner(end - 1), cta1 = last / NW;
        const bool one_last = last % NW == NW - 1 && slices.start(last + 1) == end;
        d.head0 = uniform ? 2 * worker : 2 * worker + 1;
        d.head_w = worker;
        d.n_head = uniform ? 1 : min(last, cta_w0 + NW - 1) - worker + 1;
        if (cta1 > static_cast<int>(blockIdx.x)) {
          d.mid_cta = blockIdx.x + 1;
          d.n_mid = cta1 - d.mid_cta + (one_last ? 1 : 0);
          d.tail_w = cta1 * NW;
          d.n_tail = one_last ? 0 : last - d.tail_w + 1;
        }
      }
      if (p.by_row)
        p.ws_cut[at.b * rows_per_seq + at.rr] = d;
      else if (d.n_head > 0)
        p.ws_cut[worker] = d;  // (at most one row that begins here is cut: the last)
    }
    float oscale[NB][2];  // of the O in registers
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < 2; ++j) oscale[nb][j] = Q8 ? pow2_inverse(ps[nb][j]) : 1.f;
    if (uniform) {
      // One piece for the CTA: the workers' m and l, then their O, summed in
      // worker order.  (The only row of every warp here.)
      float2* mls = reinterpret_cast<float2*>(smem + Ly::OFF_ML);
      if (r0 == 0) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            mls[wk * HEADS + 8 * nb + 2 * quad + j] = make_float2(m[nb][j], l[nb][j]);
      }
      __syncthreads();
      const long long piece = 2LL * blockIdx.x * NW;
      // The slots have been read (the barrier above): worker w's O goes there.
      constexpr int RING = NSLOT * Ly::SLOT;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = 8 * nb + 2 * quad + j;
          float mm = -INFINITY, sum = 0.f;
#pragma unroll
          for (int w = 0; w < NW; ++w) mm = fmaxf(mm, mls[w * HEADS + r].x);
          const float mref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            const float2 ml = mls[w * HEADS + r];
            sum = fmaf(ex2_approx(ml.x - mref), ml.y, sum);
          }
          float f = ex2_approx(m[nb][j] - mref) * oscale[nb][j];
          // sum = 0: every page of the row was absent.
          if (cta_whole) f = sum == 0.f ? 0.f : f / sum;
          if (wk == 0 && r0 == 0 && r < heads) {
            const long long orow = static_cast<long long>(at.b) * p.nq + h0 + r;
            if (!cta_whole)
              p.ws_ml[piece * HEADS + r] = make_float2(mm, sum);
            else if (p.lse != nullptr)
              p.lse[orow] = sum == 0.f ? -INFINITY : (mm + __log2f(sum)) * 0.69314718055994531f;
          }
          float* dst = reinterpret_cast<float*>(smem + wk * RING) + r * Ly::C_STRIDE;
#pragma unroll
          for (int i = 0; i < MO; ++i) {
            if constexpr (Q8) {  // rows r0, r0 + 8 of the m-tile: columns 2 r0 and 2 r0 + 1
              *reinterpret_cast<float2*>(dst + 16 * i + 2 * r0) =
                  make_float2(o[i][nb][j] * f, o[i][nb][2 + j] * f);
            } else {
              dst[16 * i + r0] = o[i][nb][j] * f;
              dst[16 * i + 8 + r0] = o[i][nb][2 + j] * f;
            }
          }
        }
      __syncthreads();
      for (int i = tid; i < HEADS * (HD / 4); i += Ly::THREADS) {
        const int r = i / (HD / 4), d = 4 * (i % (HD / 4));
        if (r >= heads) break;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float4 z = *reinterpret_cast<const float4*>(
              smem + w * RING + (r * Ly::C_STRIDE + d) * sizeof(float));
          y.x += z.x;
          y.y += z.y;
          y.z += z.z;
          y.w += z.w;
        }
        if (cta_whole)
          *reinterpret_cast<uint2*>(
              p.out + (static_cast<long long>(at.b) * p.nq + h0 + r) * HD + d) =
              make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
        else
          *reinterpret_cast<float4*>(p.ws_o + (piece * HEADS + r) * HD + d) = y;
      }
    } else {
      // This warp's own row, or its piece of one: straight from the registers.
      const bool whole = begins && ends;
      const long long piece = 2LL * worker + (begins ? 1 : 0);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = 8 * nb + 2 * quad + j;
          const float sum = l[nb][j];
          const float f = whole ? (sum == 0.f ? 0.f : oscale[nb][j] / sum) : oscale[nb][j];
          const long long orow = static_cast<long long>(at.b) * p.nq + h0 + r;
          const long long prow = piece * HEADS + r;
          if (r0 == 0 && r < heads) {
            if (!whole)
              p.ws_ml[prow] = make_float2(m[nb][j], sum);
            else if (p.lse != nullptr)
              p.lse[orow] =
                  sum == 0.f ? -INFINITY : (m[nb][j] + __log2f(sum)) * 0.69314718055994531f;
          }
#pragma unroll
          for (int i = 0; i < MO; ++i) {
            float2 y = make_float2(o[i][nb][j] * f, o[i][nb][2 + j] * f);
            int d = 16 * i + 2 * r0;
            if constexpr (!Q8) {
              // Rows r0 and r0 + 8 are columns r0 and r0 + 8: a neighbour's
              // value makes a pair.
              const bool odd = (r0 & 1) != 0;
              const float z = __shfl_xor_sync(0xFFFFFFFFu, odd ? y.x : y.y, 4);
              y = odd ? make_float2(z, y.y) : make_float2(y.x, z);
              d = 16 * i + (odd ? r0 + 7 : r0);
            }
            if (r < heads) {
              if (whole)
                *reinterpret_cast<uint32_t*>(p.out + orow * HD + d) = pack_bf16x2(y.x, y.y);
              else
                *reinterpret_cast<float2*>(p.ws_o + prow * HD + d) = y;
            }
          }
        }
    }
  }
}

// Joins the pieces of the rows that were cut.  Block (x, y): row x of the
// batch, and of its q heads the y-th part; or, where there are more rows than
// CTAs, every gridDim.y-th of the rows that begin in the slices of CTA x's
// workers.  A programmatic dependent of the decode kernel.  A unit of HD / 4
// threads takes one head and every `groups`-th of its pieces, each thread 4
// columns; the groups are summed in shared memory.  Each warp reads the
// pieces' (m, l) itself, while its first loads of O are in flight: two round
// trips to L2 per row.
constexpr int kJoinThreads = 1024;
constexpr int kJoinPieces = 288;  // most pieces of a row: one per CTA, and the workers of two
constexpr int kJoinBatch = 5;     // loads of O in flight per thread

struct JoinShared {
  float4 sums[kJoinThreads];
  float weight[kDecMaxHeads][kJoinPieces];
  float stats[kDecMaxHeads][2];  // m, l
  int place[kJoinPieces];
};

template <int HD>
__device__ __forceinline__ void join_row(const PagedDecodeParams& p, const DecodeCut& c, int part_of,
                                         int parts, JoinShared& sh) {
  constexpr int COLS = HD / 4;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int j = tid % COLS, unit = tid / COLS, units = blockDim.x / COLS;
  const int g = c.rr / p.hblocks, hrow = g * p.group + (c.rr % p.hblocks) * p.piece_rows;
  const int heads = min(p.piece_rows, (g + 1) * p.group - hrow);
  const int pieces = c.n_head + c.n_mid + c.n_tail;
  for (int i = tid; i < pieces; i += blockDim.x) {
    int at = i < c.n_head ? 2 * (c.head_w + i) : 2 * p.workers * (c.mid_cta + i - c.n_head);
    if (i == 0 && c.n_head > 0) at = c.head0;
    if (i >= c.n_head + c.n_mid) at = 2 * (c.tail_w + i - c.n_head - c.n_mid);
    sh.place[i] = at * p.piece_rows;
  }
  __syncthreads();
  // This block's heads, and how many groups share the pieces of one.
  const int per = (heads + parts - 1) / parts;
  const int ra = part_of * per, rb = min(heads, ra + per);
  int groups = 1;
  while (2 * groups * per <= units && 2 * groups <= pieces) groups *= 2;
  const int y = unit % groups, step = units / groups;
  // One warp per head makes its weights; the others' first loads of O are in
  // flight meanwhile.
  for (int r = ra + warp; r < rb; r += blockDim.x / 32) {
    float2 ml[kJoinPieces / 32];
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int k = 0; k < kJoinPieces / 32; ++k) {
      ml[k] = make_float2(-INFINITY, 0.f);
      if (32 * k + lane < pieces) ml[k] = p.ws_ml[sh.place[32 * k + lane] + r];
    }
#pragma unroll
    for (int k = 0; k < kJoinPieces / 32; ++k) m = fmaxf(m, ml[k].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    const float mref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int k = 0; k < kJoinPieces / 32; ++k) {
      if (32 * k >= pieces) break;
      const float w = ex2_approx(ml[k].x - mref);
      sh.weight[r][32 * k + lane] = w;
      l = fmaf(w, ml[k].y, l);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
    if (lane == 0) {
      sh.stats[r][0] = m;
      sh.stats[r][1] = l;
    }
  }
  float4 o[kJoinBatch];
  auto load = [&](int r, int i) {
    return *reinterpret_cast<const float4*>(p.ws_o + static_cast<long long>(sh.place[i] + r) * HD + 4 * j);
  };
  const int r0 = ra + unit / groups;
  if (r0 < rb) {
#pragma unroll
    for (int k = 0; k < kJoinBatch; ++k)
      if (y + k * groups < pieces) o[k] = load(r0, y + k * groups);
  }
  __syncthreads();
  for (int base = ra; base < rb; base += step) {
    const int r = base + unit / groups;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rb) {
      for (int i = y; i < pieces; i += kJoinBatch * groups) {
#pragma unroll
        for (int k = 0; k < kJoinBatch; ++k) {
          const int ii = i + k * groups;
          if (ii < pieces) {
            if (base > ra || i > y) o[k] = load(r, ii);
            const float w = sh.weight[r][ii];
            acc.x = fmaf(w, o[k].x, acc.x);
            acc.y = fmaf(w, o[k].y, acc.y);
            acc.z = fmaf(w, o[k].z, acc.z);
            acc.w = fmaf(w, o[k].w, acc.w);
          }
        }
      }
    }
    if (groups > 1) {
      sh.sums[tid] = acc;
      __syncthreads();
      if (y == 0) {
        for (int k = 1; k < groups; ++k) {
          const float4 z = sh.sums[tid + k * COLS];
          acc.x += z.x;
          acc.y += z.y;
          acc.z += z.z;
          acc.w += z.w;
        }
      }
      __syncthreads();
    }
    if (r < rb && y == 0) {
      const float m = sh.stats[r][0], l = sh.stats[r][1];
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const long long orow = static_cast<long long>(c.b) * p.nq + hrow + r;
      *reinterpret_cast<uint2*>(p.out + orow * HD + 4 * j) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      if (j == 0 && p.lse != nullptr)
        p.lse[orow] = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
    }
  }
  __syncthreads();  // the shared tables are reused by the next row
}

template <int HD>
__global__ void __launch_bounds__(kJoinThreads)
    paged_join_kernel(const __grid_constant__ PagedDecodeParams p) {
  __shared__ JoinShared sh;
  const int lane = threadIdx.x & 31, nw = p.workers;
  griddep_launch_dependents();
  griddep_wait();
  if (p.by_row) {
    const DecodeCut c = p.ws_cut[blockIdx.x];
    if (c.n_head + c.n_mid + c.n_tail > 0) join_row<HD>(p, c, blockIdx.y, gridDim.y, sh);
    return;
  }
  // Lane i looks at the row of worker i.
  uint32_t some = __ballot_sync(0xFFFFFFFFu, lane < nw && p.ws_cut[blockIdx.x * nw + lane].n_head > 0);
  for (int turn = 0; some != 0u; some &= some - 1u, ++turn)
    if (turn % static_cast<int>(gridDim.y) == static_cast<int>(blockIdx.y))
      join_row<HD>(p, p.ws_cut[blockIdx.x * nw + __ffs(static_cast<int>(some)) - 1], 0, 1, sh);
}

}  // namespace cpattn
