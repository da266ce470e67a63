// Decode attention over the paged KV cache: one new token per sequence,
//   O[b, h] = sum_t p_t v_t / l,  p_t = 2^(x_t - m),  x_t = scale log2(e) <q, k_t>,
//   m = max_t x_t,  l = sum_t p_t,  LSE = (m + log2 l) ln 2
// over the cached tokens of kv head g = h / G.
//
// HBM-bound: every cached row is read once and used for the G q heads of its
// kv head, 4 HD G flops per 4 HD bytes (bf16), far below what even the
// legacy tensor path delivers per byte.  So the kernel is built around an
// unbroken stream of TMA copies, and computes with mma.sync (M = 16 rows:
// the q heads of one kv head, padded): tcgen05's M = 128 would leave 7/8 of
// its rows empty and would need e4m3 converted to fp16 through shared memory
// first, while here the conversion sits in registers between ldmatrix and mma.
//
// Work split.  The cache is cut into tiles of TT tokens of one row = (sequence,
// kv head, block of up to 16 q heads).  All tiles of all rows form one list
// (sequence-major, then kv head), and each CTA takes an equal, contiguous
// slice of it, whatever the lengths are: one long sequence and many ragged
// ones are balanced alike, and nothing depends on lengths the host does not
// know.  A CTA holds at most two rows only in part (its first and its last);
// it writes their O, m, l to the workspace and a second kernel joins the
// pieces in order, so results do not depend on timing:
//   m = max m_i,  O = sum 2^(m_i - m) O_i / sum 2^(m_i - m) l_i.
//
// Roles (288 threads, two CTAs per SM): warps 0-7 compute, warp 8 issues TMA
// copies into a ring of slots (K and V tiles alternate).  Per tile, warp w
// computes S for TT/8 of the tokens and all heads, the warps agree on the row
// maxima (one named barrier), write P to shared memory (a second one), and
// warp w multiplies P with HD/8 of V's columns.
//
// e4m3 (Q8): K and V are converted to fp16 (exact) in registers.  Q is fp16,
// scaled by a power of two per head so that its largest element is in
// [1, 2): elements below 2^-14 of it lose bits, at most 2^-25 of the largest.
// A K row's scale multiplies its logit.  A V row's scale multiplies its
// probability; to stay in fp16's range, P is stored as
// p_t (s_t / s_ref) 2^14, s_ref the largest scale so far and at least 2^-100
// (O is rescaled when it grows, as for m), rounded once to fp16's 11 bits.
// bf16: P is carried as a bf16 hi + lo pair (16 bits) against bf16 V.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "paged.cuh"
#include "ptx.cuh"

namespace cpattn {

constexpr int kDecWarps = 8;                     // compute warps
constexpr int kDecThreads = 32 * (kDecWarps + 1);
constexpr int kDecRows = 16;                     // q heads of a row (mma M)
constexpr uint32_t kDecBarrier = 1;              // named barrier of the compute warps
constexpr float kPScale = 16384.f;               // Q8: P is stored times 2^14
constexpr float kMinSref = 7.888609052210118e-31f;  // 2^-100: kPScale / s_ref stays finite

template <int HD, bool Q8>
struct DecodeLayout {
  static constexpr int ESZ = Q8 ? 1 : 2;
  static constexpr int TT = Q8 ? 128 : 64;       // tokens per tile
  static constexpr int BOXW = 128 / ESZ;         // values per 128-byte box row
  static constexpr int NBOX = HD / BOXW;         // column blocks of a tile
  static constexpr int SLOT = TT * HD * ESZ;
  static constexpr int NSLOT = 96 * 1024 / SLOT; // 96 KB of copies in flight per CTA
  static constexpr int WTOK = TT / kDecWarps;    // tokens per warp in Q K^T
  static constexpr int NT = WTOK / 8;            // their n-tiles
  static constexpr int DW = HD / kDecWarps;      // V columns per warp
  static constexpr int P_STRIDE = TT + 8;        // 16-bit values; rows 16 bytes apart mod 128
  static constexpr int Q_STRIDE = HD + 8;
  static constexpr int P_BYTES = kDecRows * P_STRIDE * 2;
  static constexpr int OFF_SCALE = NSLOT * SLOT;
  static constexpr int OFF_P = OFF_SCALE + (Q8 ? NSLOT * TT * 4 : 0);
  static constexpr int OFF_Q = OFF_P + P_BYTES * (Q8 ? 1 : 2);
  static constexpr int OFF_MAX = OFF_Q + kDecRows * Q_STRIDE * 2;  // [16][8] row maxima by warp
  static constexpr int OFF_SUM = OFF_MAX + kDecRows * kDecWarps * 4;
  static constexpr int OFF_SMAX = OFF_SUM + kDecRows * kDecWarps * 4;  // [8] largest V scale by warp
  static constexpr int OFF_QEXP = OFF_SMAX + kDecWarps * 4;            // [16] 2^e of each Q row
  static constexpr int OFF_BAR = OFF_QEXP + kDecRows * 4;
  static constexpr int OFF_BAD = OFF_BAR + 2 * NSLOT * 8;  // [NSLOT] pages of the tile that are absent
  static constexpr int OFF_MISC = OFF_BAD + NSLOT * 4;     // start of the slice, abort flag
  static constexpr int SMEM_BYTES = OFF_MISC + 64;
  static_assert(OFF_BAR % 8 == 0 && OFF_SCALE % 128 == 0 && OFF_P % 16 == 0 && OFF_Q % 16 == 0,
                "shared memory alignment");
  static_assert(2 * (SMEM_BYTES + 1024) <= 228 * 1024, "two CTAs per SM");
};

struct PagedDecodeParams {
  CUtensorMap tm_k;  // [pool rows][HD], box BOXW x 1 x min(page_size, TT)
  CUtensorMap tm_v;
  PagedPool pool;
  const int* lens;            // [num_seqs]; <= 0: no tokens
  const __nv_bfloat16* q;     // [num_seqs][NQ][HD]
  __nv_bfloat16* out;
  float* lse;                 // or null
  float* ws_o;                // [2 * CTAs][16][HD] O of a CTA's first / last row
  float2* ws_ml;              // [2 * CTAs][16] its m and l
  int4* ws_desc;              // [CTAs] (b, kv head * hblocks + block, pieces, 0)
  int* status;
  unsigned long long timeout_ns;
  int pool_rows;              // num_pages * NKV * page_size
  int debug_flags;
  int num_ctas;               // CTAs of the decode kernel
  int num_seqs, nq, group, hblocks;  // hblocks: blocks of 16 q heads per kv head
  float scale_log2;
};

enum : int { kSiteDecFull = 9, kSiteDecEmpty = 10 };  // after the prefill's sites

// ------------------------------------------------------------------ mma.sync
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}

// Shared address of 16-byte chunk `chunk` of row `row` in the column block at
// `base` (rows of 128 bytes, as a 128-byte-swizzled TMA box stores them).
__device__ __forceinline__ uint32_t sw128(uint32_t base, int row, int chunk) {
  return base + row * 128 + ((chunk ^ (row & 7)) << 4);
}

// ------------------------------------------------------------- the slices
// Tile list position: sequence b, row rr = kv head * hblocks + head block, tile.
struct DecodeSpot {
  int b, rr, tile;
};

// Tokens of sequence b, cut to what its table row can name.
__device__ __forceinline__ int decode_len(const PagedDecodeParams& p, int b) {
  const long long room = static_cast<long long>(p.pool.max_pages) << p.pool.page_shift;
  return static_cast<int>(max(0LL, min(static_cast<long long>(__ldg(p.lens + b)), room)));
}

// Whole block (kDecThreads threads): tiles over all rows, and this CTA's slice
// [s0, s1) of them; *spot receives the position of s0 (valid if s0 < s1).
// `active` CTAs share the list, one tile each at least.
template <int TT>
__device__ __forceinline__ long long decode_slice(const PagedDecodeParams& p, int rows_per_seq,
                                                  long long* s0, long long* s1, int* active,
                                                  DecodeSpot* spot) {
  __shared__ long long warp_sum[kDecWarps + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.num_seqs + kDecThreads - 1) / kDecThreads;
  const int b0 = min(p.num_seqs, tid * per), b1 = min(p.num_seqs, b0 + per);
  const long long room = static_cast<long long>(p.pool.max_pages) << p.pool.page_shift;
  long long sum = 0;
  for (int b = b0; b < b1; ++b) {
    sum += (decode_len(p, b) + TT - 1) / TT;
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
  __syncthreads();
  long long base = 0, total = 0;
  for (int w = 0; w <= kDecWarps; ++w) {
    if (w < warp) base += warp_sum[w];
    total += warp_sum[w];
  }
  total *= rows_per_seq;
  *active = static_cast<int>(min(total, static_cast<long long>(gridDim.x)));
  const int c = blockIdx.x;
  *s0 = c < *active ? total * c / *active : 0;
  *s1 = c < *active ? total * (c + 1) / *active : 0;
  long long at = (base + inc - sum) * rows_per_seq;  // list index of sequence b0's first tile
  if (*s0 < *s1 && at <= *s0 && *s0 < at + sum * rows_per_seq) {
    for (int b = b0; b < b1; ++b) {
      const int nt = (decode_len(p, b) + TT - 1) / TT;
      const long long n = static_cast<long long>(nt) * rows_per_seq;
      if (*s0 < at + n) {
        const long long off = *s0 - at;
        spot->b = b;
        spot->rr = static_cast<int>(off / nt);
        spot->tile = static_cast<int>(off % nt);
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  return total;
}

// ------------------------------------------------------------------ kernel
template <int HD, bool Q8>
__global__ void __launch_bounds__(kDecThreads, 2)
    paged_decode_kernel(const __grid_constant__ PagedDecodeParams p) {
  using Ly = DecodeLayout<HD, Q8>;
  constexpr int TT = Ly::TT, NT = Ly::NT, DW = Ly::DW, NSLOT = Ly::NSLOT;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();
  // Swizzled copies need a 1024-byte aligned base (which the launch gives).
  if ((sbase & 1023u) != 0) {
    if (tid == 0 && p.status != nullptr) atomicCAS(p.status, kStatusOk, kStatusLayout);
    if (tid == 0) p.ws_desc[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }
  auto full = [&](int s) { return sbase + Ly::OFF_BAR + 8u * static_cast<uint32_t>(s); };
  auto empty = [&](int s) { return sbase + Ly::OFF_BAR + 8u * static_cast<uint32_t>(NSLOT + s); };
  volatile uint32_t* bad_pages = reinterpret_cast<volatile uint32_t*>(smem + Ly::OFF_BAD);
  DecodeSpot* spot = reinterpret_cast<DecodeSpot*>(smem + Ly::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Ly::OFF_MISC + 32);
  if (tid == 0) {
    for (int s = 0; s < NSLOT; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kDecWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  const int rows_per_seq = p.pool.nkv * p.hblocks;
  long long s0, s1;
  int active;
  const long long total = decode_slice<TT>(p, rows_per_seq, &s0, &s1, &active, spot);
  const BoundedWait wait{abort_flag, p.status, p.timeout_ns, nullptr, 0u, 0};

  // Sequences without tokens: zeros, and an LSE of -infinity.
  for (int b = blockIdx.x; b < p.num_seqs; b += gridDim.x) {
    if (decode_len(p, b) > 0) continue;
    uint4* o = reinterpret_cast<uint4*>(p.out + static_cast<long long>(b) * p.nq * HD);
    for (int i = tid; i < p.nq * (HD / 8); i += kDecThreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
    if (p.lse != nullptr)
      for (int h = tid; h < p.nq; h += kDecThreads)
        p.lse[static_cast<long long>(b) * p.nq + h] = -INFINITY;
  }
  if (s0 >= s1) {
    if (tid == 0) p.ws_desc[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }
  DecodeSpot at = *spot;
  int n = decode_len(p, at.b);
  int nt = (n + TT - 1) / TT;

  if (warp == kDecWarps) {
    // ---------------------------------------------------------- TMA producer
    const int ps = 1 << p.pool.page_shift;
    const int chunk = min(ps, TT);            // tokens per box
    const int chunk_shift = min(p.pool.page_shift, TT == 64 ? 6 : 7);
    const int chunks = TT >> chunk_shift;     // boxes (of each column block) per tile
    if (lane == 0) {
      prefetch_tmap(&p.tm_k);
      prefetch_tmap(&p.tm_v);
    }
    int slot = 0, round = 0;
    uint32_t phase = 0;
    long long issued = 0;
    // Lane i holds the pool row of the tile's i-th box: where it starts, or
    // p.pool_rows (out of range: TMA fills zeros) when it lies behind the last
    // token or its page is absent (bad).
    auto rows_of = [&](const DecodeSpot& s, int len, bool* bad) {
      *bad = false;
      const long long t = static_cast<long long>(s.tile) * TT + (lane << chunk_shift);
      if (lane >= chunks || t >= len) return p.pool_rows;
      const int id = page_id(p.pool, s.b, static_cast<int>(t >> p.pool.page_shift), p.status);
      if (id < 0) {
        *bad = true;
        return p.pool_rows;
      }
      return static_cast<int>(pool_row(p.pool, id, s.rr / p.hblocks, static_cast<int>(t) & (ps - 1)));
    };
    auto load = [&](const CUtensorMap* m, const float* scales, int row, uint32_t bad) {
      bool ok = true;
      if (round > 0) ok = wait(empty(slot), phase ^ 1u, kSiteDecEmpty);
      if (!__all_sync(0xFFFFFFFFu, ok)) return false;
      const uint32_t here = __ballot_sync(0xFFFFFFFFu, lane < chunks && row < p.pool_rows);
      const uint32_t dst = sbase + slot * Ly::SLOT;
      if (lane == 0) {
        bad_pages[slot] = bad;
        mbar_arrive_expect_tx(full(slot),
                              Ly::SLOT + (Q8 ? __popc(here) * (chunk * 4) : 0));
      }
      __syncwarp();
      if (lane < chunks) {
#pragma unroll
        for (int c = 0; c < Ly::NBOX; ++c)
          tma_load_3d(dst + c * (TT * 128) + (lane << chunk_shift) * 128, m, full(slot),
                      c * Ly::BOXW, 0, row);
        if (Q8 && row < p.pool_rows)
          bulk_load(sbase + Ly::OFF_SCALE + slot * (TT * 4) + (lane << chunk_shift) * 4,
                    scales + row, chunk * 4, full(slot));
      }
      if (++slot == NSLOT) {
        slot = 0;
        phase ^= 1u;
        round = 1;
      }
      ++issued;
      return true;
    };
    bool ok = true;
    bool bad;
    int row = rows_of(at, n, &bad);
    for (long long s = s0; ok && s < s1; ++s) {
      // The next tile's pages are looked up before this tile's slots are waited for.
      const int cur = row;
      const uint32_t badm = __ballot_sync(0xFFFFFFFFu, bad);
      if (s + 1 < s1) {
        if (++at.tile == nt) {
          at.tile = 0;
          if (++at.rr == rows_per_seq) {
            at.rr = 0;
            do {
              n = decode_len(p, ++at.b);
            } while (n == 0);
            nt = (n + TT - 1) / TT;
          }
        }
        row = rows_of(at, n, &bad);
      }
      ok = load(&p.tm_k, p.pool.k_scales, cur, badm) && load(&p.tm_v, p.pool.v_scales, cur, badm);
    }
    if (!ok && lane == 0) {
      // Let copies already issued land before this CTA can exit.
      const long long first = issued > NSLOT ? issued - NSLOT : 0;
      for (long long z = first; z < issued; ++z)
        mbar_wait_drain(full(static_cast<int>(z % NSLOT)), static_cast<uint32_t>((z / NSLOT) & 1),
                        200ull * 1000 * 1000);
    }
    return;
  }

  // ------------------------------------------------------------ compute warps
  // A warp whose wait expired (ok = false) waits for no more copies: its loops
  // run to their end on stale data, every warp still meets every barrier, and
  // the status word tells the host.
  bool ok = true;
  bool drop_one = (p.debug_flags & kDebugDropArrive) && blockIdx.x == 0 && tid == 0;
  const int quad = lane & 3, r0 = lane >> 2;      // accumulator rows r0 and r0 + 8
  float* maxs = reinterpret_cast<float*>(smem + Ly::OFF_MAX);
  float* sums = reinterpret_cast<float*>(smem + Ly::OFF_SUM);
  float* smaxs = reinterpret_cast<float*>(smem + Ly::OFF_SMAX);
  float* qexp = reinterpret_cast<float*>(smem + Ly::OFF_QEXP);
  uint16_t* qs = reinterpret_cast<uint16_t*>(smem + Ly::OFF_Q);
  uint32_t* ps32 = reinterpret_cast<uint32_t*>(smem + Ly::OFF_P);
  const uint32_t p_sm = sbase + Ly::OFF_P, q_sm = sbase + Ly::OFF_Q;
  const int chunk_shift = min(p.pool.page_shift, TT == 64 ? 6 : 7);
  const int dim0 = warp * DW;                     // this warp's V columns
  constexpr int NO = DW / 8;                      // their n-tiles
  int slot = 0;
  uint32_t phase = 0;
  auto next_slot = [&]() {
    if (++slot == NSLOT) {
      slot = 0;
      phase ^= 1u;
    }
  };

  long long s = s0;
  while (s < s1) {
    const int g = at.rr / p.hblocks, h0 = g * p.group + (at.rr % p.hblocks) * kDecRows;
    const int heads = min(kDecRows, (g + 1) * p.group - h0);
    const int tile0 = at.tile;
    const int tiles = static_cast<int>(min(static_cast<long long>(nt - tile0), s1 - s));

    // Q of the row into shared memory: warp w stages rows 2w and 2w + 1; bf16
    // as it is, or (Q8) fp16 scaled by a power of two, with the dims of each
    // 16-block in the order in which the e4m3 K fragments come out of ldmatrix.
    bar_sync(kDecBarrier, 32 * kDecWarps);  // the last row's Q and sums are no longer read
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = 2 * warp + j;
      const __nv_bfloat16* src = p.q + (static_cast<long long>(at.b) * p.nq + h0 + r) * HD;
      uint32_t w[HD / 64];
      uint32_t big = 0;
#pragma unroll
      for (int i = 0; i < HD / 64; ++i) {
        w[i] = r < heads ? __ldg(reinterpret_cast<const uint32_t*>(src) + 32 * i + lane) : 0u;
        big = max(big, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
      }
      if constexpr (Q8) {
        big = __reduce_max_sync(0xFFFFFFFFu, big);
        // 2^-e as a float, e the exponent of the row's largest value (a row of
        // zeros or subnormals: 2^126, where the product stays finite).
        const int e = max(static_cast<int>(big >> 7), 1) - 127;
        const float down = e > 126 ? exp2f(-127.f) * (e == 128 ? 0.5f : 1.f) : exp2f(static_cast<float>(-e));
        if (lane == 0) qexp[r] = e > 126 ? exp2f(127.f) * (e == 128 ? 2.f : 1.f) : exp2f(static_cast<float>(e));
#pragma unroll
        for (int i = 0; i < HD / 64; ++i) {
          const int d = 2 * (32 * i + lane);     // dims d, d + 1 (d even)
          const int k = d & 15;                  // dim 4a + 2c -> position 2a + 8c
          const int pos = (d & ~15) + (k >> 2) * 2 + ((k >> 1) & 1) * 8;
          *reinterpret_cast<uint32_t*>(qs + r * Ly::Q_STRIDE + pos) =
              pack_f16x2(__uint_as_float(w[i] << 16) * down,
                         __uint_as_float(w[i] & 0xFFFF0000u) * down);
        }
      } else {
#pragma unroll
        for (int i = 0; i < HD / 64; ++i)
          *reinterpret_cast<uint32_t*>(qs + r * Ly::Q_STRIDE + 2 * (32 * i + lane)) = w[i];
      }
    }
    bar_sync(kDecBarrier, 32 * kDecWarps);
    float sl[2] = {p.scale_log2, p.scale_log2};
    if (Q8) {
      sl[0] *= qexp[r0];
      sl[1] *= qexp[r0 + 8];
    }

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float sref = kMinSref;  // Q8: the largest V scale so far
    float o[NO][4];
#pragma unroll
    for (int i = 0; i < NO; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;

    for (int v = 0; v < tiles; ++v) {
      const int valid = min(TT, n - (tile0 + v) * TT);  // tokens of the tile

      // ---- S = Q K^T for this warp's tokens
      const int kslot = slot;
      if (ok) ok = wait(full(kslot), phase, kSiteDecFull);
      __syncwarp();
      const uint32_t kb = sbase + kslot * Ly::SLOT;
      const uint32_t bad = bad_pages[kslot];
      float c[NT][4], c2[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[t][j] = c2[t][j] = 0.f;
      if constexpr (Q8) {
#pragma unroll
        for (int blk = 0; blk < HD / 64; ++blk) {  // 64 dims: four k16 steps
          uint32_t kr[NT][4];
#pragma unroll
          for (int t = 0; t < NT; ++t)
            ldsm4(kr[t], sw128(kb + (blk >> 1) * (TT * 128), warp * Ly::WTOK + t * 8 + (lane & 7),
                               (blk & 1) * 4 + (lane >> 3)));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t a[4];
            ldsm4(a, q_sm + ((lane & 15) * Ly::Q_STRIDE + (4 * blk + j) * 16 + (lane >> 4) * 8) * 2);
#pragma unroll
            for (int t = 0; t < NT; ++t)
              mma16816<true>((j & 1) ? c2[t] : c[t], a,
                             e4m3x2_to_f16x2(static_cast<uint16_t>(kr[t][j])),
                             e4m3x2_to_f16x2(static_cast<uint16_t>(kr[t][j] >> 16)));
          }
        }
      } else {
#pragma unroll
        for (int blk = 0; blk < HD / 32; ++blk) {  // 32 dims: two k16 steps
          uint32_t kr[4];
          ldsm4(kr, sw128(kb + (blk >> 1) * (TT * 128), warp * Ly::WTOK + (lane & 7),
                          (blk & 1) * 4 + (lane >> 3)));
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t a[4];
            ldsm4(a, q_sm + ((lane & 15) * Ly::Q_STRIDE + (2 * blk + j) * 16 + (lane >> 4) * 8) * 2);
            mma16816<false>(j ? c2[0] : c[0], a, kr[2 * j], kr[2 * j + 1]);
          }
        }
      }
      // Logits in log2 units, by value: what is no token is -infinity.
      float x[NT][4];
      float mx[2] = {-INFINITY, -INFINITY};
      bool seen[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int tok = warp * Ly::WTOK + t * 8 + quad * 2;
        float ks[2] = {1.f, 1.f};
        if (Q8) {
          const float2 f = *reinterpret_cast<const float2*>(smem + Ly::OFF_SCALE +
                                                            kslot * (TT * 4) + tok * 4);
          ks[0] = f.x;
          ks[1] = f.y;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          seen[t][j] = tok + j < valid && !((bad >> (tok >> chunk_shift)) & 1u);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float y = (c[t][2 * i + j] + c2[t][2 * i + j]) * (sl[i] * ks[j]);
            x[t][2 * i + j] = seen[t][j] ? y : -INFINITY;
            mx[i] = fmaxf(mx[i], x[t][2 * i + j]);
          }
        }
      }
      __syncwarp();
      if (lane == 0 && !drop_one) mbar_arrive(empty(kslot));
      drop_one = false;
      next_slot();

      // ---- V's scales of this warp's tokens (with the V tile)
      const int vslot = slot;
      float vs[NT][2];
      float smx = 0.f;
      if (Q8) {
        if (ok) ok = wait(full(vslot), phase, kSiteDecFull);
        __syncwarp();
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int tok = warp * Ly::WTOK + t * 8 + quad * 2;
          const float2 f = *reinterpret_cast<const float2*>(smem + Ly::OFF_SCALE +
                                                            vslot * (TT * 4) + tok * 4);
          vs[t][0] = f.x;
          vs[t][1] = f.y;
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (seen[t][j]) smx = fmaxf(smx, fabsf(vs[t][j]));
        }
      }

      // ---- row maxima over the tile
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xFFFFFFFFu, mx[0], d));
        mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xFFFFFFFFu, mx[1], d));
        if (Q8) smx = fmaxf(smx, __shfl_xor_sync(0xFFFFFFFFu, smx, d));
      }
      if (quad == 0) {
        maxs[r0 * kDecWarps + warp] = mx[0];
        maxs[(r0 + 8) * kDecWarps + warp] = mx[1];
        if (Q8 && lane == 0) smaxs[warp] = smx;
      }
      bar_sync(kDecBarrier, 32 * kDecWarps);
      float alpha[2];
      float mref[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 f0 = *reinterpret_cast<const float4*>(maxs + (r0 + 8 * i) * kDecWarps);
        const float4 f1 = *reinterpret_cast<const float4*>(maxs + (r0 + 8 * i) * kDecWarps + 4);
        const float mn = fmaxf(m[i], fmaxf(fmaxf(fmaxf(f0.x, f0.y), fmaxf(f0.z, f0.w)),
                                           fmaxf(fmaxf(f1.x, f1.y), fmaxf(f1.z, f1.w))));
        mref[i] = mn == -INFINITY ? 0.f : mn;
        alpha[i] = ex2_approx(m[i] - mref[i]);
        m[i] = mn;
        l[i] *= alpha[i];
      }
      float pscale = 1.f;
      if (Q8) {
        const float4 f0 = *reinterpret_cast<const float4*>(smaxs);
        const float4 f1 = *reinterpret_cast<const float4*>(smaxs + 4);
        const float sn = fmaxf(sref, fmaxf(fmaxf(fmaxf(f0.x, f0.y), fmaxf(f0.z, f0.w)),
                                           fmaxf(fmaxf(f1.x, f1.y), fmaxf(f1.z, f1.w))));
        alpha[0] *= sref / sn;
        alpha[1] *= sref / sn;
        sref = sn;
        pscale = kPScale / sn;
      }

      // ---- P: probabilities of this warp's tokens, to shared memory
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int tok = warp * Ly::WTOK + t * 8 + quad * 2;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float e0 = ex2_approx(x[t][2 * i] - mref[i]);
          const float e1 = ex2_approx(x[t][2 * i + 1] - mref[i]);
          l[i] += e0 + e1;
          uint32_t* dst = ps32 + ((r0 + 8 * i) * Ly::P_STRIDE + tok) / 2;
          if constexpr (Q8) {
            // s_t / s_ref first: a scale may be far below s_ref, never above it.
            *dst = pack_f16x2(seen[t][0] ? e0 * (vs[t][0] * pscale) : 0.f,
                              seen[t][1] ? e1 * (vs[t][1] * pscale) : 0.f);
          } else {
            const uint32_t hi = pack_bf16x2(e0, e1);
            *dst = hi;
            dst[Ly::P_BYTES / 4] = pack_bf16x2(e0 - __uint_as_float(hi << 16),
                                               e1 - __uint_as_float(hi & 0xFFFF0000u));
          }
        }
      }
#pragma unroll
      for (int i = 0; i < NO; ++i) {
        o[i][0] *= alpha[0];
        o[i][1] *= alpha[0];
        o[i][2] *= alpha[1];
        o[i][3] *= alpha[1];
      }
      bar_sync(kDecBarrier, 32 * kDecWarps);

      // ---- O += P V for this warp's columns
      if (!Q8) {
        if (ok) ok = wait(full(vslot), phase, kSiteDecFull);
        __syncwarp();
      }
      const uint32_t vb = sbase + vslot * Ly::SLOT + (dim0 / Ly::BOXW) * (TT * 128);
      const int ch0 = (dim0 % Ly::BOXW) * Ly::ESZ / 16;
      if (valid < TT) {
        // Slots behind the last token may hold anything; 0 * NaN must not
        // reach O.  Each warp clears its own columns.
        constexpr int CH = DW * Ly::ESZ / 16;
        for (int i = lane; i < (TT - valid) * CH; i += 32)
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                           sw128(vb, valid + i / CH, ch0 + i % CH)),
                       "r"(0)
                       : "memory");
        __syncwarp();
      }
      if constexpr (Q8) {
#pragma unroll
        for (int kt = 0; kt < TT / 32; ++kt) {  // 32 tokens: two k16 steps
          uint32_t a0[4], a1[4];
          const uint32_t pa = p_sm + ((lane & 15) * Ly::P_STRIDE + kt * 32 + (lane >> 4) * 8) * 2;
          ldsm4(a0, pa);
          ldsm4(a1, pa + 32);
#pragma unroll
          for (int ch = 0; ch < DW / 16; ++ch) {
            uint32_t vr[4];
            ldsm4_t(vr, sw128(vb, kt * 32 + lane, ch0 + ch));
            // Each register holds two tokens x two dims; regrouped by dim.
#pragma unroll
            for (int j = 0; j < 4; ++j) vr[j] = __byte_perm(vr[j], 0u, 0x3120);
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // even dims, odd dims
              const int sh = 16 * half;
              mma16816<true>(o[2 * ch + half], a0, e4m3x2_to_f16x2(static_cast<uint16_t>(vr[0] >> sh)),
                             e4m3x2_to_f16x2(static_cast<uint16_t>(vr[1] >> sh)));
              mma16816<true>(o[2 * ch + half], a1, e4m3x2_to_f16x2(static_cast<uint16_t>(vr[2] >> sh)),
                             e4m3x2_to_f16x2(static_cast<uint16_t>(vr[3] >> sh)));
            }
          }
        }
      } else {
#pragma unroll
        for (int kt = 0; kt < TT / 16; ++kt) {
          uint32_t hi[4], lo[4];
          const uint32_t pa = p_sm + ((lane & 15) * Ly::P_STRIDE + kt * 16 + (lane >> 4) * 8) * 2;
          ldsm4(hi, pa);
          ldsm4(lo, pa + Ly::P_BYTES);
#pragma unroll
          for (int ch = 0; ch < NO; ch += 2) {
            uint32_t vr[4];
            ldsm4_t(vr, sw128(vb, kt * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), ch0 + ch + (lane >> 4)));
            mma16816<false>(o[ch], hi, vr[0], vr[1]);
            mma16816<false>(o[ch + 1], hi, vr[2], vr[3]);
            mma16816<false>(o[ch], lo, vr[0], vr[1]);
            mma16816<false>(o[ch + 1], lo, vr[2], vr[3]);
          }
        }
      }
      // Cleared slots: these writes come before the copy that reuses the slot.
      if (valid < TT) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(vslot));
      next_slot();
    }

    // ---- the row's (or piece's) end: l over all tokens, then O
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], d);
      if (quad == 0) sums[(r0 + 8 * i) * kDecWarps + warp] = l[i];
    }
    bar_sync(kDecBarrier, 32 * kDecWarps);
    const bool whole = tile0 == 0 && tiles == nt;
    const int piece = 2 * blockIdx.x + (tile0 == 0 ? 1 : 0);
    const float oscale = Q8 ? sref * (1.f / kPScale) : 1.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + 8 * i;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) sum += sums[r * kDecWarps + w];
      if (r >= heads) continue;
      const long long orow = static_cast<long long>(at.b) * p.nq + h0 + r;
      // l = 0: every page of the row was absent.
      const float f = whole ? (sum == 0.f ? 0.f : oscale / sum) : oscale;
      float y[DW / 4];  // this thread's columns: Q8 runs of four, else of two
#pragma unroll
      for (int k = 0; k < NO; ++k) {
        y[2 * k] = o[k][2 * i] * f;
        y[2 * k + 1] = o[k][2 * i + 1] * f;
      }
#pragma unroll
      for (int k = 0; k < NO; k += 2) {
        if constexpr (Q8) {
          // n-tiles k, k + 1: even and odd dims of a 16-column chunk
          const int d = dim0 + 8 * k + 4 * quad;
          const float e[4] = {y[2 * k], y[2 * k + 2], y[2 * k + 1], y[2 * k + 3]};
          if (whole)
            *reinterpret_cast<uint2*>(p.out + orow * HD + d) =
                make_uint2(pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]));
          else
            *reinterpret_cast<float4*>(p.ws_o + (static_cast<long long>(piece) * kDecRows + r) * HD + d) =
                make_float4(e[0], e[1], e[2], e[3]);
        } else {
#pragma unroll
          for (int kk = k; kk < k + 2; ++kk) {
            const int d = dim0 + 8 * kk + 2 * quad;
            if (whole)
              *reinterpret_cast<uint32_t*>(p.out + orow * HD + d) = pack_bf16x2(y[2 * kk], y[2 * kk + 1]);
            else
              *reinterpret_cast<float2*>(p.ws_o + (static_cast<long long>(piece) * kDecRows + r) * HD + d) =
                  make_float2(y[2 * kk], y[2 * kk + 1]);
          }
        }
      }
      if (warp == 0 && quad == 0) {
        if (!whole)
          p.ws_ml[piece * kDecRows + r] = make_float2(m[i], sum);
        else if (p.lse != nullptr)
          p.lse[orow] = sum == 0.f ? -INFINITY : (m[i] + __log2f(sum)) * 0.69314718055994531f;
      }
    }
    s += tiles;
    if (s >= s1 && tid == 0) {
      // The CTA whose slice begins a row that others continue describes it.
      int4 d = make_int4(0, 0, 0, 0);
      if (tile0 == 0 && tiles < nt) {
        const long long last = s - tiles + nt - 1;  // list index of the row's last tile
        const long long cta = ((last + 1) * active - 1) / total;
        d = make_int4(at.b, at.rr, static_cast<int>(cta) - static_cast<int>(blockIdx.x) + 1, 0);
      }
      p.ws_desc[blockIdx.x] = d;
    }
    if (s < s1) {
      at.tile = 0;
      if (++at.rr == rows_per_seq) {
        at.rr = 0;
        do {
          n = decode_len(p, ++at.b);
        } while (n == 0);
        nt = (n + TT - 1) / TT;
      }
    }
  }
}

// Joins the pieces of the rows that were cut.  Block (x, y): row x of the
// batch when there are at most as many rows as CTAs, found by a search of
// their descriptions, else the row that CTA x began; q heads y, y + gridDim.y,
// ... of it.  Most blocks of a large batch find nothing to do.  A programmatic
// dependent of the decode kernel.  Thread (j, y): output elements 4j .. 4j+3
// over the pieces y, y + GROUPS, ..., summed over y in shared memory: a long
// row has a piece from every CTA, and their loads should all be in flight.
constexpr int kJoinThreads = 512;
constexpr int kJoinMaxPieces = 1024;  // checked by the host against the CTAs of a launch

template <int HD>
__global__ void __launch_bounds__(kJoinThreads)
    paged_join_kernel(const __grid_constant__ PagedDecodeParams p) {
  constexpr int GROUPS = kJoinThreads / (HD / 4);
  __shared__ float4 part[GROUPS][HD / 4];
  __shared__ float weight[kJoinMaxPieces];
  __shared__ float stats[2];
  __shared__ int owner;
  const int tid = threadIdx.x, j = tid % (HD / 4), y = tid / (HD / 4);
  const int rows_per_seq = p.pool.nkv * p.hblocks;
  const bool by_row = static_cast<long long>(p.num_seqs) * rows_per_seq <= p.num_ctas;
  if (tid == 0) owner = by_row ? -1 : static_cast<int>(blockIdx.x);
  __syncthreads();
  griddep_wait();
  if (by_row) {
    for (int c = tid; c < p.num_ctas; c += kJoinThreads) {
      const int4 d = p.ws_desc[c];
      if (d.z > 0 && d.x * rows_per_seq + d.y == static_cast<int>(blockIdx.x)) owner = c;
    }
    __syncthreads();
    if (owner < 0) return;
  }
  const int cta = owner;
  const int4 d = p.ws_desc[cta];
  const int pieces = d.z;
  if (pieces == 0) return;
  const int g = d.y / p.hblocks, h0 = g * p.group + (d.y % p.hblocks) * kDecRows;
  const int heads = min(kDecRows, (g + 1) * p.group - h0);
  // Piece 0 is CTA cta's last row, the others the first rows of those behind it.
  auto slot = [&](int i) { return 2 * (cta + i) + (i == 0 ? 1 : 0); };
  for (int r = blockIdx.y; r < heads; r += gridDim.y) {
    if (tid < 32) {
      float m = -INFINITY, l = 0.f;
      for (int i = tid; i < pieces; i += 32) m = fmaxf(m, p.ws_ml[slot(i) * kDecRows + r].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const float mref = m == -INFINITY ? 0.f : m;
      for (int i = tid; i < pieces; i += 32) {
        const float2 ml = p.ws_ml[slot(i) * kDecRows + r];
        const float w = ex2_approx(ml.x - mref);
        weight[i] = w;
        l = fmaf(w, ml.y, l);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
      if (tid == 0) {
        stats[0] = m;
        stats[1] = l;
      }
    }
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = y; i < pieces; i += GROUPS) {
      const float4 o = *reinterpret_cast<const float4*>(
          p.ws_o + (static_cast<long long>(slot(i)) * kDecRows + r) * HD + 4 * j);
      const float w = weight[i];
      acc.x = fmaf(w, o.x, acc.x);
      acc.y = fmaf(w, o.y, acc.y);
      acc.z = fmaf(w, o.z, acc.z);
      acc.w = fmaf(w, o.w, acc.w);
    }
    part[y][j] = acc;
    __syncthreads();
    if (y == 0) {
#pragma unroll
      for (int k = 1; k < GROUPS; ++k) {
        acc.x += part[k][j].x;
        acc.y += part[k][j].y;
        acc.z += part[k][j].z;
        acc.w += part[k][j].w;
      }
      const float m = stats[0], l = stats[1];
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const long long orow = static_cast<long long>(d.x) * p.nq + h0 + r;
      *reinterpret_cast<uint2*>(p.out + orow * HD + 4 * j) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      if (j == 0 && p.lse != nullptr)
        p.lse[orow] = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
    }
    __syncthreads();  // weight, stats and part are reused by the next head
  }
}

}  // namespace cpattn
