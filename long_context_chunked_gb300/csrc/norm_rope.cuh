// Norms of queries and keys for each head, with the position rotation in the
// same pass, and the same with the new tokens' K and V going into their pages:
//   y = x / sqrt(mean_d x_d^2 + eps) w_d          (per head; without w: y = x)
//   (a, b) -> (a cos - b sin, b cos + a sin)       for each pair of the first ROT dims
// with the angle position * inv_freq of the pair, cos and sin times `scale`.
// Pairs are dims (i, i + ROT/2), or neighbours (2 i, 2 i + 1).
//
// Angles.  A pair's frequency is kept as the whole number round(2^64 inv_freq /
// 2 pi): turns per position in 64-bit fixed point.  Its product with the position,
// modulo 2^64, is the fraction of a turn, without any rounding of its own: the
// reduction that fp32 cannot make for far positions is the integer's overflow.
// Its upper 32 bits are an eighth turn at most from a quarter turn, whose number
// turns (cos, sin) of the rest, x radians at most pi / 4: from their Taylor series
// to x^9 and x^8, off by x^11 / 11! < 1.8e-9 and x^10 / 10! < 2.5e-8.
//
// HBM-bound if it takes few enough instructions: Q and K are read and written once,
// 8 flops a value.  A head's row lies in HD / 8 lanes, eight values each, so that
// both values of a pair are in one lane and a norm is one sum over those lanes.
// With the weights multiplied into cos and sin once for a row's heads,
//   y_a = r (x_a (w_a cos) - x_b (w_b sin)),  y_b = r (x_b (w_b cos) + x_a (w_a sin)),
// r = 1 / sqrt(mean + eps), a head takes four products of pairs of values in
// packed fp32 instructions, and r.
//   17421 rows of 32 + 4 heads of 128: 51.1 us for 321 MB (6.3 TB/s, 92 % of a copy's);
// 20161 rows of 32 + 2 of 256: 107 us (702 MB, 6.6 TB/s), with K and V going to bf16
// pages 113.8 (743 MB, 6.5), to e4m3 pages 115.3, to e2m1 pages 115.1 (712 MB); the first
// case to e4m3 pages 60.8 us for 340 MB (5.6 TB/s, 64 % of the issue slots: what each unit
// of K and V needs for its scale, two reductions and a division, is not hidden whole),
// to e2m1 pages 56.6 (331 MB, 5.9 TB/s).  7 rows: 3.1 and 3.5 us as nodes of a graph, to
// e2m1 pages 3.8.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "paged.cuh"
#include "ptx.cuh"

namespace cpattn {

struct NormRopeParams {
  PagedPool pool;                  // (append only)
  const __nv_bfloat16* q;          // row r at r * q_stride, NQ heads of HD
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;          // (append only)
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_out;            // (dense only)
  const void* q_weight;            // [HD] bf16 or fp32, or null
  const void* k_weight;
  const unsigned long long* steps; // [rot / 2] turns per position, times 2^64
  const int* positions;            // [rows]; < 0: the row is skipped
  const int* slots;                // [rows] page * page_size + slot; < 0: not stored
  long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;  // elements
  int* status;
  float eps, scale;
  int weight_f32;
  int rows, nq, nkv, rot, neighbours;
  int batch;                       // units per batch: 1 or kNormBatch
};

// Where a lane's two runs of four dims begin: `l` of a head's HD / 8 lanes.
__device__ __forceinline__ void lane_dims(int l, int rot, bool neighbours, int* d0, int* d1) {
  if (!neighbours && l < rot / 8) {
    *d0 = 4 * l;
    *d1 = rot / 2 + 4 * l;
  } else {
    *d0 = 8 * l;
    *d1 = 8 * l + 4;
  }
}

// A lane's eight values: the first and second values of its four pairs, two and
// two.  Its runs of four dims hold them as (a0 a1 a2 a3), (b0 b1 b2 b3), or, where
// neighbours are pairs, (a0 b0 a2 b2), (a1 b1 a3 b3): one is made of the other by
// regrouping the runs' first words, and the second.
struct Pairs {
  f32x2 a[2], b[2];
};
__device__ __forceinline__ void regroup(uint2& r0, uint2& r1) {
  const uint2 s0 = r0, s1 = r1;
  r0 = make_uint2(__byte_perm(s0.x, s1.x, 0x5410), __byte_perm(s0.y, s1.y, 0x5410));
  r1 = make_uint2(__byte_perm(s0.x, s1.x, 0x7632), __byte_perm(s0.y, s1.y, 0x7632));
}
// Factors of a row's heads: w_a cos, -w_b sin, w_b cos, w_a sin, of pairs 0, 1 and 2, 3.
struct Factors {
  f32x2 ac[2], bs[2], bc[2], as[2];
};

// (r0, r1: the lane's two runs of four bf16 values; turn: they turn.  What does not is
// a product with its own factor alone: 0 times the other value would be NaN where that
// is infinite.)
template <int HD, bool NEIGHBOURS>
__device__ __forceinline__ Pairs norm_and_turn(uint2 r0, uint2 r1, bool norm, float eps, bool turn,
                                               const Factors& f) {
  if (NEIGHBOURS) regroup(r0, r1);
  const Pairs x = {{bf16x2_to_f32x2(r0.x), bf16x2_to_f32x2(r0.y)}, {bf16x2_to_f32x2(r1.x), bf16x2_to_f32x2(r1.y)}};
  f32x2 s2 = mul2(x.a[0], x.a[0]);
  s2 = fma2(x.a[1], x.a[1], s2);
  s2 = fma2(x.b[0], x.b[0], s2);
  s2 = fma2(x.b[1], x.b[1], s2);
  const float2 s = split(s2);
  float sum = s.x + s.y;
#pragma unroll
  for (int o = HD / 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  const float r = norm ? rsqrtf(fmaf(sum, 1.f / HD, eps)) : 1.f;
  const f32x2 r2 = pair_of(r, r);
  Pairs y;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    y.a[i] = mul2(x.a[i], f.ac[i]);
    y.b[i] = mul2(x.b[i], f.bc[i]);
  }
  if (turn) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      y.a[i] = fma2(x.b[i], f.bs[i], y.a[i]);
      y.b[i] = fma2(x.a[i], f.as[i], y.b[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    y.a[i] = mul2(y.a[i], r2);
    y.b[i] = mul2(y.b[i], r2);
  }
  return y;
}
// Rounded to bf16, as the lane's runs.
template <bool NEIGHBOURS>
__device__ __forceinline__ void as_runs(const Pairs& y, uint2& r0, uint2& r1) {
  const float2 a0 = split(y.a[0]), a1 = split(y.a[1]), b0 = split(y.b[0]), b1 = split(y.b[1]);
  r0 = make_uint2(pack_bf16x2(a0.x, a0.y), pack_bf16x2(a1.x, a1.y));
  r1 = make_uint2(pack_bf16x2(b0.x, b0.y), pack_bf16x2(b1.x, b1.y));
  if (NEIGHBOURS) regroup(r0, r1);
}
// The same as fp32, dims d0 .. d0 + 3 and d1 .. d1 + 3.
template <bool NEIGHBOURS>
__device__ __forceinline__ void as_values(const Pairs& y, float (&x)[8]) {
  const float2 a0 = split(y.a[0]), a1 = split(y.a[1]), b0 = split(y.b[0]), b1 = split(y.b[1]);
  x[0] = a0.x;
  x[1] = NEIGHBOURS ? b0.x : a0.y;
  x[2] = a1.x;
  x[3] = NEIGHBOURS ? b1.x : a1.y;
  x[4] = NEIGHBOURS ? a0.y : b0.x;
  x[5] = b0.y;
  x[6] = NEIGHBOURS ? a1.y : b1.x;
  x[7] = b1.y;
}

// cos and sin of two angles, given in turns times 2^32 (modulo 2^32), times `scale`.
__device__ __forceinline__ void cos_sin(uint32_t t0, uint32_t t1, float scale, f32x2* cs, f32x2* sn) {
  const uint32_t q0 = t0 + 0x20000000u, q1 = t1 + 0x20000000u;  // quarters: the upper two bits
  // 2 pi / 2^32, and what is left of it in fp32.
  constexpr double kTurn = 6.283185307179586 / 4294967296.;
  constexpr float kUnit = static_cast<float>(kTurn), kRest = static_cast<float>(kTurn - kUnit);
  auto both = [](float v) { return pair_of(v, v); };
  const f32x2 n = pair_of(static_cast<float>(static_cast<int>(t0 - (q0 & 0xC0000000u))),
                          static_cast<float>(static_cast<int>(t1 - (q1 & 0xC0000000u))));
  const f32x2 x = fma2(n, both(kUnit), mul2(n, both(kRest)));
  const f32x2 z = mul2(x, x);
  f32x2 s = fma2(z, both(1.f / 362880.f), both(-1.f / 5040.f));
  s = fma2(z, s, both(1.f / 120.f));
  s = fma2(z, s, both(-1.f / 6.f));
  s = fma2(mul2(z, x), s, x);
  f32x2 c = fma2(z, both(1.f / 40320.f), both(-1.f / 720.f));
  c = fma2(z, c, both(1.f / 24.f));
  c = fma2(z, c, both(-0.5f));
  c = fma2(z, c, both(1.f));
  const float2 fs = split(s), fc = split(c);
  // Quarter 0: (c, s), 1: (-s, c), 2: (-c, -s), 3: (s, -c).
  auto turn = [&](uint32_t q, float a, float b, float* oc, float* os) {
    const bool odd = (q & 0x40000000u) != 0u;
    const float u = odd ? b : a, v = odd ? a : b;
    *oc = __uint_as_float(__float_as_uint(u) ^ ((q + 0x40000000u) & 0x80000000u)) * scale;
    *os = __uint_as_float(__float_as_uint(v) ^ (q & 0x80000000u)) * scale;
  };
  float c0, c1, s0, s1;
  turn(q0, fc.x, fs.x, &c0, &s0);
  turn(q1, fc.y, fs.y, &c1, &s1);
  *cs = pair_of(c0, c1);
  *sn = pair_of(s0, s1);
}

// Work split: a unit is 512 bytes of a row (a head of 256, two of 128), a batch up
// to kNormBatch units of one kind (Q, K or V), and each of the grid's warps takes an
// equal, contiguous slice of the list of all rows' batches: a row, of many rows, in
// blocks that follow one another, or a share of all of it in resident blocks (the
// host's choice).  Its next batches are copied
// to shared memory while it works on one.  What all batches of a row and kind
// share (pointers, factors) is made once for them: instructions, not memory, bound
// this kernel first (17421 rows, 32 + 4 heads of 128: 520 of them per batch, 57 us,
// when every batch looked for its place by itself).
constexpr int kNormThreads = 256;
constexpr int kNormBatch = 4;
constexpr int kNormSide = 2;    // units whose arithmetic is in flight together
constexpr int kNormBlocks = 3;  // per SM
constexpr int kNormSlots = 3;   // batches of a warp in flight, or being read

// Shared memory: the slots; for each warp a row's cos and sin, a lane's eight values
// together, and (e2m1) a K unit on its way from the rotation's order to that of the
// pages; the weights, Q's and K's; the steps.
__host__ __device__ constexpr int norm_off_turn(int fmt) {
  return kNormThreads / 32 * (kNormSlots * kNormBatch * 512);
}
__host__ __device__ constexpr int norm_off_weights(int fmt) {
  return norm_off_turn(fmt) + kNormThreads / 32 * (fmt == kE2m1 ? 2048 : 1024);
}
__host__ __device__ constexpr int norm_rope_smem(int fmt) { return norm_off_weights(fmt) + 2048 + 1024; }

__device__ __forceinline__ uint32_t magnitude(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(x[j]) & 0x7FFFFFFFu);
  return m;
}

// FMT: the pages' format, or -1: K goes to k_out.  NEIGHBOURS: pairs (2 i, 2 i + 1).
template <int HD, bool NEIGHBOURS, int FMT>
__global__ void __launch_bounds__(kNormThreads, kNormBlocks)
    norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr bool APPEND = FMT >= 0;
  constexpr int LANES = HD / 8, PER = 32 / LANES;  // lanes of a head, heads of a unit
  constexpr int WARPS = kNormThreads / 32, SLOT = kNormBatch * 512, SLOTS = kNormSlots;
  constexpr int KINDS = APPEND ? 3 : 2;            // Q, K, V
  extern __shared__ __align__(1024) uint8_t smem[];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % LANES, sub = lane / LANES;
  const bool turn = l < p.rot / 8;
  int d0, d1;
  lane_dims(l, p.rot, NEIGHBOURS, &d0, &d1);

  // The list: bq batches of Q, bk of K and (append) bk of V for each row.
  const int step = p.batch * PER;  // heads of a batch
  const int bq = (p.nq + step - 1) / step, bk = (p.nkv + step - 1) / step;
  const int per_row = bq + (KINDS - 1) * bk;
  const long long total = static_cast<long long>(p.rows) * per_row;
  const int w = blockIdx.x * WARPS + warp, ws = gridDim.x * WARPS;
  const long long t0 = total * w / ws;
  const int mine = static_cast<int>(total * (w + 1) / ws - t0);  // batches of this warp
  struct Segment {  // batches of one row and kind, from the `first`
    int row, kind, first, left;
  };
  auto sized = [&](Segment& s) { s.left = (s.kind == 0 ? bq : bk) - s.first; };
  auto next = [&](Segment& s) {
    s.first = 0;
    if (++s.kind == KINDS) {
      s.kind = 0;
      ++s.row;
    }
    sized(s);
  };
  Segment at = {static_cast<int>(t0 / per_row), 0, static_cast<int>(t0 % per_row), 0};
  while (at.first >= (at.kind == 0 ? bq : bk)) at.first -= at.kind++ == 0 ? bq : bk;
  sized(at);

  // ------------------------------------------------- the copies, ahead of the work
  const uint32_t slots_at = smem_u32(smem + warp * (SLOTS * SLOT)) + 16 * lane;
  Segment ahead = at;
  const __nv_bfloat16* src = nullptr;  // this lane's 16 bytes of the next batch
  int src_heads = 0, to_copy = mine, slot_in = 0;
  auto source = [&]() {
    src = (ahead.kind == 0   ? p.q + ahead.row * p.q_stride
           : ahead.kind == 1 ? p.k + ahead.row * p.k_stride
                             : p.v + ahead.row * p.v_stride) +
          static_cast<long long>(ahead.first) * (step * HD) + 8 * lane;
    src_heads = (ahead.kind == 0 ? p.nq : p.nkv) - ahead.first * step - sub;
  };
  source();
  auto copy_batch = [&]() {
    if (to_copy > 0) {
      const int heads = min(src_heads, step);
#pragma unroll
      for (int i = 0; i < kNormBatch; ++i)
        if (i * PER < heads) copy16_async(slots_at + slot_in + i * 512, src + i * (PER * HD));
      slot_in = slot_in == (SLOTS - 1) * SLOT ? 0 : slot_in + SLOT;
      src += step * HD;
      src_heads -= step;
      --to_copy;
      if (--ahead.left == 0) {
        next(ahead);
        if (to_copy > 0) source();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < SLOTS - 1; ++i) copy_batch();

  // The next row's position and slot, loaded a row ahead.
  int pos = -1, slot = -1;
  auto load_place = [&](int row) {
    if (row >= p.rows) return;
    pos = load_now(p.positions + row);
    if (APPEND) slot = load_now(p.slots + row);
  };
  load_place(at.row);
  float4* turns = reinterpret_cast<float4*>(smem + norm_off_turn(FMT) + warp * 1024) + 2 * lane;
  float* weights = reinterpret_cast<float*>(smem + norm_off_weights(FMT));
  unsigned long long* steps = reinterpret_cast<unsigned long long*>(smem + norm_off_weights(FMT) + 2048);
  for (int i = threadIdx.x; i < p.rot / 2; i += kNormThreads) steps[i] = load_now(p.steps + i);
  for (int i = threadIdx.x; i < 2 * HD; i += kNormThreads) {
    const void* from = i < HD ? p.q_weight : p.k_weight;
    const int d = i & (HD - 1);
    weights[i] = from == nullptr    ? 1.f
                 : p.weight_f32 != 0 ? load_now(static_cast<const float*>(from) + d)
                                     : __bfloat162float(load_now(static_cast<const __nv_bfloat16*>(from) + d));
  }
  __syncthreads();

  // First dims of the pairs' values, in pairs j = 0 .. 3.
  auto dim_of = [&](int j, bool second) {
    return NEIGHBOURS ? ((j & 1) ? d1 : d0) + 2 * (j >> 1) + (second ? 1 : 0) : (second ? d1 : d0) + j;
  };
  int row = -1, slot_out = 0, left = mine;
  bool live = false;
  long long page_row = -1;  // (append) of the row's place, kv head 0; -1: not stored
  const uint8_t* slots = smem + warp * (SLOTS * SLOT);
  // The next batch of the warp: waits for it, and sends for one more.
  auto take = [&]() {
    copy_batch();
    asm volatile("cp.async.wait_group %0;" ::"n"(SLOTS - 1) : "memory");
    __syncwarp();
    const uint8_t* batch = slots + slot_out;
    slot_out = slot_out == (SLOTS - 1) * SLOT ? 0 : slot_out + SLOT;
    return batch;
  };
#pragma unroll 1
  while (left > 0) {
    if (at.row != row) {
      row = at.row;
      live = pos >= 0;
      page_row = -1;
      if (APPEND && live && slot >= 0) {
        if (slot < p.pool.num_pages << p.pool.page_shift)
          page_row = pool_row(p.pool, slot >> p.pool.page_shift, 0, slot & ((1 << p.pool.page_shift) - 1));
        else if (lane == 0 && p.status != nullptr)
          atomicCAS(p.status, kStatusOk, kStatusPage);
      }
      // (Pair j is that of dim d0 + j, or of dims d0, d1, d0 + 2 and d1 + 2; what does
      // not turn: 1 and 0.)
      uint32_t part[4] = {0u, 0u, 0u, 0u};
      if (turn) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          part[j] = static_cast<uint32_t>((steps[4 * l + (NEIGHBOURS ? ((j & 1) << 1) + (j >> 1) : j)] *
                                           static_cast<unsigned long long>(pos)) >> 32);
      }
      f32x2 c[2], s[2];
      const float scale = turn ? p.scale : 1.f;
      cos_sin(part[0], part[1], scale, &c[0], &s[0]);
      cos_sin(part[2], part[3], scale, &c[1], &s[1]);
      const float2 c0 = split(c[0]), c1 = split(c[1]), s0 = split(s[0]), s1 = split(s[1]);
      turns[0] = make_float4(c0.x, c0.y, c1.x, c1.y);
      turns[1] = make_float4(s0.x, s0.y, s1.x, s1.y);
      load_place(row + 1);
    }
    const int kind = at.kind, batches = min(at.left, left);
    int h0 = at.first * step + sub;        // unit i of the next batch: head h0 + i PER
    int heads = (kind == 0 ? p.nq : p.nkv) - h0;  // from there on
    left -= batches;
    at.left -= batches;
    if (at.left == 0) next(at);
    if (!live || (kind != 0 && APPEND && page_row < 0)) {
#pragma unroll 1
      for (int b = 0; b < batches; ++b) take();
      continue;
    }
    const long long head_rows = 1LL << p.pool.page_shift;  // pool rows from a kv head to the next
    if (kind == 2) {
      if constexpr (APPEND) {
        long long to = page_row + h0 * head_rows;
#pragma unroll 1
        for (int b = 0; b < batches; ++b, heads -= step, to += step * head_rows) {
          const uint8_t* batch = take();
#pragma unroll
          for (int i = 0; i < kNormBatch; ++i) {
            if (i >= p.batch || i * PER >= heads + sub) break;
            const uint4 v = *reinterpret_cast<const uint4*>(batch + i * 512 + 16 * lane);
            PackedRow<FMT> y;
            if constexpr (FMT == kBf16) {
              y.x = v;
            } else {
              float x[8];
              bf16x8_to_f32x8(v, x);
              quantise<HD>(x, amax_bits(v) << 16, y);
            }
            if (i * PER < heads) store_row<HD>(p.pool, false, to + i * PER * head_rows, l, y);
          }
          __syncwarp();  // the slot has been read
        }
      }
      continue;
    }
    // Q or K.
    const bool norm = (kind == 0 ? p.q_weight : p.k_weight) != nullptr;
    Factors f;
    {
      const float* wt = weights + kind * HD;
      const float4 c4 = turns[0], s4 = turns[1];
      const float cs[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const f32x2 c = pair_of(cs[2 * i], cs[2 * i + 1]), s = pair_of(sn[2 * i], sn[2 * i + 1]);
        const f32x2 wa = pair_of(wt[dim_of(2 * i, false)], wt[dim_of(2 * i + 1, false)]);
        const f32x2 wb = pair_of(wt[dim_of(2 * i, true)], wt[dim_of(2 * i + 1, true)]);
        f.ac[i] = mul2(wa, c);
        f.as[i] = mul2(wa, s);
        f.bc[i] = mul2(wb, c);
        f.bs[i] = mul2(mul2(wb, s), pair_of(-1.f, -1.f));
      }
    }
    const int run0 = sub * (2 * HD) + 2 * d0, run1 = sub * (2 * HD) + 2 * d1;
    auto turned = [&](const uint8_t* unit) {
      return norm_and_turn<HD, NEIGHBOURS>(*reinterpret_cast<const uint2*>(unit + run0),
                                           *reinterpret_cast<const uint2*>(unit + run1), norm, p.eps, turn, f);
    };
    if (FMT > 0 && kind == 1) {
      if constexpr (FMT > 0) {
        // K into quantised pages.
        long long to = page_row + h0 * head_rows;
#pragma unroll 1
        for (int b = 0; b < batches; ++b, heads -= step, to += step * head_rows) {
          const uint8_t* batch = take();
#pragma unroll(FMT == kE4m3 ? kNormBatch : 1)
          for (int i = 0; i < kNormBatch; ++i) {
            if (i >= p.batch || i * PER >= heads + sub) break;
            float x[8];
            as_values<NEIGHBOURS>(turned(batch + i * 512), x);
            PackedRow<FMT> y;
            if constexpr (FMT == kE4m3) {
              quantise<HD>(x, magnitude(x), y);
              if (i * PER < heads) {
                const long long at_row = to + i * PER * head_rows;
                uint8_t* dst = static_cast<uint8_t*>(p.pool.k) + at_row * HD;
                *reinterpret_cast<uint32_t*>(dst + d0) = y.x.x;
                *reinterpret_cast<uint32_t*>(dst + d1) = y.x.y;
                if (l == 0) p.pool.k_scales[at_row] = y.s;
              }
            } else {
              float* own = reinterpret_cast<float*>(smem + norm_off_turn(FMT) + (WARPS + warp) * 1024) + sub * HD;
              __syncwarp();
              *reinterpret_cast<float4*>(own + d0) = make_float4(x[0], x[1], x[2], x[3]);
              *reinterpret_cast<float4*>(own + d1) = make_float4(x[4], x[5], x[6], x[7]);
              __syncwarp();
#pragma unroll
              for (int j = 0; j < 8; ++j) x[j] = own[8 * l + j];
              quantise<HD>(x, magnitude(x), y);
              if (i * PER < heads) store_row<HD>(p.pool, true, to + i * PER * head_rows, l, y);
            }
          }
          __syncwarp();  // the slot has been read
        }
      }
      continue;
    }
    // Rows of bf16: unit i of a batch goes to dst + i apart.
    const bool paged = APPEND && kind == 1;
    const long long apart = paged ? PER * HD * head_rows : PER * HD;
    __nv_bfloat16* dst = paged ? static_cast<__nv_bfloat16*>(p.pool.k) + (page_row + h0 * head_rows) * HD
                               : (kind == 0 ? p.q_out + row * p.q_out_stride : p.k_out + row * p.k_out_stride) +
                                     static_cast<long long>(h0) * HD;
    auto put = [&](int i, const Pairs& y) {
      uint2 r0, r1;
      as_runs<NEIGHBOURS>(y, r0, r1);
      if (i * PER < heads) {
        *reinterpret_cast<uint2*>(dst + i * apart + d0) = r0;
        *reinterpret_cast<uint2*>(dst + i * apart + d1) = r1;
      }
    };
    if (p.batch == 1) {
#pragma unroll 1
      for (int b = 0; b < batches; ++b, heads -= step, dst += apart) {
        put(0, turned(take()));
        __syncwarp();  // the slot has been read
      }
    } else {
#pragma unroll 1
      for (int b = 0; b < batches; ++b, heads -= step, dst += kNormBatch * apart) {
        const uint8_t* batch = take();
        // (A unit behind the last head is what the slot held before, and goes nowhere.)
#pragma unroll
        for (int g = 0; g < kNormBatch; g += kNormSide) {
          if (g * PER >= heads + sub) break;  // (alike in the warp)
          Pairs y[kNormSide];
#pragma unroll
          for (int i = 0; i < kNormSide; ++i) y[i] = turned(batch + (g + i) * 512);
#pragma unroll
          for (int i = 0; i < kNormSide; ++i) put(g + i, y[i]);
        }
        __syncwarp();  // the slot has been read
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace cpattn
