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
// The upper 32 bits, as a signed fraction of a half turn, go to sincospif.
//
// HBM-bound: Q and K are read and written once, 8 flops a value.  A head's row
// lies in HD / 8 lanes, eight values each, so that both values of a pair are in
// one lane and a norm is one sum over those lanes; a warp keeps a row's cos, sin
// and the norms' weights in registers for all the heads that it takes.
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

template <int HD>
__device__ __forceinline__ void norm_and_turn(float (&x)[8], const float* w, int d0, int d1, float eps,
                                              bool turn, bool neighbours, const float (&cs)[4],
                                              const float (&sn)[4]) {
  if (w != nullptr) {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
#pragma unroll
    for (int o = HD / 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    const float r = rsqrtf(fmaf(sum, 1.f / HD, eps));
    const float4 w0 = *reinterpret_cast<const float4*>(w + d0), w1 = *reinterpret_cast<const float4*>(w + d1);
    x[0] *= r * w0.x;
    x[1] *= r * w0.y;
    x[2] *= r * w0.z;
    x[3] *= r * w0.w;
    x[4] *= r * w1.x;
    x[5] *= r * w1.y;
    x[6] *= r * w1.z;
    x[7] *= r * w1.w;
  }
  auto pair = [&](float& a, float& b, int j) {
    const float a0 = a;
    a = fmaf(a0, cs[j], -b * sn[j]);
    b = fmaf(b, cs[j], a0 * sn[j]);
  };
  if (turn && neighbours) {
#pragma unroll
    for (int j = 0; j < 4; ++j) pair(x[2 * j], x[2 * j + 1], j);
  } else if (turn) {
#pragma unroll
    for (int j = 0; j < 4; ++j) pair(x[j], x[j + 4], j);
  }
}

__device__ __forceinline__ void bf16x4_to_f32(uint2 x, float* f) {
  f[0] = __uint_as_float(x.x << 16);
  f[1] = __uint_as_float(x.x & 0xFFFF0000u);
  f[2] = __uint_as_float(x.y << 16);
  f[3] = __uint_as_float(x.y & 0xFFFF0000u);
}

// Work split: a unit is 512 bytes of a row (a head of 256, two of 128), a batch up
// to kNormBatch units of one kind (Q, K or V), and each warp takes an equal,
// contiguous slice of the list of all rows' batches.  Its next batches are copied
// to shared memory while it works on one: what bounds the kernel is how much of
// it is in flight.
#ifndef X_NSLOTS
#define X_NSLOTS 6
#define X_NBLK 2
#endif
constexpr int kNormThreads = 256;
constexpr int kNormBatch = 4;
constexpr int kNormSlots = X_NSLOTS;   // batches of a warp in flight, or being read
constexpr int kNormBlocks = X_NBLK;  // per SM

__host__ __device__ constexpr int norm_rope_smem(int fmt) {
  // The slots; (e2m1) for each warp a K unit on its way from the rotation's order to
  // that of the pages; the weights.
  return kNormThreads / 32 * (kNormSlots * kNormBatch * 512 + (fmt == kE2m1 ? 1024 : 0)) + 2048;
}

// Four values to d0 .. and four to d1 .. of a row.
__device__ __forceinline__ void put_runs(__nv_bfloat16* row, int d0, int d1, const float (&x)[8]) {
  *reinterpret_cast<uint2*>(row + d0) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  *reinterpret_cast<uint2*>(row + d1) = make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ uint32_t magnitude(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(x[j]) & 0x7FFFFFFFu);
  return m;
}

// FMT: the pages' format, or -1: K goes to k_out.
template <int HD, int FMT>
__global__ void __launch_bounds__(kNormThreads, kNormBlocks)
    norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr bool APPEND = FMT >= 0;
  constexpr int LANES = HD / 8, PER = 32 / LANES;  // lanes of a head, heads of a unit
  constexpr int WARPS = kNormThreads / 32, SLOT = kNormBatch * 512;
  extern __shared__ __align__(16) uint8_t smem[];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % LANES, sub = lane / LANES;
  const uint8_t* slots = smem + warp * (kNormSlots * SLOT);
  const uint32_t slots_at = smem_u32(slots);
  const bool neighbours = p.neighbours != 0, turn = l < p.rot / 8;
  int d0, d1;
  lane_dims(l, p.rot, neighbours, &d0, &d1);

  // The list: bq batches of Q, bk of K and (append) bk of V for each row.
  const int uq = (p.nq + PER - 1) / PER, uk = (p.nkv + PER - 1) / PER;
  const int bq = (uq + p.batch - 1) / p.batch, bk = (uk + p.batch - 1) / p.batch;
  const int per_row = bq + (APPEND ? 2 : 1) * bk;
  const long long total = static_cast<long long>(p.rows) * per_row;
  const int w = blockIdx.x * WARPS + warp, ws = gridDim.x * WARPS;
  const long long t0 = total * w / ws, t1 = total * (w + 1) / ws;
  struct Place {  // of a batch
    int row, j;
  };
  auto next = [&](Place& b) {
    if (++b.j == per_row) {
      b.j = 0;
      ++b.row;
    }
  };
  auto kind_of = [&](int j) { return j < bq ? 0 : (j < bq + bk ? 1 : 2); };
  Place at = {static_cast<int>(t0 / per_row), static_cast<int>(t0 % per_row)}, ahead = at;
  long long copied = t0;
  int slot_in = 0;
  auto copy_batch = [&]() {
    if (copied < t1) {
      const int kind = kind_of(ahead.j), first = (ahead.j - (kind == 0 ? 0 : (kind == 1 ? bq : bq + bk))) * p.batch;
      const int heads = kind == 0 ? p.nq : p.nkv;
      const __nv_bfloat16* src = (kind == 0   ? p.q + ahead.row * p.q_stride
                                  : kind == 1 ? p.k + ahead.row * p.k_stride
                                              : p.v + ahead.row * p.v_stride) +
                                 static_cast<long long>(first) * (PER * HD) + 8 * lane;
#pragma unroll
      for (int i = 0; i < kNormBatch; ++i)
        if (i < p.batch && (first + i) * PER + sub < heads)
          copy16_async(slots_at + slot_in * SLOT + i * 512 + 16 * lane, src + i * (PER * HD));
      if (++slot_in == kNormSlots) slot_in = 0;
      next(ahead);
      ++copied;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < kNormSlots - 1; ++i) copy_batch();

  // The next row's position and slot, loaded a row ahead.
  int pos = -1, slot = -1;
  auto load_place = [&](int row) {
    if (row >= p.rows) return;
    pos = load_now(p.positions + row);
    if (APPEND) slot = load_now(p.slots + row);
  };
  load_place(at.row);
  unsigned long long step[4] = {};
  if (turn) {
#pragma unroll
    for (int j = 0; j < 4; ++j) step[j] = load_now(p.steps + 4 * l + j);
  }
  float* weights = reinterpret_cast<float*>(smem + norm_rope_smem(FMT) - 2048);  // Q's, then K's
  for (int i = threadIdx.x; i < 2 * HD; i += kNormThreads) {
    const void* from = i < HD ? p.q_weight : p.k_weight;
    const int d = i & (HD - 1);
    if (from != nullptr)
      weights[i] = p.weight_f32 != 0 ? load_now(static_cast<const float*>(from) + d)
                                     : __bfloat162float(load_now(static_cast<const __nv_bfloat16*>(from) + d));
  }
  const float* wq = p.q_weight != nullptr ? weights : nullptr;
  const float* wk = p.k_weight != nullptr ? weights + HD : nullptr;
  __syncthreads();

  int row = -1, slot_out = 0;
  bool live = false;
  long long page_row = -1;  // (append) of the row's place, kv head 0; -1: not stored
  float cs[4], sn[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) cs[j] = sn[j] = 0.f;
#pragma unroll 1
  for (long long t = t0; t < t1; ++t) {
    copy_batch();
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
      if (turn) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int part = static_cast<int>((step[j] * static_cast<unsigned long long>(pos)) >> 32);
          sincospif(static_cast<float>(part) * 4.6566128730773926e-10f, &sn[j], &cs[j]);
          sn[j] *= p.scale;
          cs[j] *= p.scale;
        }
      }
      load_place(row + 1);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kNormSlots - 1) : "memory");
    __syncwarp();
    const uint8_t* batch = slots + slot_out * SLOT;
    if (++slot_out == kNormSlots) slot_out = 0;
    const int kind = kind_of(at.j), first = (at.j - (kind == 0 ? 0 : (kind == 1 ? bq : bq + bk))) * p.batch;
    const int units = min(p.batch, (kind == 0 ? uq : uk) - first);
    const int h0 = first * PER + sub, heads = kind == 0 ? p.nq : p.nkv;  // unit i: head h0 + i PER
    next(at);
    if (!live || (APPEND && kind != 0 && page_row < 0)) {
    } else if (kind != 2) {
      // Unit i, normed and turned, in lane_dims' order.
      auto turned = [&](int i, float (&x)[8]) {
        const uint8_t* raw = batch + i * 512 + sub * (2 * HD);
        bf16x4_to_f32(*reinterpret_cast<const uint2*>(raw + 2 * d0), x);
        bf16x4_to_f32(*reinterpret_cast<const uint2*>(raw + 2 * d1), x + 4);
        norm_and_turn<HD>(x, kind == 0 ? wq : wk, d0, d1, p.eps, turn, neighbours, cs, sn);
      };
      if (FMT == kE2m1 && kind == 1) {
        if constexpr (FMT == kE2m1) {
          float* mine = reinterpret_cast<float*>(smem + WARPS * (kNormSlots * SLOT) + warp * 1024) + sub * HD;
#pragma unroll 1
          for (int i = 0; i < units; ++i) {
            float x[8];
            turned(i, x);
            __syncwarp();
            *reinterpret_cast<float4*>(mine + d0) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4*>(mine + d1) = make_float4(x[4], x[5], x[6], x[7]);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = mine[8 * l + j];
            PackedRow<FMT> y;
            quantise<HD>(x, magnitude(x), false, y);
            const int h = h0 + i * PER;
            if (h < heads)
              store_row<HD>(p.pool, true, page_row + (static_cast<long long>(h) << p.pool.page_shift), l, y);
          }
        }
      } else {
        auto put = [&](int i, const float (&x)[8]) {
          const int h = h0 + i * PER;
          if (APPEND && kind == 1) {
            const long long to = page_row + (static_cast<long long>(h) << p.pool.page_shift);
            if constexpr (FMT == kE4m3) {
              PackedRow<FMT> y;
              quantise<HD>(x, magnitude(x), false, y);
              if (h < heads) {
                uint8_t* dst = static_cast<uint8_t*>(p.pool.k) + to * HD;
                *reinterpret_cast<uint32_t*>(dst + d0) = y.x.x;
                *reinterpret_cast<uint32_t*>(dst + d1) = y.x.y;
                if (l == 0) p.pool.k_scales[to] = y.s;
              }
            } else if (h < heads) {
              put_runs(static_cast<__nv_bfloat16*>(p.pool.k) + to * HD, d0, d1, x);
            }
          } else if (h < heads) {
            put_runs((kind == 0 ? p.q_out + row * p.q_out_stride : p.k_out + row * p.k_out_stride) +
                         static_cast<long long>(h) * HD,
                     d0, d1, x);
          }
        };
        if (units == 1) {
          float x[8];
          turned(0, x);
          put(0, x);
        } else {
          // Side by side.  (Units behind the last one are what the slot holds, and
          // go nowhere: their heads are no heads.)
          float x[kNormBatch][8];
#pragma unroll
          for (int i = 0; i < kNormBatch; ++i) turned(i, x[i]);
#pragma unroll
          for (int i = 0; i < kNormBatch; ++i) put(i, x[i]);
        }
      }
    } else if constexpr (APPEND) {
#pragma unroll
      for (int i = 0; i < kNormBatch; ++i) {
        if (i >= units) break;
        const uint4 v = *reinterpret_cast<const uint4*>(batch + i * 512 + 16 * lane);
        PackedRow<FMT> y;
        if constexpr (FMT == kBf16) {
          y.x = v;
        } else {
          float x[8];
          bf16x8_to_f32x8(v, x);
          quantise<HD>(x, amax_bits(v) << 16, true, y);
        }
        const int h = h0 + i * PER;
        if (h < heads)
          store_row<HD>(p.pool, false, page_row + (static_cast<long long>(h) << p.pool.page_shift), l, y);
      }
    }
    __syncwarp();  // the slot has been read
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace cpattn
