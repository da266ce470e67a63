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
  int parts;                       // warps that share a row
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

__device__ __forceinline__ void load_weights(const void* w, int f32, int d0, int d1, float (&out)[8]) {
  if (w == nullptr) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int d = j < 4 ? d0 + j : d1 + j - 4;
    out[j] = f32 != 0 ? load_now(static_cast<const float*>(w) + d)
                      : __bfloat162float(load_now(static_cast<const __nv_bfloat16*>(w) + d));
  }
}

template <int HD>
__device__ __forceinline__ void norm_and_turn(float (&x)[8], bool norm, const float (&w)[8], float eps,
                                              bool turn, bool neighbours, const float (&cs)[4],
                                              const float (&sn)[4]) {
  if (norm) {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
#pragma unroll
    for (int o = HD / 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    const float r = rsqrtf(fmaf(sum, 1.f / HD, eps));
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
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

constexpr int kNormThreads = 256;
constexpr int kNormBatch = 4;  // heads (HD = 128: pairs of heads) in flight per warp

// FMT: the pages' format, or -1: K goes to k_out.
template <int HD, int FMT>
__global__ void __launch_bounds__(kNormThreads)
    norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr bool APPEND = FMT >= 0;
  constexpr int LANES = HD / 8, PER = 32 / LANES;  // lanes of a head, heads of a warp
  // A K row on its way from the rotation's order to that of the pages.
  __shared__ __align__(16) float stage[APPEND ? kNormThreads / 32 * PER * HD : 1];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % LANES, sub = lane / LANES;
  const bool neighbours = p.neighbours != 0, turn = l < p.rot / 8;
  int d0, d1;
  lane_dims(l, p.rot, neighbours, &d0, &d1);
  unsigned long long step[4] = {};
  if (turn) {
#pragma unroll
    for (int j = 0; j < 4; ++j) step[j] = load_now(p.steps + 4 * l + j);
  }
  // Units of PER heads: Q's, K's, V's.
  const int uq = (p.nq + PER - 1) / PER, uk = (p.nkv + PER - 1) / PER;
  const int units = uq + (APPEND ? 2 : 1) * uk, per = (units + p.parts - 1) / p.parts;
  const long long items = static_cast<long long>(p.rows) * p.parts;
  const long long warps = static_cast<long long>(gridDim.x) * (kNormThreads / 32);
  for (long long it = static_cast<long long>(blockIdx.x) * (kNormThreads / 32) + warp; it < items;
       it += warps) {
    const int row = static_cast<int>(it / p.parts);
    const int u0 = static_cast<int>(it % p.parts) * per, u1 = min(units, u0 + per);
    const int pos = load_now(p.positions + row);
    if (pos < 0) continue;
    int slot = -1;
    if constexpr (APPEND) {
      slot = load_now(p.slots + row);
      if (slot >= p.pool.num_pages << p.pool.page_shift) {
        if (u0 < u1 && lane == 0 && p.status != nullptr) atomicCAS(p.status, kStatusOk, kStatusPage);
        slot = -1;
      }
    }
    float cs[4], sn[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned long long t = step[j] * static_cast<unsigned long long>(pos);
      sincospif(static_cast<float>(static_cast<int>(t >> 32)) * 4.6566128730773926e-10f, &sn[j], &cs[j]);
      sn[j] *= p.scale;
      cs[j] *= p.scale;
    }
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {  // Q, then K
      const int a = max(u0, kind == 0 ? 0 : uq), b = min(u1, kind == 0 ? uq : uq + uk);
      if (a >= b || (APPEND && kind == 1 && slot < 0)) continue;
      const void* weight = kind == 0 ? p.q_weight : p.k_weight;
      float w[8];
      load_weights(weight, p.weight_f32, d0, d1, w);
      const int heads = kind == 0 ? p.nq : p.nkv;
      const __nv_bfloat16* src = kind == 0 ? p.q + row * p.q_stride : p.k + row * p.k_stride;
      __nv_bfloat16* dst = kind == 0 ? p.q_out + row * p.q_out_stride
                                     : (APPEND ? nullptr : p.k_out + row * p.k_out_stride);
      for (int u = a; u < b; u += kNormBatch) {
        uint2 raw[kNormBatch][2];
#pragma unroll
        for (int i = 0; i < kNormBatch; ++i) {
          const int h = min((u + i - (kind == 0 ? 0 : uq)) * PER + sub, heads - 1);
          raw[i][0] = load_now(reinterpret_cast<const uint2*>(src + h * HD + d0));
          raw[i][1] = load_now(reinterpret_cast<const uint2*>(src + h * HD + d1));
        }
#pragma unroll
        for (int i = 0; i < kNormBatch; ++i) {
          if (u + i >= b) break;
          const int h = (u + i - (kind == 0 ? 0 : uq)) * PER + sub;
          float x[8];
          bf16x4_to_f32(raw[i][0], x);
          bf16x4_to_f32(raw[i][1], x + 4);
          norm_and_turn<HD>(x, weight != nullptr, w, p.eps, turn, neighbours, cs, sn);
          if constexpr (APPEND) {
            if (kind == 1) {
              float* mine = stage + (warp * PER + sub) * HD;
              __syncwarp();
              *reinterpret_cast<float4*>(mine + d0) = make_float4(x[0], x[1], x[2], x[3]);
              *reinterpret_cast<float4*>(mine + d1) = make_float4(x[4], x[5], x[6], x[7]);
              __syncwarp();
              float y[8];
              uint32_t mag = 0;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                y[j] = mine[8 * l + j];
                mag = max(mag, __float_as_uint(y[j]) & 0x7FFFFFFFu);
              }
              const long long at =
                  h < heads ? pool_row(p.pool, slot >> p.pool.page_shift, h,
                                       slot & ((1 << p.pool.page_shift) - 1))
                            : -1;
              store_row<HD, FMT>(p.pool, true, at, l, y, mag);
              continue;
            }
          }
          if (h < heads) {
            *reinterpret_cast<uint2*>(dst + h * HD + d0) =
                make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
            *reinterpret_cast<uint2*>(dst + h * HD + d1) =
                make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
          }
        }
      }
    }
    if constexpr (APPEND) {
      if (slot < 0) continue;
      const int a = max(u0, uq + uk) - uq - uk, b = u1 - uq - uk;
      for (int u = a; u < b; ++u) {
        const int h = u * PER + sub;
        const uint4 raw = load_now(reinterpret_cast<const uint4*>(
                                       p.v + row * p.v_stride + min(h, p.nkv - 1) * HD) + l);
        const long long at = h < p.nkv ? pool_row(p.pool, slot >> p.pool.page_shift, h,
                                                  slot & ((1 << p.pool.page_shift) - 1))
                                       : -1;
        if constexpr (FMT == kBf16) {
          if (at >= 0) reinterpret_cast<uint4*>(p.pool.v)[at * (HD / 8) + l] = raw;
        } else {
          float x[8];
          bf16x8_to_f32x8(raw, x);
          store_row<HD, FMT>(p.pool, false, at, l, x, amax_bits(raw) << 16);
        }
      }
    }
  }
}

}  // namespace cpattn
