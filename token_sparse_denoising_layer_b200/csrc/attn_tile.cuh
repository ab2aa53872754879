// attn_tile.cuh - softmax arithmetic on one 128-key row of scores, shared by
// the attention kernels.
#pragma once

#include <stdint.h>

#include "ptx.cuh"

namespace hsa {

constexpr int kKV = 128;       // keys per tile

// Largest P (and so row sum) a tile may reach before the running max must be
// raised: far inside the range of bf16 and of the fp32 row sums and O.
constexpr float kSumLimit = 18446744073709551616.0f;  // 2^64

__device__ __forceinline__ float row_max(const uint32_t (&sr)[kKV]) {
  float mx[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) mx[u] = __uint_as_float(sr[u]);
#pragma unroll
  for (int e = 8; e < kKV; ++e) mx[e & 7] = fmaxf(mx[e & 7], __uint_as_float(sr[e]));
  return fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
               fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
}

// P = exp2(S*c - m) as bf16 pairs in w (packed f32x2 arithmetic: two lanes
// per FMA/add instruction); returns the row sum of P.
__device__ __forceinline__ float exp_row(const uint32_t (&sr)[kKV], float c, float m,
                                         uint32_t (&w)[kKV / 2]) {
  float rs0[4] = {0.f, 0.f, 0.f, 0.f}, rs1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < kKV; e += 2) {
    float xa, xb;
    fma2(xa, xb, __uint_as_float(sr[e]), __uint_as_float(sr[e + 1]), c, -m);
    const float a = ex2_approx(xa);
    const float b = ex2_approx(xb);
    add2(rs0[(e >> 1) & 3], rs1[(e >> 1) & 3], a, b);
    w[e / 2] = pack_bf16(a, b);
  }
  return ((rs0[0] + rs1[0]) + (rs0[1] + rs1[1])) + ((rs0[2] + rs1[2]) + (rs0[3] + rs1[3]));
}

}  // namespace hsa
