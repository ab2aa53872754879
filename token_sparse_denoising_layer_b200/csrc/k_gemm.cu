// k_gemm.cu - active-row GEMMs of the HSA layer on the 5th-generation tensor
// cores (tcgen05.mma, fp32 accumulators in TMEM, operands staged by TMA).
//
// C[m, j] = sum_k A[m, k] * B[j, k], A = compact bf16 activations of the
// active rows [M = |A_i|, K], B = a Linear weight [Ncols, K].  The epilogue
// is where the sparse structure of the method lives ("Technical Summary:
// Heterogeneous Step Allocation (HSA) for Efficient Video Generation",
// section 2.2): fresh K/V rows are scattered into the KV cache rows idx[m],
// and out-projection / MLP results are added into residual rows idx[m].
//
// Persistent: one CTA per SM walks its share of the 128 x BN output tiles
// (BN = 256, 192 or 128), K-block 64, through a multi-stage TMA ring that runs
// on across tiles.  Warp 0 issues TMA, warp 1 owns TMEM and issues the MMAs
// (one thread) into one of two TMEM accumulators, and eight epilogue warps
// drain the other accumulator (two per TMEM lane quarter, one per column
// half), so a tile's epilogue overlaps the next tile's main loop.
//
// The same kernels take signed 8-bit operands (kS8): C is then an exact 32-bit
// integer sum, scaled by a_scale[m] b_scale[j] before the epilogue.  32760 x 8960 x
// 1536: 277 us, 3250 TOP/s, twice the burst rate of bf16; x 1536 x 8960: 315 us.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <string>

#include "internal.h"
#include "ptx.cuh"

namespace hsa {

namespace {

constexpr int kBM = 128;
constexpr int kBK = 64;
constexpr int kGemmThreads = 320;  // TMA warp, MMA warp, 8 epilogue warps
constexpr int kEpiWarps = 8;
// relative cost per output element of a CTA-pair tile vs a 1-CTA 256-wide tile
constexpr double kPairCost = 0.8;

// Shared-memory staging for the residual epilogue: one 32 x 32 fp32 chunk
// per epilogue warp.  The 16-byte group g of row r is stored at group
// g ^ (r & 7), which keeps both the row-wise writes and the column-wise reads
// below free of bank conflicts without padding.
constexpr int kStageWarpFloats = 32 * 32;
constexpr int kEpiStageBytes = kEpiWarps * kStageWarpFloats * 4;

template <int BN>
struct GemmCfg {
  static constexpr int kStages = BN == 128 ? 6 : 4;
  // two accumulators of BN fp32 columns, allocated as a power of two
  static constexpr uint32_t kTmemCols = 2 * BN <= 256 ? 256 : 512;
  static constexpr int kABytes = kBM * kBK * 2;
  static constexpr int kBBytes = BN * kBK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kBarBytes = 256;
  static constexpr int kSmem = kStages * kStageBytes + kBarBytes + kEpiStageBytes + 1024;
};

struct EpiParams {
  int M, Ncols, Kd, epi;
  __nv_bfloat16* out;
  int ld_out;
  __nv_bfloat16* kc[kMaxCaches];  // EPI_QKV: n_caches copies of the K and V caches
  __nv_bfloat16* vc[kMaxCaches];
  int n_caches;
  float* x;
  int ld_x;
  const float* gate;
  const int32_t* idx;
  int N;
  int* flag;
  const float* a_scale;  // 8-bit operands: C = a_scale[m] b_scale[j] (integer sum)
  const float* b_scale;
};

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// GELU, erf form, of two values: v Phi(v), with Phi(v) = 1 - erfc(v / sqrt 2) / 2
// for v >= 0 and erfc(|v| / sqrt 2) / 2 for v < 0.  erfc(z), z >= 0, is the
// Chebyshev fit of Press, Teukolsky, Vetterling & Flannery, Numerical Recipes,
// section 6.2: t = 1 / (1 + z/2), erfc(z) = t exp(-z^2 + P(t)) with a degree-9
// P, a fractional error below 1.2e-7 for every z.  A relative bound matters
// here: for v < 0 the result is a small tail value that is then rounded to
// bf16.  Evaluated on packed f32x2 lanes with P's coefficients negated (Horner
// commutes with negation), and the 1/2 folded into the exponent; two MUFU
// operations per value, no branches.
__device__ __forceinline__ F2 gelu_x2(F2 v) {
  const F2 zn = F2{fabsf(v.x) * -0.70710678118654752440f, fabsf(v.y) * -0.70710678118654752440f};
  const F2 d = fma_x2(zn, splat(-0.5f), splat(1.0f));  // 1 + z/2
  const F2 t = F2{rcp_approx(d.x), rcp_approx(d.y)};
  F2 q = fma_x2(splat(-0.17087277f), t, splat(0.82215223f));  // -P(t) by Horner
  q = fma_x2(q, t, splat(-1.48851587f));
  q = fma_x2(q, t, splat(1.13520398f));
  q = fma_x2(q, t, splat(-0.27886807f));
  q = fma_x2(q, t, splat(0.18628806f));
  q = fma_x2(q, t, splat(-0.09678418f));
  q = fma_x2(q, t, splat(-0.37409196f));
  q = fma_x2(q, t, splat(-1.00002368f));
  q = fma_x2(q, t, splat(1.26551223f));
  q = fma_x2(zn, zn, q);  // z^2 - P(t)
  // log2 of erfc(z) / 2 / t: (P(t) - z^2) log2(e) - 1
  const F2 s = fma_x2(q, splat(-1.4426950408889634f), splat(-1.0f));
  const F2 he = mul_x2(t, F2{ex2_approx(s.x), ex2_approx(s.y)});  // erfc(z) / 2
  const F2 phi = F2{v.x >= 0.f ? 1.0f - he.x : he.x, v.y >= 0.f ? 1.0f - he.y : he.y};
  return mul_x2(v, phi);
}

// 32 fp32 accumulators -> 32 bf16 (rounded to nearest even) in four 16-byte words.
__device__ __forceinline__ void pack_bf16x32(const uint32_t (&r)[32], uint4 (&w)[4]) {
#pragma unroll
  for (int v = 0; v < 4; ++v)
    w[v] = make_uint4(pack_bf16(__uint_as_float(r[8 * v]), __uint_as_float(r[8 * v + 1])),
                      pack_bf16(__uint_as_float(r[8 * v + 2]), __uint_as_float(r[8 * v + 3])),
                      pack_bf16(__uint_as_float(r[8 * v + 4]), __uint_as_float(r[8 * v + 5])),
                      pack_bf16(__uint_as_float(r[8 * v + 6]), __uint_as_float(r[8 * v + 7])));
}

// 32 fp32 accumulators -> 32 bf16 at dst (64 contiguous bytes, 16-byte aligned).
template <bool kGelu>
__device__ __forceinline__ void store_bf16x32(__nv_bfloat16* dst, const uint32_t (&r)[32]) {
  uint4* d4 = reinterpret_cast<uint4*>(dst);
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a = __uint_as_float(r[8 * v + 2 * e]);
      float b = __uint_as_float(r[8 * v + 2 * e + 1]);
      if (kGelu) {
        const F2 g = gelu_x2(F2{a, b});
        a = g.x;
        b = g.y;
      }
      w[e] = pack_bf16(a, b);
    }
    d4[v] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}


// x[dst_row(r), col .. col+31] += chunk row r for the warp's 32 rows, as
// vector reductions that L2 performs, so the epilogue never waits for the
// residual rows it updates.  The chunk (row r in lane r's registers) goes
// through shared memory so that one reduction instruction covers four rows
// and 128 contiguous bytes of each: lanes 8k'..8k'+7 own row 4k + k'.  Each
// element gets exactly one addition per launch: x + v rounded once (with a
// gate, gate * v is rounded first).
__device__ __forceinline__ void resid_chunk(const EpiParams& p, const uint32_t (&r)[32],
                                            int32_t dst_row, int col, float* stage) {
  const int lane = threadIdx.x & 31;
  float* srow = stage + lane * 32;
#pragma unroll
  for (int v = 0; v < 8; ++v)
    *reinterpret_cast<float4*>(srow + 4 * (v ^ (lane & 7))) =
        make_float4(__uint_as_float(r[4 * v]), __uint_as_float(r[4 * v + 1]),
                    __uint_as_float(r[4 * v + 2]), __uint_as_float(r[4 * v + 3]));
  __syncwarp();
  const int g4 = lane & 7;  // this lane's 16-byte group of the row
  float4 g = make_float4(1.f, 1.f, 1.f, 1.f);
  if (p.gate != nullptr) g = __ldg(reinterpret_cast<const float4*>(p.gate + col + 4 * g4));
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int rr = 4 * k + (lane >> 3);
    const int32_t d = __shfl_sync(0xffffffffu, dst_row, rr);
    float4 v = *reinterpret_cast<const float4*>(stage + rr * 32 + 4 * (g4 ^ (rr & 7)));
    if (d >= 0) {
      if (p.gate != nullptr) {
        v.x *= g.x;
        v.y *= g.y;
        v.z *= g.z;
        v.w *= g.w;
      }
      float* dst = p.x + static_cast<size_t>(d) * p.ld_x + col + 4 * g4;
      asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(dst), "f"(v.x),
                   "f"(v.y), "f"(v.z), "f"(v.w)
                   : "memory");
    }
  }
  __syncwarp();  // the stage is reused by the next chunk
}

// Scales of one chunk's columns (zero past Ncols).
__device__ __forceinline__ void load_scales(const EpiParams& p, int col, F2 (&s)[16]) {
  if (col + 32 <= p.Ncols) {
    const float4* s4 = reinterpret_cast<const float4*>(p.b_scale + col);
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      const float4 x = __ldg(s4 + v);
      s[2 * v] = F2{x.x, x.y};
      s[2 * v + 1] = F2{x.z, x.w};
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      s[e] = F2{col + 2 * e < p.Ncols ? __ldg(p.b_scale + col + 2 * e) : 0.f,
                col + 2 * e + 1 < p.Ncols ? __ldg(p.b_scale + col + 2 * e + 1) : 0.f};
  }
}

// Integer sums of one chunk of a row -> fp32 products: float(sum) * sa * sb[j].
// The integer sum is exact, so three roundings to 32 bits are all there are
// before the epilogue's own.
__device__ __forceinline__ void dequant_chunk(uint32_t (&r)[32], float sa, const F2 (&s)[16]) {
  const F2 sa2 = splat(sa);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const F2 x = mul_x2(mul_x2(F2{__int2float_rn(static_cast<int>(r[2 * e])),
                                  __int2float_rn(static_cast<int>(r[2 * e + 1]))},
                               sa2),
                        s[e]);
    r[2 * e] = __float_as_uint(x.x);
    r[2 * e + 1] = __float_as_uint(x.y);
  }
}

// 32 fp32 values of this lane's row -> bf16 in the warp's stage, columns 32 half ..
// of a row of 64.  The 16-byte group g of row r lies at group g ^ (r & 7):
// free of bank conflicts by rows and by columns.
__device__ __forceinline__ void stage_half(uint8_t* stage, const uint32_t (&r)[32], int half) {
  const int lane = threadIdx.x & 31;
  uint4 w[4];
  pack_bf16x32(r, w);
#pragma unroll
  for (int v = 0; v < 4; ++v)
    *reinterpret_cast<uint4*>(stage + lane * 128 + 16 * ((4 * half + v) ^ (lane & 7))) = w[v];
}

// Send the warp's staged rows off, 64 columns of them from `col` on, as one tiled
// store that clips what lies past M or Ncols.  The warp does not wait for it:
// an SM stores about 32 bytes a clock, so a 128 x 256 tile's rows take 2000 clocks.
__device__ __forceinline__ void store_staged(const CUtensorMap* tm_out, const uint8_t* stage,
                                             int m0, int col) {
  fence_proxy_async_smem();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    tma_store_2d(tm_out, stage, col, m0);
    tma_store_commit();
  }
}

// Store 32 staged columns (the first half of the stage's rows) where no second
// half follows: one instruction covers eight rows and 64 bytes of each.
__device__ __forceinline__ void store_half(const EpiParams& p, const uint8_t* stage, int m0, int col) {
  const int lane = threadIdx.x & 31, g = lane & 3;
  __syncwarp();
  uint4 w[4];  // read all before the first is stored: a load waits behind a store
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int rr = 8 * k + (lane >> 2);
    w[k] = *reinterpret_cast<const uint4*>(stage + rr * 128 + 16 * (g ^ (rr & 7)));
  }
  if (col + 8 * g < p.Ncols) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int rr = 8 * k + (lane >> 2);
      if (m0 + rr < p.M)
        *reinterpret_cast<uint4*>(p.out + static_cast<size_t>(m0 + rr) * p.ld_out + col + 8 * g) = w[k];
    }
  }
  __syncwarp();  // the stage is reused by the next tile
}

// Store staged columns col .. end - 1 (up to 64) of a bf16 output whose rows are
// not 16-byte aligned, in the widest stores that the row length allows: 8 bytes
// a lane and two rows an instruction, 4 bytes and one row, or 2 bytes and half a
// row.  Eight instructions' rows are read before the first is stored.  (5000 x 700 x
// 3000: 21 us, 3004 25, 3002 31, 3001 30; 4-byte stores from an odd row's first
// even place on took 43.)
__device__ __forceinline__ void store_ragged(const EpiParams& p, const uint8_t* stage, int m0,
                                             int col, int end) {
  const int lane = threadIdx.x & 31;
  const int rows = p.M - m0 < 32 ? p.M - m0 : 32;
  const size_t ld = p.ld_out;
  auto at = [&](int r, int e) { return stage + r * 128 + 16 * ((e >> 3) ^ (r & 7)) + 2 * (e & 7); };
  __nv_bfloat16* out = p.out + m0 * ld + col;
  __syncwarp();
  if ((p.ld_out & 3) == 0) {
    const int e = 4 * (lane & 15);
#pragma unroll
    for (int r0 = 0; r0 < 32; r0 += 16) {
      uint2 w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = *reinterpret_cast<const uint2*>(at(r0 + 2 * k + (lane >> 4), e));
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = r0 + 2 * k + (lane >> 4);
        if (r < rows && col + e < end) *reinterpret_cast<uint2*>(out + r * ld + e) = w[k];
      }
    }
  } else if ((p.ld_out & 1) == 0) {
    const int e = 2 * lane;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 8) {
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = *reinterpret_cast<const uint32_t*>(at(r0 + k, e));
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (r0 + k < rows && col + e < end) *reinterpret_cast<uint32_t*>(out + (r0 + k) * ld + e) = w[k];
    }
  } else {
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 8) {
      uint16_t w[8][2];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        w[k][0] = *reinterpret_cast<const uint16_t*>(at(r0 + k, lane));
        w[k][1] = *reinterpret_cast<const uint16_t*>(at(r0 + k, lane + 32));
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        uint16_t* dst = reinterpret_cast<uint16_t*>(out + (r0 + k) * ld);
        if (r0 + k < rows && col + lane < end) dst[lane] = w[k][0];
        if (r0 + k < rows && col + lane + 32 < end) dst[lane + 32] = w[k][1];
      }
    }
  }
  __syncwarp();  // the stage is reused by the next 64 columns
}

// Drain one accumulator tile: this warp's 32 rows (TMEM lanes at tbase),
// output row m (this lane's), columns n0 .. n0 + kCols - 1.  TMEM loads run
// one 32-column chunk ahead of the chunk being stored.  `sa` is the row's scale
// (8-bit operands).
template <bool kS8, int kCols, int kEpi>
__device__ __forceinline__ void drain_tile(const EpiParams& p, const CUtensorMap* tm_out,
                                           uint32_t tbase, int m, int n0, float sa, float* stage) {
  constexpr int NC = kCols / 32;
  const bool mrow = m < p.M;
  int32_t dst_row = -1;
  if ((kEpi == EPI_QKV || kEpi == EPI_RESID) && mrow) {
    dst_row = __ldg(p.idx + m);
    if (!row_ok(dst_row, p.N, p.flag)) dst_row = -1;
  }
  uint32_t ra[32], rb[32];
  __syncwarp();
  tmem_ld32_nowait(tbase, ra);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    uint32_t(&cur)[32] = (c & 1) ? rb : ra;
    uint32_t(&nxt)[32] = (c & 1) ? ra : rb;
    F2 sb[16];
    if (kS8) load_scales(p, n0 + 32 * c, sb);  // on their way while TMEM is waited for
    tmem_wait_ld();
    if (c + 1 < NC) {
      __syncwarp();
      tmem_ld32_nowait(tbase + 32 * (c + 1), nxt);
    }
    const int col = n0 + 32 * c;
    if (col >= p.Ncols) continue;  // uniform over the warp
    if (kS8) dequant_chunk(cur, sa, sb);
    if (kS8 && kEpi == EPI_STORE) {
      uint8_t* bytes = reinterpret_cast<uint8_t*>(stage);
      const int m0 = m - (threadIdx.x & 31);
      const bool last = c + 1 == NC || col + 32 >= p.Ncols;
      if (!(c & 1)) {  // the stage may still be on its way out
        if ((threadIdx.x & 31) == 0) tma_store_wait_read();
        __syncwarp();
      }
      stage_half(bytes, cur, c & 1);
      if ((p.ld_out & 7) != 0) {
        if ((c & 1) || last)
          store_ragged(p, bytes, m0, col - 32 * (c & 1), min(p.Ncols, col + 32));
      } else if (c & 1) {
        store_staged(tm_out, bytes, m0, col - 32);
      } else if (last) {
        store_half(p, bytes, m0, col);
      }
    } else if (kEpi == EPI_RESID) {
      resid_chunk(p, cur, dst_row, col, stage);
    } else if (mrow) {
      if (kEpi == EPI_STORE || kEpi == EPI_GELU) {
        store_bf16x32<kEpi == EPI_GELU>(p.out + static_cast<size_t>(m) * p.ld_out + col, cur);
      } else {  // EPI_QKV
        const int D = p.ld_out;
        const int which = col / D;
        const int cc = col - which * D;
        if (which == 0) {
          store_bf16x32<false>(p.out + static_cast<size_t>(m) * D + cc, cur);
        } else if (dst_row >= 0 && p.n_caches == 1) {
          __nv_bfloat16* cache = which == 1 ? p.kc[0] : p.vc[0];
          store_bf16x32<false>(cache + static_cast<size_t>(dst_row) * D + cc, cur);
        } else if (dst_row >= 0) {
          // the fresh row into every copy of this layer's cache (this GPU's,
          // and peers' when a sharded step writes them directly)
          uint4 w4[4];
          pack_bf16x32(cur, w4);
#pragma unroll
          for (int g = 0; g < kMaxCaches; ++g) {
            if (g >= p.n_caches) break;
            __nv_bfloat16* cache = which == 1 ? p.kc[g] : p.vc[g];
            uint4* d4 = reinterpret_cast<uint4*>(cache + static_cast<size_t>(dst_row) * D + cc);
            d4[0] = w4[0];
            d4[1] = w4[1];
            d4[2] = w4[2];
            d4[3] = w4[3];
          }
        }
      }
    }
  }
}

template <bool kS8, int kCols>
__device__ __forceinline__ void drain(const EpiParams& p, const CUtensorMap* tm_out, uint32_t tbase,
                                      int m, int n0, float sa, float* stage) {
  switch (p.epi) {
    case EPI_STORE: drain_tile<kS8, kCols, EPI_STORE>(p, tm_out, tbase, m, n0, sa, stage); break;
    case EPI_GELU: drain_tile<kS8, kCols, EPI_GELU>(p, tm_out, tbase, m, n0, sa, stage); break;
    case EPI_QKV: drain_tile<kS8, kCols, EPI_QKV>(p, tm_out, tbase, m, n0, sa, stage); break;
    case EPI_RESID: drain_tile<kS8, kCols, EPI_RESID>(p, tm_out, tbase, m, n0, sa, stage); break;
    default: break;
  }
}

// A K-block is 128 bytes of every operand row: 64 bf16 or 128 signed bytes.
// Either way it is four MMA steps of 32 bytes, so the two operand types share
// the tiles, the ring and the descriptors; 8-bit rows may end inside the last
// K-block (TMA fills the rest with zeros).
template <bool kS8>
__host__ __device__ constexpr int k_block() {
  return kS8 ? 2 * kBK : kBK;
}

template <bool kS8, int BN>
__global__ void __launch_bounds__(kGemmThreads, 1)
    k_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
           const __grid_constant__ CUtensorMap tmO, EpiParams p, int n_tiles, int total_tiles) {
  using Cfg = GemmCfg<BN>;
  constexpr int S = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + S * Cfg::kABytes;
  float* stage = reinterpret_cast<float*>(sB + S * Cfg::kBBytes);  // 1024-byte aligned
  uint64_t* full = reinterpret_cast<uint64_t*>(sB + S * Cfg::kBBytes + kEpiStageBytes);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;     // [2] accumulator buffer ready for the epilogue
  uint64_t* acc_empty = acc_full + 2; // [2] accumulator buffer drained
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kKB = k_block<kS8>();
  const int nk = (p.Kd + kKB - 1) / kKB;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kEpiWarps);  // one arrival per epilogue warp
    }
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, Cfg::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;

  // Tiles are visited t = blockIdx.x, +gridDim.x, ...; tile t covers rows
  // (t / n_tiles) * 128 and columns (t % n_tiles) * BN, so tiles running at the
  // same time share A row blocks and sweep the (L2-resident) weight.
  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      for (int t = blockIdx.x; t < total_tiles && ok; t += gridDim.x) {
        const int m0 = (t / n_tiles) * kBM, n0 = (t % n_tiles) * BN;
        for (int kb = 0; kb < nk; ++kb, ++it) {
          const int s = it % S;
          if (!mbar_wait(&empty[s], ((it / S) & 1) ^ 1)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], Cfg::kStageBytes);
          tma_load_2d(sA + s * Cfg::kABytes, &tmA, &full[s], kb * kKB, m0);
          tma_load_2d(sB + s * Cfg::kBBytes, &tmB, &full[s], kb * kKB, n0);
        }
      }
      if (!ok) {  // let copies already in flight land before the CTA exits
        for (int k = it > S ? it - S : 0; k < it; ++k) (void)mbar_wait(&full[k % S], (k / S) & 1);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc =
          kS8 ? idesc_s8(kBM, BN) : idesc_bf16(kBM, BN, false, false);
      int it = 0, lt = 0;
      for (int t = blockIdx.x; t < total_tiles && ok; t += gridDim.x, ++lt) {
        const int b = lt & 1;
        if (!mbar_wait(&acc_empty[b], ((lt >> 1) & 1) ^ 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t acc = tmem + b * BN;
        for (int kb = 0; kb < nk; ++kb, ++it) {
          const int s = it % S;
          if (!mbar_wait(&full[s], (it / S) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA + s * Cfg::kABytes);
          const uint32_t b0 = smem_u32(sB + s * Cfg::kBBytes);
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {
            const uint64_t ad = sdesc_sw128(a0 + kk * 32, 16, 1024);
            const uint64_t bd = sdesc_sw128(b0 + kk * 32, 16, 1024);
            if (kS8) umma_s8(acc, ad, bd, idesc, (kb > 0 || kk > 0) ? 1u : 0u);
            else umma_bf16(acc, ad, bd, idesc, (kb > 0 || kk > 0) ? 1u : 0u);
          }
          umma_commit(&empty[s]);
        }
        umma_commit(&acc_full[b]);
      }
    }
  } else {
    // epilogue: warp w reads TMEM lanes [32*(w%4), +32) = tile rows, and
    // column half (w - 2) / 4 of the tile
    const int q = warp & 3;
    const int half = (warp - 2) >> 2;
    const int row = 32 * q + lane;
    int lt = 0;
    for (int t = blockIdx.x; t < total_tiles; t += gridDim.x, ++lt) {
      const int b = lt & 1;
      const int m = (t / n_tiles) * kBM + row, n0 = (t % n_tiles) * BN + half * (BN / 2);
      const float sa = kS8 && m < p.M ? __ldg(p.a_scale + m) : 0.f;
      if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[b], (lt >> 1) & 1))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t tbase =
          tmem + b * BN + half * (BN / 2) + (static_cast<uint32_t>(32 * q) << 16);
      drain<kS8, BN / 2>(p, &tmO, tbase, m, n0, sa, stage + (warp - 2) * kStageWarpFloats);
      // the buffer may be refilled once every lane's TMEM reads are done
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[b]);
    }
    if (kS8 && lane == 0) tma_store_wait();  // rows in flight read this CTA's shared memory
  }
  if (!ok) atomicOr(p.flag, DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

// ------------------------------------------------------------ CTA-pair GEMM
// 256 x 256 output tiles computed by a cluster of two CTAs with one
// tcgen05.mma.cta_group::2 per K-step: each CTA stages its own 128 rows of A
// and one 128-row half of B, so a CTA moves half the B bytes of a 1-CTA
// 128 x 256 tile through shared memory for the same MMA work.  Rank 0 issues
// the MMAs; both CTAs load, and both run the epilogue on the 128 rows of the
// accumulator held in their own TMEM.

constexpr int kPairStages = 6;
constexpr int kPairABytes = 128 * kBK * 2;
constexpr int kPairBBytes = 128 * kBK * 2;
constexpr int kPairStageBytes = kPairABytes + kPairBBytes;
constexpr int kPairSmem = kPairStages * kPairStageBytes + 256 + kEpiStageBytes + 1024;

template <bool kS8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    k_gemm_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmO, EpiParams p, int n_tiles, int total_tiles) {
  constexpr int S = kPairStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + S * kPairABytes;
  float* stage = reinterpret_cast<float*>(sB + S * kPairBBytes);  // 1024-byte aligned
  uint64_t* full = reinterpret_cast<uint64_t*>(sB + S * kPairBBytes + kEpiStageBytes);  // used in rank 0
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;      // [2]
  uint64_t* acc_empty = acc_full + 2;  // [2], used in rank 0
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  constexpr int kKB = k_block<kS8>();
  const int nk = (p.Kd + kKB - 1) / kKB;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpiWarps);  // every epilogue warp of both CTAs
    }
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // both CTAs' barriers initialised and TMEM allocated
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      for (int t = pair; t < total_tiles && ok; t += npairs) {
        const int m0 = (t / n_tiles) * 256 + rank * 128, n0 = (t % n_tiles) * 256 + rank * 128;
        for (int kb = 0; kb < nk; ++kb, ++it) {
          const int s = it % S;
          if (!mbar_wait(&empty[s], ((it / S) & 1) ^ 1)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kPairStageBytes);
          const uint32_t lead = to_leader(smem_u32(&full[s]));
          tma_load_2d_pair(sA + s * kPairABytes, &tmA, lead, kb * kKB, m0);
          tma_load_2d_pair(sB + s * kPairBBytes, &tmB, lead, kb * kKB, n0);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc =
          kS8 ? idesc_s8(256, 256) : idesc_bf16(256, 256, false, false);
      int it = 0, lt = 0;
      for (int t = pair; t < total_tiles && ok; t += npairs, ++lt) {
        const int b = lt & 1;
        if (!mbar_wait<true>(&acc_empty[b], ((lt >> 1) & 1) ^ 1)) {  // both CTAs' epilogues
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t acc = tmem + b * 256;
        for (int kb = 0; kb < nk; ++kb, ++it) {
          const int s = it % S;
          if (!mbar_wait(&full[s], (it / S) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA + s * kPairABytes);
          const uint32_t b0 = smem_u32(sB + s * kPairBBytes);
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {
            const uint64_t ad = sdesc_sw128(a0 + kk * 32, 16, 1024);
            const uint64_t bd = sdesc_sw128(b0 + kk * 32, 16, 1024);
            if (kS8) umma_s8_pair(acc, ad, bd, idesc, (kb > 0 || kk > 0) ? 1u : 0u);
            else umma_bf16_pair(acc, ad, bd, idesc, (kb > 0 || kk > 0) ? 1u : 0u);
          }
          umma_commit_pair(&empty[s], 0x3);
        }
        umma_commit_pair(&acc_full[b], 0x3);
      }
    }
  } else {
    const int q = warp & 3;
    const int half = (warp - 2) >> 2;  // column half of the tile
    const int row = 32 * q + lane;
    const uint32_t lead_empty0 = to_leader(smem_u32(&acc_empty[0]));
    const uint32_t lead_empty1 = to_leader(smem_u32(&acc_empty[1]));
    int lt = 0;
    for (int t = pair; t < total_tiles; t += npairs, ++lt) {
      const int b = lt & 1;
      const int m = (t / n_tiles) * 256 + rank * 128 + row, n0 = (t % n_tiles) * 256 + half * 128;
      const float sa = kS8 && m < p.M ? __ldg(p.a_scale + m) : 0.f;
      if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[b], (lt >> 1) & 1))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t tbase = tmem + b * 256 + half * 128 + (static_cast<uint32_t>(32 * q) << 16);
      drain<kS8, 128>(p, &tmO, tbase, m, n0, sa, stage + (warp - 2) * kStageWarpFloats);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (kS8) mbar_arrive_cluster_tmem(b == 0 ? lead_empty0 : lead_empty1);
        else mbar_arrive_cluster(b == 0 ? lead_empty0 : lead_empty1);
      }
    }
    if (kS8 && lane == 0) tma_store_wait();  // rows in flight read this CTA's shared memory
  }
  if (!ok) atomicOr(p.flag, DEV_TIMEOUT);
  tc_fence_before();
  cluster_sync();  // no CTA leaves while its peer may still signal its barriers
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// The caches an EPI_QKV launch writes: the list when one is given, else the pair.
void set_caches(EpiParams& p, const GemmArgs& a) {
  if (a.n_caches > 0) {
    p.n_caches = a.n_caches;
    for (int g = 0; g < a.n_caches; ++g) {
      p.kc[g] = static_cast<__nv_bfloat16*>(a.k_caches[g]);
      p.vc[g] = static_cast<__nv_bfloat16*>(a.v_caches[g]);
    }
  } else {
    p.n_caches = 1;
    p.kc[0] = static_cast<__nv_bfloat16*>(a.k_cache);
    p.vc[0] = static_cast<__nv_bfloat16*>(a.v_cache);
  }
}

static_assert(kPairSmem <= 227 * 1024, "CTA-pair GEMM exceeds the shared memory of a CTA");
static_assert(GemmCfg<256>::kSmem <= 227 * 1024 && GemmCfg<192>::kSmem <= 227 * 1024 &&
                  GemmCfg<128>::kSmem <= 227 * 1024,
              "GEMM tile exceeds the shared memory of a CTA");

EpiParams epi_params(const Ctx& c, const GemmArgs& a) {
  EpiParams p{};
  p.M = a.M;
  p.Ncols = a.Ncols;
  p.Kd = a.Kd;
  p.epi = a.epi;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.ld_out = a.ld_out;
  set_caches(p, a);
  p.x = a.x;
  p.ld_x = a.ld_x;
  p.gate = a.gate;
  p.idx = a.idx;
  p.N = a.N;
  p.flag = c.flag;
  p.a_scale = a.a_scale;
  p.b_scale = a.b_scale;
  return p;
}

// Operand maps with boxes of box_a and box_b rows of one K-block, and for 8-bit
// operands the map of an aligned plain output (else unused).
template <bool kS8>
bool operand_maps(const GemmArgs& a, uint32_t box_a, uint32_t box_b, CUtensorMap* ta,
                  CUtensorMap* tb, CUtensorMap* to, std::string* why) {
  if (kS8) {
    if (!make_tmap_s8(ta, a.A, a.M, a.Kd, a.ld_a, box_a, why) ||
        !make_tmap_s8(tb, a.B, a.Ncols, a.Kd, a.ld_b, box_b, why))
      return false;
    *to = *ta;
    return a.epi != EPI_STORE || a.ld_out % 8 != 0 ||
           make_tmap_bf16(to, a.out, a.M, a.Ncols, a.ld_out, 32, why);
  }
  const bool made = make_tmap_bf16(ta, a.A, a.M, a.Kd, a.Kd, box_a, why) &&
                    make_tmap_bf16(tb, a.B, a.Ncols, a.Kd, a.Kd, box_b, why);
  *to = *ta;
  return made;
}

template <bool kS8>
cudaError_t launch_pair(const Ctx& c, const GemmArgs& a, std::string* why) {
  CUtensorMap ta, tb, to;
  if (!operand_maps<kS8>(a, 128, 128, &ta, &tb, &to, why)) return cudaErrorInvalidValue;
  const EpiParams p = epi_params(c, a);
  static std::atomic<uint64_t> smem_set{0};  // per device
  {
    const cudaError_t e = ensure_smem_limit(k_gemm_pair<kS8>, kPairSmem, c.device, smem_set);
    if (e != cudaSuccess) return e;
  }
  const int n_tiles = (a.Ncols + 255) / 256;
  const int total = n_tiles * ((a.M + 255) / 256);
  const int pairs = total < c.num_sms / 2 ? total : c.num_sms / 2;
  k_gemm_pair<kS8><<<2 * pairs, kGemmThreads, kPairSmem, c.stream>>>(ta, tb, to, p, n_tiles, total);
  c.launches += 1;
  return cudaGetLastError();
}

template <bool kS8, int BN>
cudaError_t launch_bn(const Ctx& c, const GemmArgs& a, std::string* why) {
  CUtensorMap ta, tb, to;
  if (!operand_maps<kS8>(a, kBM, BN, &ta, &tb, &to, why)) return cudaErrorInvalidValue;
  const EpiParams p = epi_params(c, a);
  constexpr int smem = GemmCfg<BN>::kSmem;
  static std::atomic<uint64_t> smem_set{0};  // per device
  {
    const cudaError_t e = ensure_smem_limit(k_gemm<kS8, BN>, smem, c.device, smem_set);
    if (e != cudaSuccess) return e;
  }
  const int n_tiles = (a.Ncols + BN - 1) / BN;
  const int total = n_tiles * ((a.M + kBM - 1) / kBM);
  const int grid = total < c.num_sms ? total : c.num_sms;
  k_gemm<kS8, BN><<<grid, kGemmThreads, smem, c.stream>>>(ta, tb, to, p, n_tiles, total);
  c.launches += 1;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gemm(const Ctx& c, const GemmArgs& a, std::string* why) {
  if (a.M <= 0) return cudaSuccess;
  Timed timed(c, TC_GEMM, 2.0 * a.M * a.Ncols * a.Kd);
  if (a.Kd % kBK != 0 || a.Ncols % 32 != 0) {
    if (why) *why = "GEMM needs K % 64 == 0 and Ncols % 32 == 0";
    return cudaErrorInvalidValue;
  }
  // Pick the tile width with the fewest tile-waves x tile width, where a
  // narrower tile costs a little more per column (more smem traffic per FLOP).
  const int mt = (a.M + kBM - 1) / kBM;
  auto cost = [&](int bn, double per_col) {
    const long tiles = static_cast<long>(mt) * ((a.Ncols + bn - 1) / bn);
    const long waves = (tiles + c.num_sms - 1) / c.num_sms;
    return static_cast<double>(waves) * bn * per_col;
  };
  double best = 1e300;
  int bn = 128;
  // CTA pairs: 256 x 256 tiles over SMs/2 pairs, about 0.8x the cost per output
  // element of a 1-CTA 256-wide tile (half the B traffic through shared memory)
  if (a.Ncols % 256 == 0 && a.M >= 256) {
    const int mt2 = (a.M + 255) / 256;
    const long tiles2 = static_cast<long>(mt2) * (a.Ncols / 256);
    const int pairs = c.num_sms / 2;
    // a pair tile is the same work per SM as a 1-CTA 128 x 256 tile
    const double pc = static_cast<double>((tiles2 + pairs - 1) / pairs) * 256 * kPairCost;
    if (pc < best) best = pc, bn = -1;
  }
  if (a.Ncols % 256 == 0 && cost(256, 1.0) < best) best = cost(256, 1.0), bn = 256;
  if (a.Ncols % 192 == 0 && cost(192, 1.03) < best) best = cost(192, 1.03), bn = 192;
  if (cost(128, 1.12) < best) best = cost(128, 1.12), bn = 128;
  if (bn == -1) return launch_pair<false>(c, a, why);
  if (bn == 256) return launch_bn<false, 256>(c, a, why);
  if (bn == 192) return launch_bn<false, 192>(c, a, why);
  return launch_bn<false, 128>(c, a, why);
}

cudaError_t launch_gemm_s8(const Ctx& c, const GemmArgs& a, std::string* why) {
  if (a.M <= 0) return cudaSuccess;
  if (a.epi == EPI_STORE) {
    bool taken = false;
    const cudaError_t e = launch_linear_s8_few(c, a, &taken, why);
    if (taken) return e;
  }
  Timed timed(c, TC_GEMM, 2.0 * a.M * a.Ncols * a.Kd);
  // As above, by tile-waves x tile width; columns may end inside a tile.
  const int mt = (a.M + kBM - 1) / kBM;
  auto cost = [&](int bn, double per_col) {
    const long tiles = static_cast<long>(mt) * ((a.Ncols + bn - 1) / bn);
    return static_cast<double>((tiles + c.num_sms - 1) / c.num_sms) * bn * per_col;
  };
  double best = 1e300;
  int bn = 128;
  if (a.Ncols >= 256 && a.M >= 256) {
    const long tiles = static_cast<long>((a.M + 255) / 256) * ((a.Ncols + 255) / 256);
    const int pairs = c.num_sms / 2;
    // (0.75: 700 x 5000 x 8000 takes 46 us in pairs, 54 in 192-wide tiles)
    best = static_cast<double>((tiles + pairs - 1) / pairs) * 256 * 0.75, bn = -1;
  }
  if (cost(256, 1.0) < best) best = cost(256, 1.0), bn = 256;
  if (cost(192, 1.03) < best) best = cost(192, 1.03), bn = 192;
  if (cost(128, 1.12) < best) best = cost(128, 1.12), bn = 128;
  if (bn == -1) return launch_pair<true>(c, a, why);
  if (bn == 256) return launch_bn<true, 256>(c, a, why);
  if (bn == 192) return launch_bn<true, 192>(c, a, why);
  return launch_bn<true, 128>(c, a, why);
}

}  // namespace hsa
