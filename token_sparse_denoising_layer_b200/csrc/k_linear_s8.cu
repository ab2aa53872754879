// k_linear_s8.cu - 8-bit products of few rows, which the tiles of k_gemm.cu
// leave most of the GPU out of:
//   out[m, j] = a_scale[m] w_scale[j] sum_k a[m, k] w[j, k]
// The sums are exact integers, so splitting K over lanes or CTAs changes no result.
//
//  - Up to kVecRows rows (single tokens): the weights are streamed once and
//    nothing is reused, so this is a matter of bytes in flight.  A warp owns
//    two weight rows and its lanes stride over K in 16-byte vectors, four-way
//    byte dot products against the rows of a (L1-resident).
//  - A few tiles of rows: a 128 x 64 tensor-core tile per CTA and, while CTAs
//    are left over, K split over a cluster of up to 8, whose CTAs add up
//    each other's accumulators through distributed shared memory.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <string>

#include "internal.h"
#include "ptx.cuh"

namespace hsa {

namespace {

// ------------------------------------------------------------ single tokens
constexpr int kVecCols = 2;  // weight rows per warp
constexpr int kVecWarps = 8;

struct VecParams {
  const int8_t* a;
  const int8_t* w;
  int64_t ld_a, ld_w;
  const float *a_scale, *w_scale;
  __nv_bfloat16* out;
  int Ncols, Kd;
};

__device__ __forceinline__ int dot16(const uint4& x, const uint4& y, int acc) {
  acc = __dp4a(static_cast<int>(x.x), static_cast<int>(y.x), acc);
  acc = __dp4a(static_cast<int>(x.y), static_cast<int>(y.y), acc);
  acc = __dp4a(static_cast<int>(x.z), static_cast<int>(y.z), acc);
  return __dp4a(static_cast<int>(x.w), static_cast<int>(y.w), acc);
}

// The first `left` bytes of a vector, the others zero.
__device__ __forceinline__ uint4 first_bytes(uint4 v, int left) {
  uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = left - 4 * i;
    if (n <= 0) r[i] = 0u;
    else if (n < 4) r[i] &= (1u << (8 * n)) - 1u;
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

template <int MR>
__global__ void __launch_bounds__(32 * kVecWarps) k_vec_s8(const __grid_constant__ VecParams p) {
  const int lane = threadIdx.x & 31;
  const int j0 = (blockIdx.x * kVecWarps + (threadIdx.x >> 5)) * kVecCols;
  if (j0 >= p.Ncols) return;
  const int8_t* w0 = p.w + j0 * p.ld_w;
  const int8_t* w1 = j0 + 1 < p.Ncols ? w0 + p.ld_w : w0;
  int acc[MR][kVecCols];
#pragma unroll
  for (int m = 0; m < MR; ++m) acc[m][0] = acc[m][1] = 0;
#pragma unroll 4
  for (int e = 16 * lane; e < p.Kd; e += 512) {
    const uint4 x0 = __ldg(reinterpret_cast<const uint4*>(w0 + e));
    const uint4 x1 = __ldg(reinterpret_cast<const uint4*>(w1 + e));
    const int left = p.Kd - e;
#pragma unroll
    for (int m = 0; m < MR; ++m) {
      uint4 y = __ldg(reinterpret_cast<const uint4*>(p.a + m * p.ld_a + e));
      if (left < 16) y = first_bytes(y, left);  // what lies past a row, in a or w, adds nothing
      acc[m][0] = dot16(x0, y, acc[m][0]);
      acc[m][1] = dot16(x1, y, acc[m][1]);
    }
  }
#pragma unroll
  for (int m = 0; m < MR; ++m) {
#pragma unroll
    for (int c = 0; c < kVecCols; ++c) {
      const int sum = __reduce_add_sync(0xffffffffu, acc[m][c]);
      if (lane == c && j0 + c < p.Ncols)
        p.out[static_cast<int64_t>(m) * p.Ncols + j0 + c] =
            __float2bfloat16_rn(__int2float_rn(sum) * __ldg(p.a_scale + m) * __ldg(p.w_scale + j0 + c));
    }
  }
}

// ------------------------------------------------------------ few tiles
constexpr int kBM = 128, kBN = 64, kKB = 128;  // tile, and bytes of K per block
constexpr int kStages = 6;
constexpr int kThreads = 192;  // TMA warp, MMA warp, 4 epilogue warps
constexpr int kABytes = kBM * kKB, kBBytes = kBN * kKB, kBlockBytes = kABytes + kBBytes;
constexpr int kAccPitch = kBN + 4;  // words: rows 16 bytes off each other in the banks
constexpr int kSmem = kStages * kBlockBytes + kBM * kAccPitch * 4 + 256 + 1024;
constexpr uint32_t kTmemCols = 64;

struct TileParams {
  int M, Ncols, nk, n_tiles, split;
  const float *a_scale, *w_scale;
  __nv_bfloat16* out;
  int* flag;
};

// 16 bytes of the same shared-memory place in CTA `rank` of the cluster.
__device__ __forceinline__ int4 ld_cluster(uint32_t saddr, uint32_t rank) {
  int4 v;
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(saddr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

__global__ void __launch_bounds__(kThreads, 1)
    k_tile_s8(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
              const __grid_constant__ TileParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + kStages * kABytes;
  int* acc = reinterpret_cast<int*>(smem + kStages * kBlockBytes);  // [128][kAccPitch]
  uint64_t* full = reinterpret_cast<uint64_t*>(acc + kBM * kAccPitch);
  uint64_t* empty = full + kStages;
  uint64_t* done = empty + kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = blockIdx.x / p.split, rank = blockIdx.x % p.split;  // a cluster is one tile
  const int m0 = tile / p.n_tiles * kBM, n0 = tile % p.n_tiles * kBN;
  const int kb0 = rank * p.nk / p.split, kb1 = (rank + 1) * p.nk / p.split;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % kStages;
        if (!mbar_wait(&empty[s], ((it / kStages) & 1) ^ 1)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&full[s], kBlockBytes);
        tma_load_2d(sA + s * kABytes, &tmA, &full[s], kb * kKB, m0);
        tma_load_2d(sB + s * kBBytes, &tmB, &full[s], kb * kKB, n0);
      }
      if (!ok)  // let copies already in flight land before the CTA exits
        for (int k = it > kStages ? it - kStages : 0; k < it; ++k)
          (void)mbar_wait(&full[k % kStages], (k / kStages) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_s8(kBM, kBN);
      int it = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % kStages;
        if (!mbar_wait(&full[s], (it / kStages) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a0 = smem_u32(sA + s * kABytes), b0 = smem_u32(sB + s * kBBytes);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_s8(tmem, sdesc_sw128(a0 + kk * 32, 16, 1024), sdesc_sw128(b0 + kk * 32, 16, 1024),
                  idesc, (it > 0 || kk > 0) ? 1u : 0u);
        umma_commit(&empty[s]);
      }
      umma_commit(done);
    }
  } else {
    // this warp's 32 rows of the accumulator into shared memory
    const int q = warp & 3, row = 32 * q + lane;
    if (__all_sync(0xffffffffu, mbar_wait(done, 0))) {
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kBN / 32; ++c) {
        uint32_t r[32];
        tmem_ld32(tmem + (static_cast<uint32_t>(32 * q) << 16) + 32 * c, r);
#pragma unroll
        for (int v = 0; v < 8; ++v)
          *reinterpret_cast<uint4*>(acc + row * kAccPitch + 32 * c + 4 * v) =
              make_uint4(r[4 * v], r[4 * v + 1], r[4 * v + 2], r[4 * v + 3]);
      }
    } else {
      ok = false;
    }
  }
  if (!ok) atomicOr(p.flag, DEV_TIMEOUT);
  tc_fence_before();
  cluster_sync();  // every CTA's sums are in its shared memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  // this CTA's share of the rows: sums of all ranks, scaled and stored, four columns a thread
  const int r0 = rank * kBM / p.split, r1 = (rank + 1) * kBM / p.split;
  const bool vec = (p.Ncols & 3) == 0;
  for (int i = threadIdx.x; i < (r1 - r0) * (kBN / 4); i += kThreads) {
    const int row = r0 + i / (kBN / 4), col = 4 * (i % (kBN / 4));
    const int m = m0 + row, n = n0 + col;
    if (m >= p.M || n >= p.Ncols) continue;
    const uint32_t at = smem_u32(acc + row * kAccPitch + col);
    int4 sum = make_int4(0, 0, 0, 0);
    for (int k = 0; k < p.split; ++k) {
      const int4 v = ld_cluster(at, k);
      sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
    }
    const float sa = __ldg(p.a_scale + m);
    __nv_bfloat16* dst = p.out + static_cast<int64_t>(m) * p.Ncols + n;
    const int s[4] = {sum.x, sum.y, sum.z, sum.w};
    float f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      f[e] = n + e < p.Ncols ? __int2float_rn(s[e]) * sa * __ldg(p.w_scale + n + e) : 0.f;
    if (vec) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < p.Ncols) dst[e] = __float2bfloat16_rn(f[e]);
    }
  }
  cluster_sync();  // no CTA leaves while another may read its sums
}

}  // namespace

cudaError_t launch_linear_s8_few(const Ctx& c, const GemmArgs& a, bool* taken, std::string* why) {
  *taken = false;
  const auto* A = static_cast<const int8_t*>(a.A);
  const auto* B = static_cast<const int8_t*>(a.B);
  auto* out = static_cast<__nv_bfloat16*>(a.out);
  // Beyond this a warp's walk over K (0.4 us per 512 bytes and pair of rows)
  // takes longer than the tile kernel's 10 us.  K = 1536, N = 8960: 3.2 us for one
  // row, 4.9 for four, tiles 10; K = 8960, N = 1536: 7.4, 19, tiles 10.
  if (a.M <= kVecRows && a.M * static_cast<int64_t>(a.Kd) <= 16384) {
    *taken = true;
    Timed timed(c, TC_GEMM, 2.0 * a.M * a.Ncols * a.Kd);
    const VecParams p{A, B, a.ld_a, a.ld_b, a.a_scale, a.b_scale, out, a.Ncols, a.Kd};
    const int per = kVecCols * kVecWarps;
    const unsigned grid = (a.Ncols + per - 1) / per;
    if (a.M == 1) k_vec_s8<1><<<grid, 32 * kVecWarps, 0, c.stream>>>(p);
    else if (a.M == 2) k_vec_s8<2><<<grid, 32 * kVecWarps, 0, c.stream>>>(p);
    else if (a.M == 3) k_vec_s8<3><<<grid, 32 * kVecWarps, 0, c.stream>>>(p);
    else k_vec_s8<kVecRows><<<grid, 32 * kVecWarps, 0, c.stream>>>(p);
    c.launches += 1;
    return cudaGetLastError();
  }
  const int nk = (a.Kd + kKB - 1) / kKB;
  const int64_t tiles = static_cast<int64_t>((a.M + kBM - 1) / kBM) * ((a.Ncols + kBN - 1) / kBN);
  if (tiles > c.num_sms) return cudaSuccess;
  *taken = true;
  Timed timed(c, TC_GEMM, 2.0 * a.M * a.Ncols * a.Kd);
  // the largest cluster that leaves each CTA two K-blocks and all of them an SM
  int split = 1;
  while (2 * split <= 8 && tiles * 2 * split <= c.num_sms && nk >= 4 * split) split *= 2;
  CUtensorMap ta, tb;
  if (!make_tmap_s8(&ta, a.A, a.M, a.Kd, a.ld_a, kBM, why) ||
      !make_tmap_s8(&tb, a.B, a.Ncols, a.Kd, a.ld_b, kBN, why))
    return cudaErrorInvalidValue;
  TileParams p{};
  p.M = a.M;
  p.Ncols = a.Ncols;
  p.nk = nk;
  p.n_tiles = (a.Ncols + kBN - 1) / kBN;
  p.split = split;
  p.a_scale = a.a_scale;
  p.w_scale = a.b_scale;
  p.out = out;
  p.flag = c.flag;
  static std::atomic<uint64_t> smem_set{0};  // per device
  cudaError_t e = ensure_smem_limit(k_tile_s8, kSmem, c.device, smem_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k_tile_s8, ta, tb, p);
  c.launches += 1;
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace hsa
