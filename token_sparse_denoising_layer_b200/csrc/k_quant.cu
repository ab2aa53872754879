// k_quant.cu - rows quantised to signed 8 bits with one fp32 scale each, the
// left operand of the 8-bit products (k_gemm.cu).
//
//   top = max_k |a[m, k]|,  scale[m] = top / 127,  q[m, k] = rint(a[m, k] * (127 / top))
// in fp32, round half to even.  |q| <= 127: a * (127 / top) is at most 127
// times two roundings of 2^-24 each.  Rows with top < 2^-100 become zeros with
// scale 0 (127 / top would leave the fp32 range); a row that holds an
// infinity or a NaN becomes zeros with scale NaN, so that its products show it.
//
// Bound by HBM: a row is read once into registers, reduced, and written.  A
// row is owned by a warp, or by 128 or 512 threads when a warp's registers
// would not hold it.  What covers the latency is rows in flight, so the register count is
// capped to what lets seven blocks of 128 threads share an SM.  32760 rows of bf16:
// K = 1536 27 us (5.5 TB/s), K = 8960 128 us (6.9 TB/s; 141 with five blocks, 185
// with 256 threads a row).

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"

namespace hsa {

namespace {

constexpr uint32_t kInfBits = 0x7f800000u;
constexpr float kTinyTop = 7.888609052210118e-31f;  // 2^-100

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// (multiplier, scale) of a row from the bit pattern of its largest magnitude;
// patterns of non-negative floats order as the floats do, NaN above infinity.
__device__ __forceinline__ float2 row_scales(uint32_t top_bits) {
  if (top_bits >= kInfBits) return make_float2(0.f, __uint_as_float(0x7fc00000u));
  const float top = __uint_as_float(top_bits);
  if (top < kTinyTop) return make_float2(0.f, 0.f);
  return make_float2(__fdiv_rn(127.0f, top), __fdiv_rn(top, 127.0f));
}

// Four values -> four signed bytes, round half to even: the product is rounded
// to fp32 by itself (__fmul_rn: a packed product was contracted into the add,
// which rounds once), then adding 1.5 * 2^23 leaves its integer in the low
// bits.  Float-to-integer conversions run at a quarter of that rate.  Not for a
// row whose multiplier is 0, where an infinity or a NaN may stand.
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d, float mul) {
  const F2 round = splat(12582912.0f);
  const F2 x = add_x2(F2{__fmul_rn(a, mul), __fmul_rn(b, mul)}, round);
  const F2 y = add_x2(F2{__fmul_rn(c, mul), __fmul_rn(d, mul)}, round);
  return __byte_perm(__byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x0040),
                     __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x0040), 0x5410);
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

// Maximum over the TH threads that share a row (one warp, or a whole block).
template <int TH>
__device__ __forceinline__ uint32_t row_top(uint32_t v) {
  v = warp_max(v);
  if (TH == 32) return v;
  __shared__ uint32_t part[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) part[warp] = v;
  __syncthreads();
  return warp_max(lane < TH / 32 ? part[lane] : 0u);
}

// 8 source values as loaded: one 16-byte vector of bf16, two of fp32; fewer at
// a row's end, where nothing past the row is read.
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 w;
  __device__ void load(const __nv_bfloat16* p, int left) {
    if (left >= 8) {
      w = *reinterpret_cast<const uint4*>(p);
      return;
    }
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
    uint32_t r[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < left) r[i >> 1] |= static_cast<uint32_t>(h[i]) << (16 * (i & 1));
    w = make_uint4(r[0], r[1], r[2], r[3]);
  }
  __device__ void zero() { w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ void get(float (&f)[8]) const {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(r[i] << 16);
      f[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ void load(const float* p, int left) {
    if (left >= 8) {
      a = reinterpret_cast<const float4*>(p)[0];
      b = reinterpret_cast<const float4*>(p)[1];
      return;
    }
    a = make_float4(left > 0 ? p[0] : 0.f, left > 1 ? p[1] : 0.f, left > 2 ? p[2] : 0.f,
                    left > 3 ? p[3] : 0.f);
    b = make_float4(left > 4 ? p[4] : 0.f, left > 5 ? p[5] : 0.f, left > 6 ? p[6] : 0.f, 0.f);
  }
  __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
};

__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(float v) { return v; }

// 256-thread blocks of 8 rows (TH = 32), or one row per block of TH threads;
// NC vectors of 8 per thread.  Needs 16-byte aligned rows.  q may lie over a
// (each row's bytes inside its own source row): a row is in registers before
// its first byte is written.
template <typename T, int TH, int NC>
__global__ void __launch_bounds__(TH == 32 ? 256 : TH, TH == 32 ? 4 : TH == 128 ? 7 : 1)
    k_quant_rows(const T* a, int64_t ld_a, int n, int Kd, int8_t* q, int64_t ld_q, float* scale) {
  const int m = TH == 32 ? blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
  if (m >= n) return;
  const int t = TH == 32 ? threadIdx.x & 31 : threadIdx.x;
  const T* row = a + m * ld_a;
  Vec8<T> v[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int e = 8 * (t + c * TH);
    v[c].load(row + e, Kd - e);
  }
  uint32_t top = 0u;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float f[8];
    v[c].get(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, abs_bits(f[i]));
  }
  const float2 s = row_scales(row_top<TH>(top));
  if (t == 0) scale[m] = s.y;
  int8_t* out = q + m * ld_q;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int e = 8 * (t + c * TH);
    float f[8];
    v[c].get(f);
    const uint32_t lo = s.x == 0.f ? 0u : quant4(f[0], f[1], f[2], f[3], s.x);
    const uint32_t hi = s.x == 0.f ? 0u : quant4(f[4], f[5], f[6], f[7], s.x);
    if (e + 8 <= Kd) {
      *reinterpret_cast<uint2*>(out + e) = make_uint2(lo, hi);
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (e + i < Kd) out[e + i] = static_cast<int8_t>((i < 4 ? lo >> (8 * i) : hi >> (8 * (i - 4))) & 0xffu);
    }
  }
}

// Rows that start anywhere (an odd Kd, a column block): W warps a row (8 rows of
// one warp, or one row, per block), NC vectors a lane.  Loads stay whole by starting from the
// aligned address `skip` values before the row, inside the row before it; each
// vector's 8 bytes are then joined with those of the next (the next lane's, or
// the next step's first lane's) and shifted by `skip`, as q's rows are aligned.
// A warp's last vector only lends its bytes: segments advance by 32 NC - 1
// vectors.  20000 x 1001 bf16: 17 us, 38 with 2-byte loads (20000 x 1000: 13).
template <typename T, int W, int NC>
__global__ void __launch_bounds__(W == 1 ? 256 : 32 * W)
    k_quant_rows_shift(const T* a, int64_t ld_a, int n, int Kd, int8_t* q, int64_t ld_q, float* scale) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int m = W == 1 ? blockIdx.x * 8 + warp : blockIdx.x;
  if (m >= n) return;
  const T* row = a + m * ld_a;
  const int skip = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  const int v0 = W == 1 ? 0 : warp * (32 * NC - 1);
  Vec8<T> v[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if (c > 0 && 8 * (v0 + 32 * c) - skip >= Kd) {  // the row ends before this step
      v[c].zero();
      continue;
    }
    const int at = 8 * (v0 + lane + 32 * c) - skip;  // place of the vector's first value in the row
    v[c].load(row + at, Kd - at);
  }
  const int before = v0 + lane == 0 ? skip : 0;  // values of the first vector that are not the row's
  uint32_t top = 0u;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float f[8];
    v[c].get(f);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c > 0 || i >= before) top = max(top, abs_bits(f[i]));
  }
  const float2 s = row_scales(row_top<32 * W>(top));
  if (lane == 0 && (W == 1 || warp == 0)) scale[m] = s.y;
  uint32_t w[NC][2];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    w[c][0] = w[c][1] = 0u;
    if (c > 0 && 8 * (v0 + 32 * c) - skip >= Kd) continue;
    float f[8];
    v[c].get(f);
    w[c][0] = s.x == 0.f ? 0u : quant4(f[0], f[1], f[2], f[3], s.x);
    w[c][1] = s.x == 0.f ? 0u : quant4(f[4], f[5], f[6], f[7], s.x);
  }
  int8_t* out = q + m * ld_q;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if (8 * (v0 + 32 * c) >= Kd) break;
    uint32_t next = __shfl_down_sync(0xffffffffu, w[c][0], 1);
    uint32_t next2 = __shfl_down_sync(0xffffffffu, w[c][1], 1);
    if (c + 1 < NC) {
      const uint32_t x = __shfl_sync(0xffffffffu, w[c + 1 < NC ? c + 1 : c][0], 0);
      const uint32_t y = __shfl_sync(0xffffffffu, w[c + 1 < NC ? c + 1 : c][1], 0);
      if (lane == 31) next = x, next2 = y;
    } else if (lane == 31) {
      continue;
    }
    const bool far = skip >= 4;
    const uint32_t x = far ? w[c][1] : w[c][0], y = far ? next : w[c][1], z = far ? next2 : next;
    const uint32_t lo = __funnelshift_r(x, y, 8 * (skip & 3)), hi = __funnelshift_r(y, z, 8 * (skip & 3));
    const int e = 8 * (v0 + lane + 32 * c);
    if (e + 8 <= Kd) {
      *reinterpret_cast<uint2*>(out + e) = make_uint2(lo, hi);
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (e + i < Kd) out[e + i] = static_cast<int8_t>((i < 4 ? lo >> (8 * i) : hi >> (8 * (i - 4))) & 0xffu);
    }
  }
}

// Rows of any alignment or length: two passes, the second served by L1 / L2.
template <typename T>
__global__ void __launch_bounds__(256) k_quant_rows_any(const T* __restrict__ a, int64_t ld_a,
                                                        int n, int Kd, int8_t* __restrict__ q,
                                                        int64_t ld_q, float* __restrict__ scale) {
  const int m = blockIdx.x;
  const T* row = a + m * ld_a;
  uint32_t top = 0u;
  for (int e = threadIdx.x; e < Kd; e += 256) top = max(top, abs_bits(to_f(row[e])));
  const float2 s = row_scales(row_top<256>(top));
  if (threadIdx.x == 0) scale[m] = s.y;
  int8_t* out = q + m * ld_q;
  for (int e = threadIdx.x; e < Kd; e += 256)
    out[e] = static_cast<int8_t>(__float2int_rn(__fmul_rn(to_f(row[e]), s.x)));
}

// ------------------------------------------------------------ LN + quantisation
__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

constexpr float kLnQuantEps = 1e-5f;  // the LayerNorm of k_rows.cu

// One active row per warp: u = LN(x[idx[m]]) (1 + mscale) + shift in fp32,
// quantised without a 16-bit stop in between.  NCH float4 per lane; the
// statistics are two-pass over registers.  D <= 128 NCH, any multiple of 128.
template <int NCH>
__global__ void __launch_bounds__(256) k_ln_gather_quant(const float* __restrict__ x,
                                                         const int32_t* __restrict__ idx, int n,
                                                         int N, int D, int8_t* __restrict__ q,
                                                         float* __restrict__ scale, int* flag,
                                                         const float* __restrict__ shift,
                                                         const float* __restrict__ mscale) {
  const int m = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (m >= n) return;
  const int r = __ldg(idx + m);
  uint32_t* out = reinterpret_cast<uint32_t*>(q + static_cast<int64_t>(m) * D);
  const int nv = D / 4;
  if (!row_ok(r, N, flag)) {
    for (int c = lane; c < nv; c += 32) out[c] = 0u;
    if (lane == 0) scale[m] = 0.f;
    return;
  }
  const float4* xr = reinterpret_cast<const float4*>(x + static_cast<int64_t>(r) * D);
  float4 v[NCH];
#pragma unroll
  for (int c = 0; c < NCH; ++c)
    v[c] = c * 32 + lane < nv ? __ldg(xr + c * 32 + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < NCH; ++c) s += (v[c].x + v[c].y) + (v[c].z + v[c].w);
  const float mean = warp_add(s) / static_cast<float>(D);
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    if (c * 32 + lane < nv) {
      const float a = v[c].x - mean, b = v[c].y - mean, e = v[c].z - mean, f = v[c].w - mean;
      ss += (a * a + b * b) + (e * e + f * f);
    }
  }
  const float rstd = 1.0f / sqrtf(warp_add(ss) / static_cast<float>(D) + kLnQuantEps);
  uint32_t top = 0u;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    if (c * 32 + lane < nv) {
      float4 y = make_float4((v[c].x - mean) * rstd, (v[c].y - mean) * rstd, (v[c].z - mean) * rstd,
                             (v[c].w - mean) * rstd);
      if (mscale != nullptr) {
        const float4 sc = __ldg(reinterpret_cast<const float4*>(mscale) + c * 32 + lane);
        const float4 sh = __ldg(reinterpret_cast<const float4*>(shift) + c * 32 + lane);
        y = make_float4(fmaf(y.x, 1.f + sc.x, sh.x), fmaf(y.y, 1.f + sc.y, sh.y),
                        fmaf(y.z, 1.f + sc.z, sh.z), fmaf(y.w, 1.f + sc.w, sh.w));
      }
      v[c] = y;
      top = max(max(max(top, abs_bits(y.x)), abs_bits(y.y)), max(abs_bits(y.z), abs_bits(y.w)));
    }
  }
  const float2 sc = row_scales(warp_max(top));
  if (lane == 0) scale[m] = sc.y;
#pragma unroll
  for (int c = 0; c < NCH; ++c)
    if (c * 32 + lane < nv)
      out[c * 32 + lane] = sc.x == 0.f ? 0u : quant4(v[c].x, v[c].y, v[c].z, v[c].w, sc.x);
}

template <typename T, int TH>
void quant_threads(const Ctx& c, const T* a, int64_t ld_a, int n, int Kd, int8_t* q, int64_t ld_q,
                   float* scale) {
  const int need = ((Kd + 7) / 8 + TH - 1) / TH;  // vectors per thread
  const unsigned grid = TH == 32 ? (n + 7) / 8 : n;
  const int threads = TH == 32 ? 256 : TH;
  if (need <= 2) k_quant_rows<T, TH, 2><<<grid, threads, 0, c.stream>>>(a, ld_a, n, Kd, q, ld_q, scale);
  else if (need <= 4) k_quant_rows<T, TH, 4><<<grid, threads, 0, c.stream>>>(a, ld_a, n, Kd, q, ld_q, scale);
  else if (need <= 6) k_quant_rows<T, TH, 6><<<grid, threads, 0, c.stream>>>(a, ld_a, n, Kd, q, ld_q, scale);
  else k_quant_rows<T, TH, 9><<<grid, threads, 0, c.stream>>>(a, ld_a, n, Kd, q, ld_q, scale);
}

template <typename T, int W, int NC>
void quant_shift(const Ctx& c, const T* a, int64_t ld_a, int n, int Kd, int8_t* q, int64_t ld_q,
                 float* scale) {
  k_quant_rows_shift<T, W, NC><<<W == 1 ? (n + 7) / 8 : n, W == 1 ? 256 : 32 * W, 0, c.stream>>>(
      a, ld_a, n, Kd, q, ld_q, scale);
}

static_assert(kMaxInPlaceK == 9 * 512 * 8, "rows up to here are in registers before they are written");

template <typename T>
cudaError_t quant_typed(const Ctx& c, const T* a, int n, int Kd, int64_t ld_a, int8_t* q,
                        int64_t ld_q, float* scale) {
  const bool vec = ld_a * static_cast<int64_t>(sizeof(T)) % 16 == 0;  // every row aligned
  const int vecs = (Kd + 7) / 8;
  if (vec && vecs <= 9 * 32) quant_threads<T, 32>(c, a, ld_a, n, Kd, q, ld_q, scale);
  else if (vec && vecs <= 9 * 128) quant_threads<T, 128>(c, a, ld_a, n, Kd, q, ld_q, scale);
  else if (vec && vecs <= 9 * 512) quant_threads<T, 512>(c, a, ld_a, n, Kd, q, ld_q, scale);
  else if (vecs <= 32 * 2 - 1) quant_shift<T, 1, 2>(c, a, ld_a, n, Kd, q, ld_q, scale);
  else if (vecs <= 32 * 4 - 1) quant_shift<T, 1, 4>(c, a, ld_a, n, Kd, q, ld_q, scale);
  else if (vecs <= 32 * 8 - 1) quant_shift<T, 1, 8>(c, a, ld_a, n, Kd, q, ld_q, scale);
  else if (vecs <= 4 * (32 * 3 - 1)) quant_shift<T, 4, 3>(c, a, ld_a, n, Kd, q, ld_q, scale);
  else if (vecs <= 4 * (32 * 5 - 1)) quant_shift<T, 4, 5>(c, a, ld_a, n, Kd, q, ld_q, scale);
  else if (vecs <= 4 * (32 * 8 - 1)) quant_shift<T, 4, 8>(c, a, ld_a, n, Kd, q, ld_q, scale);
  else if (vecs <= 8 * (32 * 8 - 1)) quant_shift<T, 8, 8>(c, a, ld_a, n, Kd, q, ld_q, scale);
  else if (vecs <= 16 * (32 * 8 - 1)) quant_shift<T, 16, 8>(c, a, ld_a, n, Kd, q, ld_q, scale);
  else k_quant_rows_any<T><<<n, 256, 0, c.stream>>>(a, ld_a, n, Kd, q, ld_q, scale);
  c.launches += 1;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quant_rows(const Ctx& c, const void* a, bool f32, int n, int Kd, int64_t ld_a,
                              int8_t* q, int64_t ld_q, float* scale) {
  Timed timed(c, TC_ROWS, static_cast<double>(n) * Kd * (f32 ? 5.0 : 3.0));
  return f32 ? quant_typed(c, static_cast<const float*>(a), n, Kd, ld_a, q, ld_q, scale)
             : quant_typed(c, static_cast<const __nv_bfloat16*>(a), n, Kd, ld_a, q, ld_q, scale);
}

cudaError_t launch_ln_gather_quant(const Ctx& c, const float* x, const int32_t* idx, int n,
                                   int8_t* q, float* scale, const float* shift,
                                   const float* mscale) {
  const int D = c.cfg.D, N = c.cfg.N;
  Timed timed(c, TC_ROWS, static_cast<double>(n) * D * 5.0);
  const dim3 grid((n + 7) / 8), block(256);
  if (D <= 4 * 128)
    k_ln_gather_quant<4><<<grid, block, 0, c.stream>>>(x, idx, n, N, D, q, scale, c.flag, shift, mscale);
  else if (D <= 12 * 128)
    k_ln_gather_quant<12><<<grid, block, 0, c.stream>>>(x, idx, n, N, D, q, scale, c.flag, shift, mscale);
  else if (D <= 20 * 128)
    k_ln_gather_quant<20><<<grid, block, 0, c.stream>>>(x, idx, n, N, D, q, scale, c.flag, shift, mscale);
  else
    k_ln_gather_quant<kMaxLnQuantD / 128><<<grid, block, 0, c.stream>>>(x, idx, n, N, D, q, scale, c.flag, shift, mscale);
  c.launches += 1;
  return cudaGetLastError();
}

}  // namespace hsa
