// k_rotary.cu - rotary positions: the table of cosines and sines, the rotation
// of head rows by it, and the pass that normalises, rotates and stores fresh
// queries, keys and values.
//
// A head's first `rot` places hold rot/2 planes; plane i of a row at table row
// p is turned by the angle whose cosine and sine are table[p][i]:
//   (u, v) -> (u cos - v sin, v cos + u sin).
// The planes are (2i, 2i+1) in the interleaved layout, (i, i + rot/2) in the
// half layout.
//
// All three kernels are bound by HBM.  A thread owns a unit of 16 places of a
// head, eight planes: two 16-byte vectors of bf16, adjacent (interleaved) or
// rot/2 apart (half), so no plane crosses threads.  A warp owns a row: its 32
// lanes hold the d/16 units of 512/d heads and step over the heads, keeping
// the row's 8 cosines and sines per lane in registers for all of them.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "ptx.cuh"

namespace hsa {

namespace {

constexpr int kRowWarps = 8;  // warps (rows) per CTA
constexpr int kQkWarps = 4;   // rows are wide in registers: small blocks leave fewer unused

// ------------------------------------------------------------ table
struct TableParams {
  double turns[kMaxRopePairs];  // frequency / 2 pi of each plane
  uint8_t axis[kMaxRopePairs];
  const int32_t* pos;           // [P, n_axes], or null: row p has position p
  int n_axes, P, half;
  float amp;
  float2* table;                // [P, half]
};

// table[p][i] = amp (cos, sin)(2 pi pos turns_i).  The angle is held in 64
// bits, as turns: only its fraction of a turn matters, and that is taken
// before anything is rounded to 32 bits, so far positions lose nothing (at
// 2^20 the fraction is good to 2^-34 of a turn).  The fraction's part below 32
// bits enters by the first-order term of the addition theorem.  One 64-bit
// product and the reduction per entry instead of a 64-bit sine and cosine.
// A thread keeps one plane and walks over rows: block (half, 256 / half).
__global__ void __launch_bounds__(256) k_rope_table(const __grid_constant__ TableParams p) {
  const int i = threadIdx.x;
  const double turns = p.turns[i];
  const int axis = p.axis[i];
  const int stride = gridDim.x * blockDim.y;
  for (int row = blockIdx.x * blockDim.y + threadIdx.y; row < p.P; row += stride) {
    const int32_t at =
        p.pos == nullptr ? row : __ldg(p.pos + static_cast<int64_t>(row) * p.n_axes + axis);
    const double full = static_cast<double>(at) * turns;
    const double frac = full - rint(full);  // [-1/2, 1/2]
    const float hi = static_cast<float>(frac);
    const float lo = static_cast<float>(frac - static_cast<double>(hi)) * 6.283185307179586f;
    float s, c;
    sincospif(2.0f * hi, &s, &c);
    p.table[static_cast<int64_t>(row) * p.half + i] =
        make_float2(p.amp * fmaf(-lo, s, c), p.amp * fmaf(lo, c, s));
  }
}

// ------------------------------------------------------------ units of 16 places
struct Unit {
  float u[8], v[8];  // plane members in half layout order: (u[i], v[i]) is plane i
};

__device__ __forceinline__ void unpack8(const uint4& w, float (&f)[8]) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(r[i] << 16);
    f[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                    pack_bf16(f[6], f[7]));
}

// The lane's cosines and sines: table row entries 8u .. 8u+7 (64 bytes).
__device__ __forceinline__ void load_turns(const float* __restrict__ table, int64_t row, int rot,
                                           int u, bool inverse, float (&cs)[8], float (&sn)[8]) {
  const float4* t4 = reinterpret_cast<const float4*>(table + row * rot + 16 * u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 w = __ldg(t4 + i);
    cs[2 * i] = w.x;
    sn[2 * i] = inverse ? -w.y : w.y;
    cs[2 * i + 1] = w.z;
    sn[2 * i + 1] = inverse ? -w.w : w.w;
  }
}

// First place (in elements) of the unit's two 8-element vectors within its head.
__device__ __forceinline__ void unit_places(int u, int rot, bool half_layout, int& a, int& b) {
  if (half_layout && 16 * u < rot) {
    a = 8 * u;
    b = a + rot / 2;
  } else {
    a = 16 * u;
    b = a + 8;
  }
}

// Turns a unit's 16 values, x[0] and x[1] its two vectors of 8.
__device__ __forceinline__ void turn(float (&x)[2][8], const float (&cs)[8], const float (&sn)[8],
                                     bool half_layout) {
  if (half_layout) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[0][i], b = x[1][i];
      x[0][i] = a * cs[i] - b * sn[i];
      x[1][i] = b * cs[i] + a * sn[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float& p = x[i >> 2][2 * (i & 3)];
      float& q = x[i >> 2][2 * (i & 3) + 1];
      const float a = p, b = q;
      p = a * cs[i] - b * sn[i];
      q = b * cs[i] + a * sn[i];
    }
  }
}

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// 8 values as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 w;
  __device__ void load(const __nv_bfloat16* p) { w = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ void store(__nv_bfloat16* p) const { __stcs(reinterpret_cast<uint4*>(p), w); }
  __device__ void get(float (&f)[8]) const { unpack8(w, f); }
  __device__ void set(const float (&f)[8]) { w = pack8(f); }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ void store(float* p) const {
    __stcs(reinterpret_cast<float4*>(p), a);
    __stcs(reinterpret_cast<float4*>(p) + 1, b);
  }
  __device__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  __device__ void set(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// ------------------------------------------------------------ rotation alone
struct RopeParams {
  const void* x;
  void* out;
  int64_t ld_x, ld_out;  // elements
  const float* table;
  const int32_t* pos;    // table row of each row, or null: its own number
  int n, heads, P, rot;
  bool half_layout, inverse;
  int* flag;
};

// kBatch steps of 512/d heads are loaded before the first is stored (out may be
// x, so the compiler cannot move a load over a store): enough bytes in flight
// to cover the latency of HBM.
template <typename T, int HD>
__global__ void __launch_bounds__(32 * kRowWarps) k_rope(RopeParams p) {
  constexpr int U = HD / 16, HG = 32 / U, kBatch = sizeof(T) == 2 ? 4 : 2;
  const int lane = threadIdx.x & 31;
  const int m = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  if (m >= p.n) return;
  const int u = lane % U, h0 = lane / U;
  const int32_t row = p.pos == nullptr ? m : __ldg(p.pos + m);
  if (!row_ok(row, p.P, p.flag)) return;
  const bool turned = 16 * u < p.rot;
  int a, b;
  unit_places(u, p.rot, p.half_layout, a, b);
  const T* x = static_cast<const T*>(p.x) + m * p.ld_x;
  T* out = static_cast<T*>(p.out) + m * p.ld_out;
  float cs[8], sn[8];
  if (turned) load_turns(p.table, row, p.rot, u, p.inverse, cs, sn);
  for (int hb = h0; hb < p.heads; hb += HG * kBatch) {
    Raw8<T> raw[kBatch][2];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = hb + k * HG;
      if (h < p.heads) {
        raw[k][0].load(x + h * HD + a);
        raw[k][1].load(x + h * HD + b);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = hb + k * HG;
      if (h >= p.heads) break;
      if (turned) {
        float f[2][8];
        raw[k][0].get(f[0]);
        raw[k][1].get(f[1]);
        turn(f, cs, sn, p.half_layout);
        raw[k][0].set(f[0]);
        raw[k][1].set(f[1]);
      }
      raw[k][0].store(out + h * HD + a);
      raw[k][1].store(out + h * HD + b);
    }
  }
}

// ------------------------------------------------------------ norm, rotation, cache write
struct QkParams {
  const __nv_bfloat16 *q_in, *k_in, *v_in;  // sources; k_in null with do_k: cache rows in place
  int64_t ld_q, ld_k, ld_v;
  __nv_bfloat16 *q, *k_cache, *v_cache;
  const float *w_q, *w_k;
  const float* table;
  const int32_t *idx, *pos;
  int n, N, P, H, rot, norm, parts;
  uint8_t part[3];  // what each of the `parts` warps of a row does: 0 q, 1 k, 2 v
  float eps;
  bool half_layout;
  int* flag;
};

// One warp per row and part, NIT steps of 512/d heads, the whole row in
// registers between its one read and its one write.  The mean square is
// summed in 32 bits: over a head by shuffles between the head's lanes, over
// the row by all lanes.  One rounding to bf16, at the store.
template <int HD, int NIT>
__global__ void __launch_bounds__(32 * kQkWarps) k_qk_norm_rope(const __grid_constant__ QkParams p) {
  constexpr int U = HD / 16, HG = 32 / U;
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kQkWarps + (threadIdx.x >> 5);
  const int m = static_cast<int>(item / p.parts);
  if (m >= p.n) return;
  const int part = p.part[item - static_cast<int64_t>(m) * p.parts];
  const int D = p.H * HD;
  const int u = lane % U, h0 = lane / U;

  const int32_t r = p.idx == nullptr ? m : __ldg(p.idx + m);
  const int32_t at = p.pos == nullptr ? r : __ldg(p.pos + m);
  bool good = row_ok(r, p.N, p.flag);
  if (p.table != nullptr && part != 2) good = row_ok(at, p.P, p.flag) && good;
  const __nv_bfloat16* src;
  __nv_bfloat16* dst;
  const float* w = nullptr;
  if (part == 0) {
    src = p.q_in + m * p.ld_q;
    dst = p.q + static_cast<int64_t>(m) * D;
    w = p.w_q;
  } else if (part == 1) {
    if (p.k_in == nullptr && m > 0 && p.idx != nullptr && __ldg(p.idx + m - 1) >= r) {
      // in place, a row named twice would be turned twice: the list must ascend
      if (lane == 0) atomicOr(p.flag, DEV_BAD_INDEX);
      good = false;
    }
    dst = p.k_cache + static_cast<int64_t>(r) * D;
    src = p.k_in != nullptr ? p.k_in + m * p.ld_k : dst;
    w = p.w_k;
  } else {
    dst = p.v_cache + static_cast<int64_t>(r) * D;
    src = p.v_in + m * p.ld_v;
  }
  if (!good) {  // skipped and reported; a query row is left zero rather than unset
    if (part == 0)
      for (int e = 8 * lane; e < D; e += 256)
        *reinterpret_cast<uint4*>(dst + e) = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const bool turned = p.table != nullptr && part != 2 && 16 * u < p.rot;
  int a, b;
  unit_places(u, p.table != nullptr && part != 2 ? p.rot : 0, p.half_layout, a, b);
  Raw8<__nv_bfloat16> raw[NIT][2];
#pragma unroll
  for (int it = 0; it < NIT; ++it) {
    const int h = h0 + it * HG;
    raw[it][0].w = raw[it][1].w = make_uint4(0u, 0u, 0u, 0u);
    if (h < p.H) {
      raw[it][0].load(src + h * HD + a);
      raw[it][1].load(src + h * HD + b);
    }
  }
  if (part == 2) {  // values go to the cache as they are
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      const int h = h0 + it * HG;
      if (h < p.H) {
        raw[it][0].store(dst + h * HD + a);
        raw[it][1].store(dst + h * HD + b);
      }
    }
    return;
  }
  float cs[8], sn[8];
  if (turned) load_turns(p.table, at, p.rot, u, false, cs, sn);
  float g[2][8];  // weights of a norm over each head: the same for all heads
  const bool per_head = p.norm == HSA_NORM_HEAD, weighted = w != nullptr && p.norm != HSA_NORM_NONE;
  if (weighted && per_head) {
    load8(w + a, g[0]);
    load8(w + b, g[1]);
  }
  float row_scale = 1.0f;
  if (p.norm == HSA_NORM_ROW) {
    float ss = 0.f;
#pragma unroll
    for (int it = 0; it < NIT; ++it)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float f[8];
        raw[it][k].get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    row_scale = rsqrtf(ss / static_cast<float>(D) + p.eps);
  }
#pragma unroll
  for (int it = 0; it < NIT; ++it) {
    const int h = h0 + it * HG;
    float f[2][8];
    raw[it][0].get(f[0]);
    raw[it][1].get(f[1]);
    if (p.norm != HSA_NORM_NONE) {
      float scale = row_scale;
      if (per_head) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[0][i], f[0][i], fmaf(f[1][i], f[1][i], ss));
#pragma unroll
        for (int o = U / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        scale = rsqrtf(ss * (1.0f / HD) + p.eps);
      }
      if (weighted && !per_head && h < p.H) {
        load8(w + h * HD + a, g[0]);
        load8(w + h * HD + b, g[1]);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[k][i] *= scale;
          if (weighted) f[k][i] *= g[k][i];
        }
    }
    if (turned) turn(f, cs, sn, p.half_layout);
    raw[it][0].set(f[0]);
    raw[it][1].set(f[1]);
    if (h < p.H) {
      raw[it][0].store(dst + h * HD + a);
      raw[it][1].store(dst + h * HD + b);
    }
  }
}

template <int HD>
cudaError_t launch_qk(const Ctx& c, const QkParams& p) {
  constexpr int HG = 512 / HD;
  const int nit = (p.H + HG - 1) / HG;
  const int64_t items = static_cast<int64_t>(p.n) * p.parts;
  const unsigned grid = static_cast<unsigned>((items + kQkWarps - 1) / kQkWarps);
  const dim3 block(32 * kQkWarps);
  if (nit <= 1) k_qk_norm_rope<HD, 1><<<grid, block, 0, c.stream>>>(p);
  else if (nit <= 3) k_qk_norm_rope<HD, 3><<<grid, block, 0, c.stream>>>(p);
  else if (nit <= 6) k_qk_norm_rope<HD, 6><<<grid, block, 0, c.stream>>>(p);
  else if (nit <= 10) k_qk_norm_rope<HD, 10><<<grid, block, 0, c.stream>>>(p);
  else k_qk_norm_rope<HD, kMaxQkSteps><<<grid, block, 0, c.stream>>>(p);
  c.launches += 1;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_table(const Ctx& c, const RopeFreqs& f, const int32_t* pos, int P,
                              float* table) {
  Timed timed(c, TC_ROWS, static_cast<double>(P) * (8.0 * f.half + 4.0 * f.n_axes));
  TableParams p{};
  for (int i = 0; i < f.half; ++i) p.turns[i] = f.turns[i], p.axis[i] = f.axis[i];
  p.pos = pos;
  p.n_axes = f.n_axes;
  p.P = P;
  p.half = f.half;
  p.amp = f.amp;
  p.table = reinterpret_cast<float2*>(table);
  const dim3 block(f.half, 256 / f.half);
  int64_t blocks = (static_cast<int64_t>(P) + block.y - 1) / block.y;
  if (blocks > c.num_sms * 8) blocks = c.num_sms * 8;
  k_rope_table<<<static_cast<unsigned>(blocks), block, 0, c.stream>>>(p);
  c.launches += 1;
  return cudaGetLastError();
}

cudaError_t launch_rope(const Ctx& c, const void* x, int64_t ld_x, bool f32, int n, int heads,
                        const float* table, int P, int rot, const int32_t* pos, bool half_layout,
                        bool inverse, void* out, int64_t ld_out) {
  const int hd = c.cfg.D / c.cfg.H;
  Timed timed(c, TC_ROWS, static_cast<double>(n) * ((f32 ? 8.0 : 4.0) * heads * hd + 4.0 * rot));
  RopeParams p{x, out, ld_x, ld_out, table, pos, n, heads, P, rot, half_layout, inverse, c.flag};
  const unsigned grid = (n + kRowWarps - 1) / kRowWarps;
  const dim3 block(32 * kRowWarps);
  if (f32 && hd == 128) k_rope<float, 128><<<grid, block, 0, c.stream>>>(p);
  else if (f32) k_rope<float, 64><<<grid, block, 0, c.stream>>>(p);
  else if (hd == 128) k_rope<__nv_bfloat16, 128><<<grid, block, 0, c.stream>>>(p);
  else k_rope<__nv_bfloat16, 64><<<grid, block, 0, c.stream>>>(p);
  c.launches += 1;
  return cudaGetLastError();
}

cudaError_t launch_qk_norm_rope(const Ctx& c, const hsa_qk_rope& a, const QkRows& r) {
  const int H = c.cfg.H, hd = c.cfg.D / H;
  QkParams p{};
  if (r.q != nullptr) p.part[p.parts++] = 0;
  if (r.k_cache != nullptr) p.part[p.parts++] = 1;
  if (r.v_cache != nullptr) p.part[p.parts++] = 2;
  Timed timed(c, TC_ROWS,
              static_cast<double>(r.n) * (4.0 * p.parts * c.cfg.D + (a.table ? 4.0 * a.rot : 0.0)));
  p.q_in = static_cast<const __nv_bfloat16*>(r.q_in != nullptr ? r.q_in : r.q);
  p.k_in = static_cast<const __nv_bfloat16*>(r.k_in);
  p.v_in = static_cast<const __nv_bfloat16*>(r.v_in);
  p.ld_q = r.q_in != nullptr ? r.ld_q : c.cfg.D;
  p.ld_k = r.ld_k;
  p.ld_v = r.ld_v;
  p.q = static_cast<__nv_bfloat16*>(r.q);
  p.k_cache = static_cast<__nv_bfloat16*>(r.k_cache);
  p.v_cache = static_cast<__nv_bfloat16*>(r.v_cache);
  p.w_q = a.w_q;
  p.w_k = a.w_k;
  p.table = a.table;
  p.idx = r.idx;
  p.pos = r.pos;
  p.n = r.n;
  p.N = c.cfg.N;
  p.P = a.P;
  p.H = H;
  p.rot = a.rot;
  p.norm = a.norm;
  p.eps = a.eps;
  p.half_layout = a.layout == HSA_ROPE_HALF;
  p.flag = c.flag;
  return hd == 128 ? launch_qk<128>(c, p) : launch_qk<64>(c, p);
}

}  // namespace hsa
