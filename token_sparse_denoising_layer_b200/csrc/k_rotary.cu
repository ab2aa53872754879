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
// head, eight planes in two 16-byte vectors of bf16, so no plane crosses
// threads.  A warp owns a row: its 32 lanes hold the d/16 units of 512/d heads
// and step over the heads, keeping the row's 8 cosines and sines per lane in
// registers for all of them.
//
// Measured: table of 131072 x 64 planes 15.3 us (67 MB written, 4.4 TB/s);
// rotation of 32760 x 12 x 128 bf16 36 us (6.1 TB/s); norm, rotation and cache write of
// 13104 x 12 x 128 47 us (5.3 TB/s), of 18900 x 40 x 128 203 us (5.8 TB/s).

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
  uint64_t turns[kMaxRopePairs];  // frequency of each plane: turns per position * 2^64
  uint8_t axis[kMaxRopePairs];
  const int32_t* pos;             // [P, n_axes], or null: row p has position p
  int n_axes, P, half;
  float amp;
  float2* table;                  // [P, half]
};

// table[p][i] = amp (cos, sin)(pos f_i).  The angle is a fixed-point count of
// 2^-64 turns, so pos * turns wraps at whole turns by itself.  A frequency is right
// to a unit or two, which a position of 2^31 makes 2^-32 of a turn, and the
// product is cut to its upper 32 bits: 2^-31 of a turn (3e-9 rad) in all at any
// position.  The nearest quarter turn k is taken off, and sine and cosine of the rest
// x, |x| <= pi / 4, are their Taylor polynomials to x^9 and x^10 (the next terms
// are below 2e-9).  k mod 4 swaps and negates them.
//
// A thread keeps two planes and walks over the rows of its block's share: one
// position and one address serve both, and the polynomials run on packed
// f32x2 (69 issued instructions an entry with one plane and 64-bit sines).
// The positions of kTableRows rows are brought to shared memory together: a
// load per row left every row waiting for HBM on its own.
constexpr int kTableRows = 256;

struct Quarter {
  uint32_t k;  // nearest quarter turn
  float x;     // what is left, in radians
};

__device__ __forceinline__ Quarter quarter_of(int32_t at, uint64_t turns) {
  const uint32_t t =
      static_cast<uint32_t>((static_cast<uint64_t>(static_cast<int64_t>(at)) * turns) >> 32);
  const uint32_t k = (t + 0x20000000u) >> 30;  // an eighth of a turn up, then down to a quarter
  return Quarter{k, static_cast<float>(static_cast<int32_t>(t - (k << 30))) * 1.4629180792671596e-9f};  // 2 pi 2^-32
}

// (cos, sin) of a quarter count and the rest's (cos, sin).
__device__ __forceinline__ float2 unfold(uint32_t k, float c, float s) {
  const float u = (k & 1) ? s : c, v = (k & 1) ? c : s;
  return make_float2(__uint_as_float(__float_as_uint(u) ^ (((k + 1) & 2u) << 30)),
                     __uint_as_float(__float_as_uint(v) ^ ((k & 2u) << 30)));
}

// Block (half / kPlanes, 256 / that); an odd count of planes takes one a thread.
template <int kPlanes>
__global__ void __launch_bounds__(256) k_rope_table(const __grid_constant__ TableParams p) {
  // The frequencies are kernel arguments: a warp reads them one at a time, as a
  // constant that differs between lanes is fetched once per lane.
  __shared__ uint64_t s_turns[kMaxRopePairs];
  __shared__ int s_axis[kMaxRopePairs];
  __shared__ int32_t s_pos[kTableRows * 3];
  const int thread = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
  const int64_t P = p.P;
  const int first = static_cast<int>(P * blockIdx.x / gridDim.x);
  const int last = static_cast<int>(P * (blockIdx.x + 1) / gridDim.x);
  for (int row0 = first; row0 < last; row0 += kTableRows) {
    const int rows = min(kTableRows, last - row0);
    __syncthreads();
    if (p.pos != nullptr) {
      const int32_t* src = p.pos + static_cast<int64_t>(row0) * p.n_axes;
      for (int j = thread; j < rows * p.n_axes; j += threads) s_pos[j] = __ldg(src + j);
    } else {
      for (int j = thread; j < rows; j += threads) s_pos[j] = row0 + j;
    }
    if (row0 == first && (thread & 31) == 0) {
      for (int j = thread >> 5; j < p.half; j += (threads + 31) >> 5) {
        s_turns[j] = p.turns[j];
        s_axis[j] = p.axis[j];
      }
    }
    __syncthreads();
    const int i = kPlanes * threadIdx.x;
    const uint64_t turns0 = s_turns[i], turns1 = s_turns[i + kPlanes - 1];
    const int32_t* pos0 = s_pos + s_axis[i];
    const int32_t* pos1 = s_pos + s_axis[i + kPlanes - 1];
    const F2 amp = splat(p.amp);
    float2* out = p.table + static_cast<int64_t>(row0) * p.half + i;
#pragma unroll 2
    for (int row = threadIdx.y; row < rows; row += blockDim.y) {
      const Quarter q0 = quarter_of(pos0[row * p.n_axes], turns0);
      const Quarter q1 = kPlanes == 2 ? quarter_of(pos1[row * p.n_axes], turns1) : q0;
      const F2 x = F2{q0.x, q1.x};
      const F2 z = mul_x2(x, x);
      F2 s = fma_x2(z, splat(1.f / 362880.f), splat(-1.f / 5040.f));
      s = fma_x2(z, s, splat(1.f / 120.f));
      s = fma_x2(z, s, splat(-1.f / 6.f));
      s = fma_x2(mul_x2(x, z), s, x);
      F2 c = fma_x2(z, splat(-1.f / 3628800.f), splat(1.f / 40320.f));
      c = fma_x2(z, c, splat(-1.f / 720.f));
      c = fma_x2(z, c, splat(1.f / 24.f));
      c = fma_x2(z, c, splat(-0.5f));
      c = fma_x2(z, c, splat(1.f));
      s = mul_x2(s, amp);
      c = mul_x2(c, amp);
      const float2 t0 = unfold(q0.k, c.x, s.x);
      float2* dst = out + static_cast<int64_t>(row) * p.half;
      if (kPlanes == 2) {
        const float2 t1 = unfold(q1.k, c.y, s.y);
        __stcs(reinterpret_cast<float4*>(dst), make_float4(t0.x, t0.y, t1.x, t1.y));
      } else {
        *dst = t0;
      }
    }
  }
}

// ------------------------------------------------------------ units of 16 places
// A lane's unit u of d/16 per head: two vectors of 8 places, at a and b.  In
// the half layout they are the two members of eight planes; past the rotated
// places, and in the interleaved layout (where a vector holds whole planes),
// b lies half of the places in question further on.  Either way a
// head's lanes cover 16 adjacent bytes each, in two runs.
template <int HD, bool kHalf>
struct Places {
  int a, b;
  bool turn_a, turn_b;  // whether the vector's places are rotated
  __device__ Places(int u, int rot) {
    if (!kHalf) {
      a = 8 * u, b = HD / 2 + 8 * u;
      turn_a = a < rot, turn_b = b < rot;
    } else {
      turn_a = turn_b = 16 * u < rot;
      if (turn_a) a = 8 * u, b = rot / 2 + 8 * u;
      else a = rot + 8 * (u - rot / 16), b = a + (HD - rot) / 2;
    }
  }
};

// 8 values as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint32_t w[4];
  __device__ void load(const __nv_bfloat16* p) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
  __device__ void store(__nv_bfloat16* p) const {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  }
  __device__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
  __device__ float get(int i) const {
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
  __device__ void set2(int i, float lo, float hi) { w[i >> 1] = pack_bf16(lo, hi); }
};
template <>
struct Raw8<float> {
  float f[8];
  __device__ void load(const float* p) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  __device__ void store(float* p) const {
    __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
  }
  __device__ float get(int i) const { return f[i]; }
  __device__ void set2(int i, float lo, float hi) { f[i] = lo, f[i + 1] = hi; }
};

// The unit's eight planes in pairs for packed f32x2 arithmetic: members u and
// v of planes 2i and 2i + 1 (interleaved: planes 0..3 lie in the first vector).
struct Planes {
  F2 u[4], v[4];
};

template <bool kHalf, typename T>
__device__ __forceinline__ void get_planes(const Raw8<T> (&x)[2], Planes& p) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kHalf) {
      p.u[i] = F2{x[0].get(2 * i), x[0].get(2 * i + 1)};
      p.v[i] = F2{x[1].get(2 * i), x[1].get(2 * i + 1)};
    } else {
      const Raw8<T>& r = x[i >> 1];
      const int j = 4 * (i & 1);
      p.u[i] = F2{r.get(j), r.get(j + 2)};
      p.v[i] = F2{r.get(j + 1), r.get(j + 3)};
    }
  }
}

template <bool kHalf, typename T>
__device__ __forceinline__ void set_planes(Raw8<T> (&x)[2], const Planes& p) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kHalf) {
      x[0].set2(2 * i, p.u[i].x, p.u[i].y);
      x[1].set2(2 * i, p.v[i].x, p.v[i].y);
    } else {
      const int j = 4 * (i & 1);
      x[i >> 1].set2(j, p.u[i].x, p.v[i].x);
      x[i >> 1].set2(j + 2, p.u[i].y, p.v[i].y);
    }
  }
}

// Cosines and sines of the unit's planes, from a row of the table.
template <bool kHalf>
__device__ __forceinline__ void load_turns(const float* __restrict__ row, int a, int b, bool turn_a,
                                           bool turn_b, float sign, F2 (&cs)[4], F2 (&sn)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool on = kHalf || i < 2 ? turn_a : turn_b;
    if (on) {
      const int at = kHalf ? 2 * a + 4 * i : (i < 2 ? a : b) + 4 * (i & 1);
      const float4 w = __ldg(reinterpret_cast<const float4*>(row + at));
      cs[i] = F2{w.x, w.z};
      sn[i] = F2{sign * w.y, sign * w.w};
    }
  }
}

template <bool kHalf>
__device__ __forceinline__ void turn(Planes& p, const F2 (&cs)[4], const F2 (&sn)[4], bool turn_a,
                                     bool turn_b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool on = kHalf || i < 2 ? turn_a : turn_b;
    if (on) {
      const F2 u = p.u[i], v = p.v[i];
      const F2 m = F2{-sn[i].x, -sn[i].y};
      p.u[i] = fma_x2(u, cs[i], mul_x2(v, m));
      p.v[i] = fma_x2(v, cs[i], mul_x2(u, sn[i]));
    }
  }
}

// ------------------------------------------------------------ rotation alone
struct RopeParams {
  const void* x;
  void* out;
  int64_t ld_x, ld_out;  // elements
  const float* table;
  const int32_t* pos;    // table row of each row, or null: its own number
  int n, heads, P, rot;
  float sign;            // -1: the inverse
  int* flag;
};

// kBatch steps of 512/d heads are loaded before the first is stored (out may be
// x, so the compiler cannot move a load over a store): enough bytes in flight
// to cover the latency of HBM.
template <typename T, int HD, bool kHalf>
__global__ void __launch_bounds__(32 * kRowWarps) k_rope(const __grid_constant__ RopeParams p) {
  constexpr int U = HD / 16, HG = 32 / U, kBatch = sizeof(T) == 2 ? 4 : 2;
  const int lane = threadIdx.x & 31;
  const int m = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  if (m >= p.n) return;
  const int u = lane % U, h0 = lane / U;
  const Places<HD, kHalf> at(u, p.rot);
  const T* x = static_cast<const T*>(p.x) + m * p.ld_x;
  T* out = static_cast<T*>(p.out) + m * p.ld_out;
  const int32_t row = p.pos == nullptr ? m : __ldg(p.pos + m);
  if (!row_ok(row, p.P, p.flag)) return;
  F2 cs[4], sn[4];
  load_turns<kHalf>(p.table + static_cast<int64_t>(row) * p.rot, at.a, at.b, at.turn_a, at.turn_b,
                    p.sign, cs, sn);
  for (int hb = h0; hb < p.heads; hb += HG * kBatch) {
    Raw8<T> raw[kBatch][2];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = hb + k * HG;
      if (h < p.heads) {
        raw[k][0].load(x + h * HD + at.a);
        raw[k][1].load(x + h * HD + at.b);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = hb + k * HG;
      if (h >= p.heads) break;
      if (at.turn_a) {  // without turns a value is copied bit for bit
        Raw8<T> y[2] = {raw[k][0], raw[k][1]};
        Planes f;
        get_planes<kHalf>(raw[k], f);
        turn<kHalf>(f, cs, sn, at.turn_a, at.turn_b);
        set_planes<kHalf>(y, f);
        raw[k][0] = y[0];
        if (at.turn_b) raw[k][1] = y[1];
      }
      raw[k][0].store(out + h * HD + at.a);
      raw[k][1].store(out + h * HD + at.b);
    }
  }
}

// ------------------------------------------------------------ norm, rotation, cache write
struct QkParams {
  const __nv_bfloat16 *q_in, *k_in, *v_in;  // sources; k_in null with k_cache: cache rows in place
  int64_t ld_q, ld_k, ld_v;
  __nv_bfloat16 *q, *k_cache, *v_cache;
  const float *w_q, *w_k;
  const float* table;
  const int32_t *idx, *pos;
  int n, N, P, H, rot, norm, parts;
  uint8_t part[3];  // what each of the `parts` warps of a row does: 0 q, 1 k, 2 v
  bool ascending;   // keys in place: a row named twice would be turned twice, so idx must ascend
  float eps;
  int* flag;
};

// Weights of the unit's places, arranged as its planes.
template <bool kHalf>
__device__ __forceinline__ void load_weights(const float* __restrict__ w, int a, int b, Planes& g) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kHalf) {
      if (i & 1) continue;
      const float4 x = __ldg(reinterpret_cast<const float4*>(w + a + 2 * i));
      const float4 y = __ldg(reinterpret_cast<const float4*>(w + b + 2 * i));
      g.u[i] = F2{x.x, x.y}, g.u[i + 1] = F2{x.z, x.w};
      g.v[i] = F2{y.x, y.y}, g.v[i + 1] = F2{y.z, y.w};
    } else {
      const float4 x = __ldg(reinterpret_cast<const float4*>(w + (i < 2 ? a : b) + 4 * (i & 1)));
      g.u[i] = F2{x.x, x.z}, g.v[i] = F2{x.y, x.w};
    }
  }
}

__device__ __forceinline__ float square_sum(const Planes& f) {
  F2 s = mul_x2(f.u[0], f.u[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = fma_x2(f.u[i], f.u[i], s);
#pragma unroll
  for (int i = 0; i < 4; ++i) s = fma_x2(f.v[i], f.v[i], s);
  return s.x + s.y;
}

// One warp per row and part, NIT steps of 512/d heads, the whole row in
// registers between its one read and its one write.  The mean square is
// summed in 32 bits: over a head by shuffles between the head's lanes, over
// the row by all lanes.  One rounding to bf16, at the store.
template <int HD, int NIT, bool kHalf>
__global__ void __launch_bounds__(32 * kQkWarps, NIT <= 3 ? 6 : 1)
    k_qk_norm_rope(const __grid_constant__ QkParams p) {
  constexpr int U = HD / 16, HG = 32 / U;
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kQkWarps + (threadIdx.x >> 5);
  const int m = static_cast<int>(item / p.parts);
  if (m >= p.n) return;
  const int part = p.part[item - static_cast<int64_t>(m) * p.parts];
  const int D = p.H * HD;
  const int u = lane % U, h0 = lane / U;

  const int32_t r = p.idx == nullptr ? m : __ldg(p.idx + m);
  const int32_t trow = p.pos == nullptr ? r : __ldg(p.pos + m);
  // The sources' rows do not depend on idx: their loads go out before its
  // value is waited for (in place they do, and follow it).
  const bool in_place = part == 1 && p.k_in == nullptr;
  const __nv_bfloat16* src = part == 0 ? p.q_in + m * p.ld_q
                             : part == 2 ? p.v_in + m * p.ld_v : p.k_in + m * p.ld_k;
  const bool rotating = p.table != nullptr && part != 2;
  const Places<HD, kHalf> at(u, rotating ? p.rot : 0);
  Raw8<__nv_bfloat16> raw[NIT][2];
  auto load_row = [&]() {
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      const int h = h0 + it * HG;
      raw[it][0].zero();
      raw[it][1].zero();
      if (h < p.H) {
        raw[it][0].load(src + h * HD + at.a);
        raw[it][1].load(src + h * HD + at.b);
      }
    }
  };
  if (!in_place) load_row();
  // One verdict for the row's parts, so that no value is written beside a key
  // that was skipped.
  bool good = row_ok(r, p.N, p.flag);
  if (p.table != nullptr) good = row_ok(trow, p.P, p.flag) && good;
  if (p.ascending && m > 0 && __ldg(p.idx + m - 1) >= r) {
    if (lane == 0) atomicOr(p.flag, DEV_BAD_INDEX);
    good = false;
  }
  __nv_bfloat16* dst = part == 0 ? p.q + static_cast<int64_t>(m) * D
                                 : (part == 1 ? p.k_cache : p.v_cache) + static_cast<int64_t>(r) * D;
  const float* w = part == 0 ? p.w_q : p.w_k;
  if (!good) {  // skipped and reported; a query row is left zero rather than unset
    if (part == 0)
      for (int e = 8 * lane; e < D; e += 256)
        *reinterpret_cast<uint4*>(dst + e) = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  if (in_place) {
    src = dst;
    load_row();
  }
  const bool per_head = p.norm == HSA_NORM_HEAD, per_row = p.norm == HSA_NORM_ROW;
  const bool plain = part == 2 || (p.norm == HSA_NORM_NONE && !rotating);
  if (!plain) {
    F2 cs[4], sn[4];
    if (rotating)
      load_turns<kHalf>(p.table + static_cast<int64_t>(trow) * p.rot, at.a, at.b, at.turn_a,
                        at.turn_b, 1.0f, cs, sn);
    Planes g;  // weights of a norm over each head: the same for all heads
    const bool weighted = w != nullptr && p.norm != HSA_NORM_NONE;
    if (weighted && per_head) load_weights<kHalf>(w, at.a, at.b, g);
    float row_scale = 1.0f;
    if (per_row) {
      float ss = 0.f;
#pragma unroll
      for (int it = 0; it < NIT; ++it) {
        Planes f;
        get_planes<kHalf>(raw[it], f);
        ss += square_sum(f);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      row_scale = rsqrtf(ss / static_cast<float>(D) + p.eps);
    }
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      const int h = h0 + it * HG;
      Planes f;
      get_planes<kHalf>(raw[it], f);
      if (p.norm != HSA_NORM_NONE) {
        float scale = row_scale;
        if (per_head) {
          float ss = square_sum(f);
#pragma unroll
          for (int o = U / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          scale = rsqrtf(ss * (1.0f / HD) + p.eps);
        }
        if (weighted && per_row && h < p.H) load_weights<kHalf>(w + h * HD, at.a, at.b, g);
        const F2 s2 = splat(scale);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f.u[i] = mul_x2(f.u[i], s2);
          f.v[i] = mul_x2(f.v[i], s2);
          if (weighted) {
            f.u[i] = mul_x2(f.u[i], g.u[i]);
            f.v[i] = mul_x2(f.v[i], g.v[i]);
          }
        }
      }
      if (rotating) turn<kHalf>(f, cs, sn, at.turn_a, at.turn_b);
      set_planes<kHalf>(raw[it], f);
      if (h < p.H) {
        raw[it][0].store(dst + h * HD + at.a);
        raw[it][1].store(dst + h * HD + at.b);
      }
    }
    return;
  }
#pragma unroll
  for (int it = 0; it < NIT; ++it) {  // values go to the cache as they are
    const int h = h0 + it * HG;
    if (h < p.H) {
      raw[it][0].store(dst + h * HD + at.a);
      raw[it][1].store(dst + h * HD + at.b);
    }
  }
}

template <int HD, int NIT>
void qk_kernel(const Ctx& c, const QkParams& p, bool half_layout) {
  const int64_t items = static_cast<int64_t>(p.n) * p.parts;
  const unsigned grid = static_cast<unsigned>((items + kQkWarps - 1) / kQkWarps);
  if (half_layout) k_qk_norm_rope<HD, NIT, true><<<grid, 32 * kQkWarps, 0, c.stream>>>(p);
  else k_qk_norm_rope<HD, NIT, false><<<grid, 32 * kQkWarps, 0, c.stream>>>(p);
}

template <int HD>
cudaError_t launch_qk(const Ctx& c, const QkParams& p, bool half_layout) {
  constexpr int HG = 512 / HD;
  const int nit = (p.H + HG - 1) / HG;
  if (nit <= 1) qk_kernel<HD, 1>(c, p, half_layout);
  else if (nit <= 3) qk_kernel<HD, 3>(c, p, half_layout);
  else if (nit <= 6) qk_kernel<HD, 6>(c, p, half_layout);
  else if (nit <= 10) qk_kernel<HD, 10>(c, p, half_layout);
  else qk_kernel<HD, kMaxQkSteps>(c, p, half_layout);
  c.launches += 1;
  return cudaGetLastError();
}

template <typename T, int HD>
void rope_kernel(const Ctx& c, const RopeParams& p, bool half_layout) {
  const unsigned grid = (p.n + kRowWarps - 1) / kRowWarps;
  if (half_layout) k_rope<T, HD, true><<<grid, 32 * kRowWarps, 0, c.stream>>>(p);
  else k_rope<T, HD, false><<<grid, 32 * kRowWarps, 0, c.stream>>>(p);
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
  const int planes = f.half % 2 == 0 ? 2 : 1;  // two keep their 16-byte stores aligned
  const dim3 block(f.half / planes, 256 / (f.half / planes));
  // whole rounds of blocks, up to 8 on an SM, with some rows for each thread
  int64_t blocks = (static_cast<int64_t>(P) + 4 * block.y - 1) / (4 * block.y);
  if (blocks > c.num_sms * 8) blocks = c.num_sms * 8;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (planes == 2) k_rope_table<2><<<grid, block, 0, c.stream>>>(p);
  else k_rope_table<1><<<grid, block, 0, c.stream>>>(p);
  c.launches += 1;
  return cudaGetLastError();
}

cudaError_t launch_rope(const Ctx& c, const void* x, int64_t ld_x, bool f32, int n, int heads,
                        const float* table, int P, int rot, const int32_t* pos, bool half_layout,
                        bool inverse, void* out, int64_t ld_out) {
  const int hd = c.cfg.D / c.cfg.H;
  Timed timed(c, TC_ROWS, static_cast<double>(n) * ((f32 ? 8.0 : 4.0) * heads * hd + 4.0 * rot));
  const RopeParams p{x, out, ld_x, ld_out, table, pos, n, heads, P, rot, inverse ? -1.0f : 1.0f, c.flag};
  if (f32 && hd == 128) rope_kernel<float, 128>(c, p, half_layout);
  else if (f32) rope_kernel<float, 64>(c, p, half_layout);
  else if (hd == 128) rope_kernel<__nv_bfloat16, 128>(c, p, half_layout);
  else rope_kernel<__nv_bfloat16, 64>(c, p, half_layout);
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
  p.ascending = r.k_cache != nullptr && r.k_in == nullptr && r.idx != nullptr;
  p.pos = r.pos;
  p.n = r.n;
  p.N = c.cfg.N;
  p.P = a.P;
  p.H = H;
  p.rot = a.rot;
  p.norm = a.norm;
  p.eps = a.eps;
  p.flag = c.flag;
  // (without a table the layout only says where a unit's vectors lie)
  const bool half_layout = a.layout == HSA_ROPE_HALF;
  return hd == 128 ? launch_qk<128>(c, p, half_layout) : launch_qk<64>(c, p, half_layout);
}

}  // namespace hsa
