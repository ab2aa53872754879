// k_cross_few.cu - cross-attention where sequences have a few queries each
// (single tokens, guided pairs of them): hsa_cross_attention's result without
// the 128-query tiles of k_cross.cu, which such sequences leave empty.
//
// Every key and value is read once for up to kFewRows rows that share it (the queries of
// a sequence times the query heads of a key head), so what bounds this is HBM
// and, before that, the bytes in flight.  A lane group of d / 8 lanes owns a
// key: 16 bytes of K and of V a lane, kBatch keys at a time.  Scores are
// summed over the group by shuffles; each group keeps its own running maximum,
// sum and output in fp32 (weights are never rounded to 16 bits here), and these are
// merged over the groups of a warp by shuffles, over the warps of a CTA in shared
// memory and over the CTAs of a cluster, which split the keys when there are
// few sequences, through distributed shared memory.  16 sequences of one query,
// 12 heads x 128, up to 512 keys: 11.5 us (the bytes alone take 5.5).

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "internal.h"
#include "ptx.cuh"

namespace hsa {

namespace {

constexpr int kBatch = 4;    // keys of a lane group at a time
constexpr int kFewRows = 4;  // rows of one pass over the keys

// Warps of a CTA: four rows' states fill the registers of half as many threads
// (16 sequences, 4 rows a key head, 2000 keys: 24 us with eight warps, 17 with four).
template <int R>
constexpr int warps_of() {
  return R == kFewRows ? 4 : 8;
}

// With more rows than one, few warps fit an SM and the next batch is on its way into
// shared memory while one is used (16 sequences, 2 rows a key head, 1024 keys: 24.1 us
// against 26.9, 4 rows, 2000 keys: 14.6 against 16.5).  One row's threads have their batch in
// registers: three CTAs an SM cover for one another (tokens as above: 11.5 us, 12.4 with the ring).
template <int R>
constexpr int ring_bytes() {
  return R == 1 ? 0 : 2 * kBatch * 2 * 16 * 32 * warps_of<R>();
}

struct FewParams {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* o;
  int64_t ld_k, bs_k, ld_v, bs_v;
  int ld;  // D
  int n, B, S, kv_heads, group, split;
  float scale_log2;
  float even;  // passes of sequences of equal length, as further_rows numbers them: sequences a pass
  const int32_t *q_start, *kv_len;
  const uint8_t* kv_mask;
  int* flag;
};

__device__ __forceinline__ int clamped(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

__device__ __forceinline__ void unpack8(const uint4& w, float (&f)[8]) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(r[i] << 16);
    f[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
  }
}

// Running softmax state of one row in one lane: maximum (log2 units), sum, and
// this lane's 8 output places, all relative to the maximum.
struct Run {
  float m, l, o[8];
  // Takes in another state of the same row (of other keys).
  __device__ __forceinline__ void merge(float m2, float l2, const float (&o2)[8]) {
    const float top = fmaxf(m, m2), a = ex2_approx(m - top), b = ex2_approx(m2 - top);
    m = top;
    l = l * a + l2 * b;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = o[i] * a + o2[i] * b;
  }
};

// A sequence of more than R rows (queries x the heads of a key head) takes more passes over
// its keys than the one by the CTA of its number.  These are numbered so that
// sequence b's second one is floor(its first row / R): with floor(x + y) >= floor(x) +
// floor(y) every sequence has room for its own, and their number is at most
// floor(n group / R) <= B (launch_cross_few chooses R so).  So each CTA has one
// at most beside its first, however unequal the sequences are: pass `slot`, here found
// in q_start as sequence b and first row r0 (b = -1: no such pass).  (32 sequences of
// 12 heads x 128, 512 keys, 31 with one query and one with 97: 59 us; 362 with all of a
// sequence's passes in one CTA.)
//
// Where sequences fill their pass, sequence `slot` (rows [q0, q1)) has the pass's number
// itself.  Else the search begins with the 32 sequences around the place that even
// lengths would give it, whose offsets arrive with the CTA's own.  (16 sequences of one
// query: 10.8 us with and without, 4 rows a key head 27.2 and 26.7; a search of all of q_start after the
// first pass 11.8 and 28.0.)
template <int R>
__device__ __forceinline__ void further_rows(const FewParams& p, int slot, int q0, int q1, int& b, int& r0) {
  const int lane = threadIdx.x & 31;
  b = -1, r0 = 0;
  if (p.q_start == nullptr || slot >= p.n * p.group / R) return;  // (equal parts have R rows at most)
  int step = 1, len = p.B;
  int lo = max(0, min(static_cast<int>(slot * p.even), p.B - 16) - 15);
  int row = __ldg(p.q_start + min(lo + lane, p.B));
  if (q0 * p.group / R <= slot && slot < q1 * p.group / R) {
    r0 = (slot - q0 * p.group / R + 1) * R;
    if (r0 < (q1 - q0) * p.group) b = slot;
    return;
  }
  // lane i: whether the numbers of sequence lo + i step begin at or before slot
  for (bool guessed = true;; guessed = false) {
    const int i = lo + lane * step;
    row = clamped(guessed ? row : __ldg(p.q_start + min(i, p.B)), 0, p.n);
    const int at = row * p.group / R;
    const uint32_t begun = __ballot_sync(0xffffffffu, i < (guessed ? p.B : lo + len) && at <= slot);
    const int c = __popc(begun);
    if (c > 0 && step == 1 && (c < 32 || !guessed)) {
      const int first = __shfl_sync(0xffffffffu, at, c - 1), first_row = __shfl_sync(0xffffffffu, row, c - 1);
      const int next = c < 32 ? __shfl_sync(0xffffffffu, row, c & 31) : clamped(__ldg(p.q_start + lo + 32), 0, p.n);
      r0 = (slot - first + 1) * R;
      if (first <= slot && r0 < (next - first_row) * p.group) b = lo + c - 1;
      return;
    }
    if (guessed) {
      if (c == 0 && lo == 0) return;  // rows before the first sequence
      lo = 0;
    } else {
      if (c == 0) return;
      lo += (c - 1) * step;
      len = min(step, len - (c - 1) * step);
    }
    step = (len + 31) / 32;
  }
}

template <int HD, int R>
__global__ void __launch_bounds__(32 * warps_of<R>(), R == 1 ? 3 : 2)
    k_cross_few(const __grid_constant__ FewParams p) {
  constexpr int kWarps = warps_of<R>();
  constexpr int L = HD / 8, G = 32 / L;  // lanes per key, keys per warp step
  __shared__ float s_ml[kWarps][R][2];
  __shared__ __align__(16) float s_o[kWarps][R][HD];
  __shared__ float c_ml[R][2];
  __shared__ __align__(16) float c_o[R][HD];
  constexpr bool kRing = ring_bytes<R>() > 0;
  extern __shared__ __align__(16) uint4 ring[];  // [2][kBatch][K, V][thread]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane / L, e = 8 * (lane % L);  // key of the warp's step, first place of this lane

  const int rank = blockIdx.x % p.split;
  const int item = blockIdx.x / p.split;
  const int kvh = item % p.kv_heads, slot = item / p.kv_heads;
  const int each = p.n / p.B;  // rows a sequence where q_start is not given
  const int raw0 = p.q_start != nullptr ? __ldg(p.q_start + slot) : slot * each;
  const int raw1 = p.q_start != nullptr ? __ldg(p.q_start + slot + 1) : raw0 + each;
  int raw_len = p.kv_len != nullptr ? __ldg(p.kv_len + slot) : p.S;
  int q0 = clamped(raw0, 0, p.n), q1 = clamped(raw1, 0, p.n);
  if (threadIdx.x == 0 && (raw0 < 0 || raw1 > p.n || raw0 > raw1 || raw_len < 0 || raw_len > p.S))
    atomicOr(p.flag, DEV_BAD_INDEX);
  // First the first rows of sequence `slot`, then further rows of a longer one, if there
  // are such: the same for every CTA of the cluster.
  int further, further_r0;
  further_rows<R>(p, slot, q0, q1, further, further_r0);
  for (int turn = 0; turn < 2; ++turn) {
    const int b = turn == 0 ? slot : further, r0 = turn == 0 ? 0 : further_r0;
    if (b < 0) break;
    if (turn > 0) {
      q0 = clamped(__ldg(p.q_start + b), 0, p.n);
      q1 = clamped(__ldg(p.q_start + b + 1), 0, p.n);
      if (p.kv_len != nullptr) raw_len = __ldg(p.kv_len + b);
    }
    const int rows = (q1 - q0) * p.group;
    if (r0 >= rows) continue;
    const int len = clamped(raw_len, 0, p.S);
    const __nv_bfloat16* kb = p.k + b * p.bs_k + kvh * HD + e;
    const __nv_bfloat16* vb = p.v + b * p.bs_v + kvh * HD + e;
    const uint8_t* mask = p.kv_mask == nullptr ? nullptr : p.kv_mask + static_cast<int64_t>(b) * p.S;
    // this CTA's keys, a multiple of a warp's batch
    const int per = ((len + p.split - 1) / p.split + G * kBatch - 1) / (G * kBatch) * (G * kBatch);
    const int first = min(len, rank * per), last = min(len, first + per);

    // A thread copies and reads its own places only, so the ring has no barriers.
    auto place = [&](int stage, int u, int kv) -> uint4& {
      return ring[((stage * kBatch + u) * 2 + kv) * (32 * kWarps) + threadIdx.x];
    };
    uint8_t ahead[kBatch];  // whether the keys on their way are seen
    auto fetch = [&](int j0, int stage) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int j = j0 + u * G + g;
        ahead[u] = 0;
        if (j < last) {
          cp_async16(&place(stage, u, 0), kb + j * p.ld_k);
          cp_async16(&place(stage, u, 1), vb + j * p.ld_v);
          ahead[u] = mask != nullptr ? __ldg(mask + j) : 1;
        }
      }
      cp_async_commit();
    };
    constexpr int kStep = kWarps * G * kBatch;
    int stage = 0;
    if (kRing) fetch(first + warp * G * kBatch, 0);
    float qf[R][8];
    Run run[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int rr = min(r0 + r, rows - 1);
      const int head = kvh * p.group + rr % p.group;
      unpack8(__ldg(reinterpret_cast<const uint4*>(
                  p.q + static_cast<int64_t>(q0 + rr / p.group) * p.ld + head * HD + e)),
              qf[r]);
#pragma unroll
      for (int i = 0; i < 8; ++i) qf[r][i] *= p.scale_log2, run[r].o[i] = 0.f;
      run[r].m = -FLT_MAX;
      run[r].l = 0.f;
    }
    for (int j0 = first + warp * G * kBatch; j0 < last; j0 += kStep, stage ^= 1) {
      uint4 kr[kBatch], vr[kBatch];
      bool see[kBatch];
      if (kRing) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) see[u] = ahead[u] != 0;
        fetch(j0 + kStep, stage ^ 1);
        cp_async_wait<1>();
#pragma unroll
        for (int u = 0; u < kBatch; ++u) kr[u] = place(stage, u, 0), vr[u] = place(stage, u, 1);
      } else {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int j = j0 + u * G + g;
          see[u] = j < last;
          kr[u] = vr[u] = make_uint4(0u, 0u, 0u, 0u);
          if (see[u]) {
            kr[u] = __ldg(reinterpret_cast<const uint4*>(kb + j * p.ld_k));
            vr[u] = __ldg(reinterpret_cast<const uint4*>(vb + j * p.ld_v));
            if (mask != nullptr) see[u] = __ldg(mask + j) != 0;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u)  // a weight of 0 would not silence a NaN
        if (!see[u]) vr[u] = make_uint4(0u, 0u, 0u, 0u);
      float s[R][kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        float kf[8];
        unpack8(kr[u], kf);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float d = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) d = fmaf(qf[r][i], kf[i], d);
          s[r][u] = d;
        }
      }
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int u = 0; u < kBatch; ++u) s[r][u] += __shfl_xor_sync(0xffffffffu, s[r][u], o);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float top = run[r].m;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          if (!see[u]) s[r][u] = -INFINITY;
          top = fmaxf(top, s[r][u]);
        }
        const float keep = ex2_approx(run[r].m - top);
        run[r].m = top;
        run[r].l *= keep;
#pragma unroll
        for (int i = 0; i < 8; ++i) run[r].o[i] *= keep;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          s[r][u] = ex2_approx(s[r][u] - top);
          run[r].l += s[r][u];
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        float vf[8];
        unpack8(vr[u], vf);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < 8; ++i) run[r].o[i] = fmaf(s[r][u], vf[i], run[r].o[i]);
      }
    }
    if (kRing) cp_async_wait<0>();
    // the lane groups of the warp
#pragma unroll
    for (int o = L; o < 32; o <<= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float o2[8];
        const float m2 = __shfl_xor_sync(0xffffffffu, run[r].m, o);
        const float l2 = __shfl_xor_sync(0xffffffffu, run[r].l, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) o2[i] = __shfl_xor_sync(0xffffffffu, run[r].o[i], o);
        run[r].merge(m2, l2, o2);
      }
    // the warps of the CTA
    if (g == 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (e == 0) s_ml[warp][r][0] = run[r].m, s_ml[warp][r][1] = run[r].l;
        float4* dst = reinterpret_cast<float4*>(&s_o[warp][r][e]);
        dst[0] = make_float4(run[r].o[0], run[r].o[1], run[r].o[2], run[r].o[3]);
        dst[1] = make_float4(run[r].o[4], run[r].o[5], run[r].o[6], run[r].o[7]);
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < R * HD; i += 32 * kWarps) {
      const int r = i / HD, c = i % HD;
      float top = -FLT_MAX;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w][r][0]);
      float l = 0.f, o = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2_approx(s_ml[w][r][0] - top);
        l = fmaf(s_ml[w][r][1], f, l);
        o = fmaf(s_o[w][r][c], f, o);
      }
      if (p.split == 1) {
        if (r0 + r < rows) {
          const int rr = r0 + r, head = kvh * p.group + rr % p.group;
          p.o[static_cast<int64_t>(q0 + rr / p.group) * p.ld + head * HD + c] =
              __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
        }
      } else {
        c_o[r][c] = o;
        if (c == 0) c_ml[r][0] = top, c_ml[r][1] = l;
      }
    }
    if (p.split == 1) {
      __syncthreads();  // the next rows reuse the shared memory
      continue;
    }
    cluster_sync();
    // the CTAs of the cluster: rank k writes the places c with c % split == k
    for (int i = threadIdx.x; i < R * (HD / p.split); i += 32 * kWarps) {
      const int r = i / (HD / p.split), c = i % (HD / p.split) * p.split + rank;
      float m[8], l[8], o[8];
      float top = -FLT_MAX;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k >= p.split) break;
        m[k] = ld_cluster_f32(&c_ml[r][0], k);
        l[k] = ld_cluster_f32(&c_ml[r][1], k);
        o[k] = ld_cluster_f32(&c_o[r][c], k);
        top = fmaxf(top, m[k]);
      }
      float ls = 0.f, os = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k >= p.split) break;
        const float f = ex2_approx(m[k] - top);
        ls = fmaf(l[k], f, ls);
        os = fmaf(o[k], f, os);
      }
      if (r0 + r < rows) {
        const int rr = r0 + r, head = kvh * p.group + rr % p.group;
        p.o[static_cast<int64_t>(q0 + rr / p.group) * p.ld + head * HD + c] =
            __float2bfloat16_rn(ls == 0.f ? 0.f : os / ls);
      }
    }
    cluster_sync();  // no CTA reuses or leaves its state while another may read it
  }
}

template <int HD, int R>
cudaError_t launch_rows(const Ctx& c, const FewParams& p) {
  constexpr int smem = ring_bytes<R>();
  static std::atomic<uint64_t> smem_set = {};  // per device
  cudaError_t e = smem > 0 ? ensure_smem_limit(k_cross_few<HD, R>, smem, c.device, smem_set) : cudaSuccess;
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = smem;
  cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.kv_heads * p.split);
  cfg.blockDim = dim3(32 * warps_of<R>());
  cfg.stream = c.stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k_cross_few<HD, R>, p);
  c.launches += 1;
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_cross_few(const Ctx& c, const hsa_cross_args& a, bool* taken) {
  const int H = c.cfg.H, hd = c.cfg.D / H, group = H / a.kv_heads;
  const int64_t items = static_cast<int64_t>(a.B) * a.kv_heads;
  // One pass over the keys for a sequence of average length (see further_rows for
  // longer ones).  With more rows the
  // 128-row tiles are as fast (16 sequences, 2 key heads, 2000 keys: 4 rows a key
  // head 14.3 us here, 8 rows 15.4 there).
  const int64_t rows = static_cast<int64_t>(a.n) * group;
  *taken = rows <= static_cast<int64_t>(a.B) * kFewRows && items * 8 < 0x7fffffff;
  if (!*taken) return cudaSuccess;
  FewParams p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k = static_cast<const __nv_bfloat16*>(a.k);
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.ld_k = a.ld_k;
  p.bs_k = a.bs_k;
  p.ld_v = a.ld_v;
  p.bs_v = a.bs_v;
  p.ld = c.cfg.D;
  p.n = a.n;
  p.B = a.B;
  p.S = a.S;
  p.kv_heads = a.kv_heads;
  p.group = group;
  const double scale = a.scale != 0.f ? a.scale : 1.0 / sqrt(static_cast<double>(hd));
  p.scale_log2 = static_cast<float>(1.4426950408889634 * scale);
  p.q_start = a.q_start;
  p.kv_len = a.kv_len;
  p.kv_mask = a.kv_mask;
  p.flag = c.flag;
  // Keys over a cluster while there are fewer than two CTAs an SM and each
  // keeps a batch for every warp.
  const int batch = 8 * kBatch * (256 / hd);
  p.split = 1;
  while (p.split < 8 && items * p.split < 2 * c.num_sms && a.S >= 2 * p.split * batch) p.split *= 2;
  const int r = rows <= a.B ? 1 : rows <= 2 * static_cast<int64_t>(a.B) ? 2 : kFewRows;
  p.even = static_cast<float>(static_cast<double>(a.B) * r / static_cast<double>(rows));
  if (hd == 128)
    return r == 1 ? launch_rows<128, 1>(c, p) : r == 2 ? launch_rows<128, 2>(c, p) : launch_rows<128, kFewRows>(c, p);
  return r == 1 ? launch_rows<64, 1>(c, p) : r == 2 ? launch_rows<64, 2>(c, p) : launch_rows<64, kFewRows>(c, p);
}

}  // namespace hsa
