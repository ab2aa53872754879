// k_cross.cu - cross-attention of ragged sequences of queries to padded
// sequences of encoder states of another length, on the 5th-generation tensor
// cores.
//
//   o[m] = sum_j softmax_j(scale q[m] . k[b][j]) v[b][j],  b the sequence of
// row m, over the keys j < kv_len[b] whose mask byte is set.
//
// Arithmetic of a tile as in the active-query attention (k_attn.cu): two
// tiles of 128 rows share every 128-key tile, S and O live in TMEM,
// P is written over S as bf16 and read from there by the second product, and
// the two query tiles ping-pong.  P is rounded because that product takes both operands
// in V's type; the row sums add it unrounded in fp32.  A weight is off by 2^-8 of
// itself at most: 2.2e-3 of the output's norm against 64 bits, 1.7e-3 of it
// the output's own rounding.  What differs:
//  - A row is a query and a head: where several query heads share a key head, some
//    of them may lie side by side in a tile (launch_hd says when), so that short
//    sequences fill it.
//  - One persistent CTA per SM walks over units of two tiles.  Key
//    sets are short (a prompt is a few tiles), so a CTA per unit spent two
//    thirds of its time on its own start and end: the next unit's descriptor, Q
//    and first keys now arrive while this one's last tile is in softmax, and
//    its first scores are computed under this one's epilogue.  (26207 queries,
//    12 heads x 128, 512 and 384 keys: 145 us with a CTA per unit, 91 now.)
//  - Which rows and keys a unit covers is read on the device.  Units are
//    numbered per head (or packed heads) so that sequence b's first one is
//    floor(its first query / a unit's queries) + b: every sequence has room for its last,
//    partial unit, the host knows their number without knowing
//    the lengths, and a unit's sequence is found by a search over q_start
//    alone.  The producer warp finds the next unit that has rows and passes
//    its descriptor to the other warps through a ring of two.
//  - Key tiles before the first and after the last seen key are not loaded.
//    In tiles with unseen keys the scores are replaced by -inf and the unseen
//    rows of V are zeroed in shared memory before the product reads them: a
//    weight of 0 would not silence a NaN there.  (8190 queries, 4096 keys, 12 heads of
//    4 x 128: 195 us without a mask, 199 with all keys seen, 232 with a tenth unseen.)
//  - Rows without any key get zeros.  Warps whose 32 rows lie past the
//    sequence's end (one query a sequence) do no softmax.
//
// Warp 0: descriptors and TMA.  Warp 1: TMEM owner and MMA issuer.  Warps 2..5
// and 6..9: the softmax warpgroups of the two query tiles.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <string>

#include "attn_tile.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace hsa {

namespace {

constexpr int kQ = 128;        // rows (queries x packed heads) a tile has room for
constexpr int kMaxPack = 32;   // query heads side by side in a tile, at most
constexpr int kStages = 2;     // K and V ring depth
constexpr int kThreads = 320;
constexpr int kSoftmaxWarps = 8;
constexpr uint32_t kTmemCols = 512;
constexpr int kStageBytes = 32 * 128;  // per softmax warp: 32 output rows x 64 columns

template <int HD>
struct CrossCfg {
  static constexpr int kRegions = HD / 64;                    // 128-byte column regions
  static constexpr int kRegionBytes = 128 * 128;
  static constexpr int kTileBytes = kRegions * kRegionBytes;  // one Q, K or V tile
  static constexpr int kStageAt = kTileBytes * (2 + 2 * kStages);
  static constexpr int kBarsAt = kStageAt + kSoftmaxWarps * kStageBytes;
  // Every CTA takes all 512 TMEM columns, so only one may be resident per SM.
  static constexpr int kSmem = HD == 64 ? 160 * 1024 : kBarsAt + 1024 + 512;
  static constexpr uint32_t kColS = 0, kColO = 2 * kKV;  // two S tiles (P over S), two O tiles
};
static_assert(CrossCfg<64>::kBarsAt + 1024 + 512 <= CrossCfg<64>::kSmem &&
                  CrossCfg<128>::kSmem <= 227 * 1024,
              "cross-attention exceeds the shared memory of a CTA");

// What the warps of a CTA need to know of a unit (or of one key range of it).
struct UnitDesc {
  int q0, rows;  // first query, rows
  int b, h;      // sequence, group of packed query heads
  int j0, nkv;   // key tiles [j0, j0 + nkv); nkv < 0: no more units
  int len;       // keys of the sequence
  int part;      // index of this key range's partial result, or -1
};

struct CrossParams {
  int n, B, S, group;  // group: query heads per key head
  bool k_shared, v_shared;  // one key (value) sequence for all (or B = 1)
  float scale_log2;
  __nv_bfloat16* o;
  int ld;
  const int32_t* q_start;
  const int32_t* kv_len;
  const uint8_t* kv_mask;
  int* flag;
  // Row r of head group h is query r / pack of head h * pack + r % pack.  A tile has
  // whole queries, tile_q of them in `tile` rows, a unit twice as many.
  int pack, tile_q, tile, unit_q;
  uint32_t over_pack;             // 65536 / pack, rounded up: divides what is below 256
  uint32_t over_unit, unit_shift;  // 2^(32 + unit_shift) / unit_q, rounded up: divides below 2^31
  // Work: units_per_head * (H / pack) units, each in `split` key ranges; with more than
  // one, partial results are merged by k_cross_combine.
  int units_per_head, units, split;
  float* part_o;
  float2* part_ml;
};

__device__ __forceinline__ int clamped(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// First query of sequence b (b = B: one past the last).
__device__ __forceinline__ int first_row(const CrossParams& p, int b) {
  return p.q_start != nullptr ? clamped(__ldg(p.q_start + b), 0, p.n) : b * (p.n / p.B);
}

__device__ __forceinline__ int over_unit(const CrossParams& p, int q) {
  return static_cast<int>(__umulhi(static_cast<uint32_t>(q), p.over_unit) >> p.unit_shift);
}

__device__ __forceinline__ int over_pack(const CrossParams& p, int r) {
  return static_cast<int>(static_cast<uint32_t>(r) * p.over_pack >> 16);
}

// Where row r of a unit starts in o; the unit's first query is q0, its head group h.
template <int HD>
__device__ __forceinline__ __nv_bfloat16* out_row(const CrossParams& p, int h, int q0, int r) {
  const int q = over_pack(p, r);
  return p.o + static_cast<size_t>(q0 + q) * p.ld + (h * p.pack + r - q * p.pack) * HD;
}

// Sequence and queries [q0, q1) of unit u of a head, by a 32-way search over the
// sequences' first units; q0 >= q1: no rows.  Executed by whole warps.  The last
// step's lanes hold the rows (and with `len`, the key counts) of all sequences
// in question, so nothing is loaded again once the sequence is known.
__device__ __forceinline__ void unit_rows(const CrossParams& p, int u, int& b, int& q0, int& q1,
                                          int* keys = nullptr) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = p.B;
  for (;;) {
    const int step = (len + 31) / 32;
    const int i = lane * step;
    int row = 0, kv = p.S;
    bool at_or_before = false;
    if (i < len || (step == 1 && i == len)) {  // the one past the last ends it
      row = first_row(p, lo + i);
      at_or_before = i < len && over_unit(p, row) + lo + i <= u;
    }
    if (keys != nullptr && p.kv_len != nullptr && step == 1 && i < len)
      kv = clamped(__ldg(p.kv_len + lo + i), 0, p.S);
    const int c = __popc(__ballot_sync(0xffffffffu, at_or_before));
    if (c == 0) {  // before the first sequence
      b = 0, q0 = 1, q1 = 0;
      return;
    }
    if (step == 1) {
      b = lo + c - 1;
      const int first = __shfl_sync(0xffffffffu, row, c - 1);
      const int last = c < 32 ? __shfl_sync(0xffffffffu, row, c & 31) : first_row(p, b + 1);
      if (keys != nullptr) *keys = __shfl_sync(0xffffffffu, kv, c - 1);
      q0 = first + (u - (over_unit(p, first) + b)) * p.unit_q;
      q1 = min(last, q0 + p.unit_q);
      return;
    }
    const int next = lo + (c - 1) * step;
    len = min(step, lo + len - next);
    lo = next;
  }
}

// Bits of the first `left` of a tile's keys.
__device__ __forceinline__ void first_bits(int left, uint32_t (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = left - 32 * i;
    w[i] = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
  }
}

// First and last + 1 key tiles of a sequence that hold a seen key (lo == hi:
// none).  Executed by one warp.
__device__ __forceinline__ void seen_tiles(const CrossParams& p, int b, int len, int& lo, int& hi) {
  lo = 0;
  hi = (len + kKV - 1) / kKV;
  if (p.kv_mask == nullptr) return;
  const int lane = threadIdx.x & 31;
  const uint8_t* row = p.kv_mask + static_cast<int64_t>(b) * p.S;
  // a tile per step, from the front and from the back: 4 bytes a lane
  auto any_seen = [&](int tile) {
    bool see = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = tile * kKV + 32 * i + lane;
      see = see || (key < len && __ldg(row + key) != 0);
    }
    return __any_sync(0xffffffffu, see);
  };
  while (lo < hi && !any_seen(lo)) ++lo;
  while (hi > lo && !any_seen(hi - 1)) --hi;
}

__device__ __forceinline__ void hide(uint32_t (&sr)[kKV], const uint32_t (&w)[4]) {
#pragma unroll
  for (int e = 0; e < kKV; ++e)
    if (!((w[e >> 5] >> (e & 31)) & 1u)) sr[e] = __float_as_uint(-INFINITY);
}

template <int HD, bool kMask>
__global__ void __launch_bounds__(kThreads, 1)
    k_cross(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
            const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
            const __grid_constant__ CrossParams p) {
  using Cfg = CrossCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;                              // [2] tiles
  uint8_t* sK = sQ + 2 * Cfg::kTileBytes;          // [kStages]
  uint8_t* sV = sK + kStages * Cfg::kTileBytes;    // [kStages]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::kBarsAt);
  uint64_t* q_full = bars;
  uint64_t* q_empty = q_full + 1;
  uint64_t* k_full = q_empty + 1;
  uint64_t* k_empty = k_full + kStages;
  uint64_t* v_full = k_empty + kStages;
  uint64_t* v_empty = v_full + kStages;
  uint64_t* s_full = v_empty + kStages;  // [2][2] per query tile, its S tiles in turn
  uint64_t* p_full = s_full + 4;         // [2][2]
  uint64_t* o_done = p_full + 4;         // [2] per query tile
  uint64_t* d_full = o_done + 2;         // [2] descriptors
  uint64_t* d_empty = d_full + 2;        // [2]
  UnitDesc* desc = reinterpret_cast<UnitDesc*>(d_empty + 2);  // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(desc + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // a barrier per lane: q_full .. v_empty, s_full, p_full, o_done, d_full, d_empty
  constexpr int kP = 6 + 4 * kStages, kD = kP + 8;  // first of p_full and of d_empty
  if (warp == 0 && lane < kD + 2) {
    mbar_init(bars + lane, lane >= kD ? 1 + kSoftmaxWarps : lane >= kP && lane < kP + 4 ? 4 : 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  if (warp > 1 && p.tile < kQ) {  // rows of Q that no copy reaches
    const int per = (kQ - p.tile) * 8;
    for (int i = threadIdx.x - 64; i < 2 * Cfg::kRegions * per; i += 32 * kSoftmaxWarps)
      *reinterpret_cast<uint4*>(sQ + i / per * Cfg::kRegionBytes + p.tile * 128 + 16 * (i % per)) =
          make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  // The producer does not wait for the others' start: it set the barriers up
  // itself and uses no TMEM, so its search and first copies run under the
  // allocation.
  uint32_t tmem = 0;
  if (warp == 0) {
    __syncwarp();
    asm volatile("bar.arrive 1, %0;" ::"n"(kThreads) : "memory");
  } else {
    tc_fence_before();
    asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
    tc_fence_after();
    tmem = *tmem_slot;
  }
  bool ok = true;

  if (warp == 0) {
    // ------------------------------------------------------------ descriptors and TMA
    const uint64_t keep = l2_policy_evict_last();  // a sequence's K/V is shared by its units
    int it = 0;     // key tiles issued so far
    int nq = 0;     // units whose Q was issued
    int nd = 0;     // descriptors published
    int seen_b = -1, lo_tile = 0, hi_tile = 0, seen_len = 0;
    const int total = p.units * p.split;
    for (int item = blockIdx.x; ok; item += gridDim.x) {
      UnitDesc d{};
      d.nkv = -1;
      bool rows = true;
      if (item < total) {
        const int unit = item / p.split, piece = item - unit * p.split;
        d.h = unit / p.units_per_head;
        int keys = 0;
        int q1;
        unit_rows(p, unit - d.h * p.units_per_head, d.b, d.q0, q1, &keys);
        rows = d.q0 < q1;
        d.rows = (q1 - d.q0) * p.pack;
        if (rows) {
          if (d.b != seen_b) {
            seen_b = d.b;
            seen_len = keys;
            seen_tiles(p, d.b, seen_len, lo_tile, hi_tile);
          }
          d.len = seen_len;
          const int all = hi_tile - lo_tile;
          d.j0 = lo_tile + piece * all / p.split;
          d.nkv = lo_tile + (piece + 1) * all / p.split - d.j0;
          d.part = p.split > 1 ? item : -1;
        }
      }
      if (!rows) continue;
      if (lane == 0) {
        const int slot = nd & 1;
        ok = mbar_wait(&d_empty[slot], ((nd >> 1) & 1) ^ 1);
        if (ok) {
          desc[slot] = d;
          mbar_arrive(&d_full[slot]);  // releases the descriptor
        }
        const int ntile = d.rows > p.tile ? 2 : 1;
        const int bk = p.k_shared ? 0 : d.b, bv = p.v_shared ? 0 : d.b;
        const int head = d.h * p.pack, kcol = head / p.group * HD;
        for (int j = 0; j < d.nkv && ok; ++j, ++it) {
          const int s = it % kStages;
          const uint32_t ph = ((it / kStages) & 1) ^ 1;
          if (!mbar_wait(&k_empty[s], ph)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&k_full[s], Cfg::kTileBytes);
          for (int r = 0; r < Cfg::kRegions; ++r)
            tma_load_3d_hint(sK + s * Cfg::kTileBytes + r * Cfg::kRegionBytes, &tmK, &k_full[s],
                             kcol + 64 * r, (d.j0 + j) * kKV, bk, keep);
          if (j == 0) {
            // Q may be replaced once the previous unit's last scores are done
            if (!mbar_wait(q_empty, (nq & 1) ^ 1)) {
              (void)mbar_wait(&k_full[s], (it / kStages) & 1);
              ok = false;
              break;
            }
            ++nq;
            mbar_arrive_expect_tx(q_full, ntile * Cfg::kRegions * p.tile * 128);
            for (int t = 0; t < ntile; ++t)
              for (int r = 0; r < Cfg::kRegions; ++r)
                tma_load_3d(sQ + t * Cfg::kTileBytes + r * Cfg::kRegionBytes, &tmQ, q_full, 64 * r, head,
                            d.q0 + t * p.tile_q);
          }
          if (!mbar_wait(&v_empty[s], ph)) {
            (void)mbar_wait(&k_full[s], (it / kStages) & 1);
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&v_full[s], Cfg::kTileBytes);
          for (int r = 0; r < Cfg::kRegions; ++r)
            tma_load_3d_hint(sV + s * Cfg::kTileBytes + r * Cfg::kRegionBytes, &tmV, &v_full[s],
                             kcol + 64 * r, (d.j0 + j) * kKV, bv, keep);
        }
        if (!ok) {  // let copies already in flight land before the CTA exits
          if (nq > 0) (void)mbar_wait(q_full, (nq - 1) & 1);
          for (int k = it > kStages ? it - kStages : 0; k < it; ++k) {
            (void)mbar_wait(&k_full[k % kStages], (k / kStages) & 1);
            (void)mbar_wait(&v_full[k % kStages], (k / kStages) & 1);
          }
        }
        ++nd;
      }
      ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0) != 0;
      if (item >= total) break;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idS = idesc_bf16(kQ, kKV, false, false);
      constexpr uint32_t idPV = idesc_bf16(kQ, HD, false, true);
      // This thread's own work shows: descriptors are one sum each (their low bits
      // are addresses / 16), and the tile index is known to the compiler (26207
      // queries, 12 heads x 128: 90.6 us; 91.6 with descriptors built for each
      // instruction, 99 with the tile index in a register as well).
      const uint64_t q_desc = sdesc_sw128(smem_u32(sQ), 16, 1024), k_desc = sdesc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t v_desc = sdesc_sw128(smem_u32(sV), Cfg::kRegionBytes, 1024);
      auto issue_s = [&](int t, int s, int buf) {
        const uint64_t a = q_desc + t * (Cfg::kTileBytes >> 4), b = k_desc + s * (Cfg::kTileBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          const int off = ((kk >> 2) * Cfg::kRegionBytes + (kk & 3) * 32) >> 4;
          umma_bf16(tmem + Cfg::kColS + buf * kKV, a + off, b + off, idS, kk > 0 ? 1u : 0u);
        }
      };
      auto issue_pv = [&](int t, int s, int buf, bool acc) {
        const uint64_t b = v_desc + s * (Cfg::kTileBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < kKV / 16; ++kk)
          umma_bf16_ta(tmem + Cfg::kColO + t * HD, tmem + Cfg::kColS + buf * kKV + kk * 8,
                       b + kk * (2048 >> 4), idPV, (acc || kk > 0) ? 1u : 0u);
      };
      int it = 0, nq = 0;  // key tiles (also: S tiles of query tile 0), units with keys
      int n1 = 0;          // S tiles of query tile 1
      for (int nd = 0;; ++nd) {
        if (!mbar_wait(&d_full[nd & 1], (nd >> 1) & 1)) {
          ok = false;
          break;
        }
        const int nkv = desc[nd & 1].nkv;
        const int ntile = desc[nd & 1].rows > p.tile ? 2 : 1;
        mbar_arrive(&d_empty[nd & 1]);
        if (nkv < 0) break;
        if (nkv == 0) continue;
        ok = mbar_wait(q_full, nq & 1);
        if (!ok) break;
        ++nq;
        auto scores = [&](int t, int j, int buf) {
          const int s = (it + j) % kStages, nth = (t == 0 ? it : n1) + j;
          if (t == 0 && !mbar_wait(&k_full[s], ((it + j) / kStages) & 1)) return false;
          tc_fence_after();
          issue_s(t, s, buf);
          umma_commit(&s_full[2 * t + (nth & 1)]);
          if (t == ntile - 1) umma_commit(&k_empty[s]);
          if (t == ntile - 1 && j == nkv - 1) umma_commit(q_empty);
          return true;
        };
        auto values = [&](int t, int j, int buf) {
          const int s = (it + j) % kStages, nth = (t == 0 ? it : n1) + j;
          // p_full of query tile 0 also says that the unseen rows of this V tile are zeroed
          if (!mbar_wait(&p_full[2 * t + (nth & 1)], (nth >> 1) & 1)) return false;
          if (t == 0 && !mbar_wait(&v_full[s], ((it + j) / kStages) & 1)) return false;
          tc_fence_after();
          issue_pv(t, s, buf, j > 0);
          if (t == ntile - 1) umma_commit(&v_empty[s]);
          if (j == nkv - 1) umma_commit(&o_done[t]);
          return true;
        };
        // Scores follow the P V that leaves their buffer: the tensor pipe works in
        // order, so that product has read P by then.
        if (ntile == 2) {  // a buffer each
          ok = scores(0, 0, 0) && scores(1, 0, 1);
          for (int j = 0; j < nkv && ok; ++j)
#pragma unroll
            for (int t = 0; t < 2 && ok; ++t) ok = values(t, j, t) && (j + 1 == nkv || scores(t, j + 1, t));
          n1 += nkv;
        } else {
          // A lone query tile takes both in turn: its next scores are computed under
          // its softmax (100 queries, 12 heads x 128, 512 keys: 12.3 us with one
          // buffer, 10.6 with both).
          ok = scores(0, 0, 0) && (nkv == 1 || scores(0, 1, 1));
          for (int j = 0; j < nkv && ok; ++j) ok = values(0, j, j & 1) && (j + 2 >= nkv || scores(0, j + 2, j & 1));
        }
        it += nkv;
        if (!ok) break;
      }
    }
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    const int t = (warp - 2) >> 2;  // query tile of this warpgroup
    const int qd = warp & 3;        // TMEM lane quarter
    const int row = 32 * qd + lane;
    const uint32_t lane_base = static_cast<uint32_t>(32 * qd) << 16;
    const uint32_t tO = tmem + lane_base + Cfg::kColO + t * HD;
    uint8_t* stage = smem + Cfg::kStageAt + (warp - 2) * kStageBytes;
    if (blockIdx.x == 0) {  // while nothing has arrived yet, one CTA looks the offsets and lengths over
      for (int i = threadIdx.x - 64; i < p.B; i += 32 * kSoftmaxWarps) {
        const int a = p.q_start != nullptr ? p.q_start[i] : 0, e = p.q_start != nullptr ? p.q_start[i + 1] : 0;
        const int len = p.kv_len != nullptr ? p.kv_len[i] : 0;
        if (a < 0 || e > p.n || a > e || len < 0 || len > p.S) atomicOr(p.flag, DEV_BAD_INDEX);
      }
      __syncwarp();
    }
    int it = 0, ns = 0, no = 0;  // key tiles of the CTA, S tiles and units of this query tile
    for (int nd = 0; ok; ++nd) {
      if (!__all_sync(0xffffffffu, mbar_wait(&d_full[nd & 1], (nd >> 1) & 1))) {
        ok = false;
        break;
      }
      const UnitDesc d = desc[nd & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&d_empty[nd & 1]);
      if (d.nkv < 0) break;
      const int warp_row = t * p.tile + 32 * qd;              // this warp's first row of the unit
      const int warp_end = min(d.rows, (t + 1) * p.tile);     // its last one is before this
      if (d.nkv == 0) {  // no key in this range: zeros, or an empty part
        const int rows = min(32, warp_end - warp_row);
        if (d.part >= 0) {
          if (lane < rows)
            p.part_ml[static_cast<size_t>(d.part) * 2 * kQ + t * kQ + row] = make_float2(-FLT_MAX, 0.f);
        } else {
          for (int r = 0; r < rows; ++r)
            if (lane < HD / 8)
              *reinterpret_cast<uint4*>(out_row<HD>(p, d.h, d.q0, warp_row + r) + 8 * lane) =
                  make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      const int ntile = d.rows > p.tile ? 2 : 1;
      if (t >= ntile) {
        it += d.nkv;
        continue;
      }
      const bool mine = warp_row < warp_end;  // whether any of this warp's rows exists
      const uint8_t* mrow = kMask ? p.kv_mask + static_cast<int64_t>(d.b) * p.S : nullptr;
      // the mask bytes of a tile's keys, four a lane, loaded one tile ahead
      uint32_t bytes[4] = {0u, 0u, 0u, 0u};
      auto load_bytes = [&](int j) {
        if (kMask) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = j * kKV + 32 * i + lane;
            bytes[i] = key < d.len ? __ldg(mrow + key) : 0u;
          }
        }
      };
      // Zeroes the unseen rows of this tile's V (whatever they hold must not meet a
      // weight of 0), while the scores are computed.
      auto clear_unseen = [&](const uint32_t (&see)[4]) {
        if (t != 0 || (see[0] & see[1] & see[2] & see[3]) == 0xffffffffu) return true;
        if (!__all_sync(0xffffffffu, mbar_wait(&v_full[it % kStages], (it / kStages) & 1))) return false;
        const uint32_t mine4 = qd == 0 ? see[0] : qd == 1 ? see[1] : qd == 2 ? see[2] : see[3];
        if (!((mine4 >> lane) & 1u)) {
          // eight lanes in a row start from bank groups of their own
          const int at = (it % kStages) * Cfg::kTileBytes + row * 128 + 16 * (lane & 7);
#pragma unroll
          for (int r = 0; r < Cfg::kRegions; ++r)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(sV + ((at + r * Cfg::kRegionBytes) ^ (16 * i))) =
                  make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        return true;
      };
      load_bytes(d.j0);
      float m_run = -FLT_MAX, l_run = 0.f;
      for (int j = 0; j < d.nkv; ++j, ++it, ++ns) {
        uint32_t see[4];
        if (kMask) {
#pragma unroll
          for (int i = 0; i < 4; ++i) see[i] = __ballot_sync(0xffffffffu, bytes[i] != 0u);
          if (j + 1 < d.nkv) load_bytes(d.j0 + j + 1);
        } else {
          first_bits(d.len - (d.j0 + j) * kKV, see);
        }
        const bool whole = (see[0] & see[1] & see[2] & see[3]) == 0xffffffffu;  // same for all rows
        const uint32_t tS = tmem + lane_base + Cfg::kColS + ((ntile == 2 ? t : j) & 1) * kKV;
        // A lone query tile may be two tiles ahead of P V: only its scores say then that
        // the load before has reached the stage, and so which phase its barrier is in.
        const auto scored = [&] {
          return __all_sync(0xffffffffu, mbar_wait(&s_full[2 * t + (ns & 1)], (ns >> 1) & 1)) != 0;
        };
        if ((ntile == 1 && j >= 2 && !scored()) || !clear_unseen(see) || !scored()) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (mine) {
          uint32_t sr[kKV];
          tmem_ld128(tS, sr);
          if (!whole) hide(sr, see);
          // As in k_attn.cu: after the first tile the exponentials are taken
          // against the running max as it stands, and only a row sum past 2^64
          // (rare) has S read again, the max raised and O and l rescaled.  A
          // row that has seen no key yet keeps the lowest finite max, so its
          // first key takes that way too.
          float m_use = m_run, alpha = 1.0f, rs;
          if (j == 0) m_use = fmaxf(row_max(sr) * p.scale_log2, -FLT_MAX);
          uint32_t w[kKV / 2];
#pragma unroll 1
          for (int pass = 0;; ++pass) {
            rs = exp_row(sr, p.scale_log2, m_use, w);
            const bool over = !(rs <= kSumLimit);
            if (j == 0 || pass == 1 || !__any_sync(0xffffffffu, over)) break;
            // a lone query tile's last P V may still be adding to O (the one before is
            // done: it was issued ahead of these scores)
            if (ntile == 1 &&
                !__all_sync(0xffffffffu, mbar_wait(&v_empty[(it - 1) % kStages], ((it - 1) / kStages) & 1))) {
              ok = false;
              break;
            }
            tc_fence_after();
            tmem_ld128(tS, sr);
            if (!whole) hide(sr, see);
            const float tmax = row_max(sr) * p.scale_log2;
            if (over) {
              m_use = fmaxf(tmax, m_run);
              alpha = ex2_approx(m_run - m_use);
            }
#pragma unroll 1
            for (int c = 0; c < HD / 32; ++c) {
              uint32_t r[32];
              tmem_ld32(tO + 32 * c, r);
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
              tmem_st32(tO + 32 * c, r);
            }
            tmem_ld128(tS, sr);
            if (!whole) hide(sr, see);
          }
          tmem_st64(tS, w);
          l_run = l_run * alpha + rs;
          m_run = m_use;
        }
        if (!ok) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * t + (ns & 1)]);
      }
      if (!ok) break;
      // epilogue: O / l -> bf16 rows through this warp's stage, or, for a
      // key-range part, the unnormalised O with its (m, l) for k_cross_combine
      if (!__all_sync(0xffffffffu, mbar_wait(&o_done[t], no & 1))) {
        ok = false;
        break;
      }
      ++no;
      if (!mine) continue;
      tc_fence_after();
      if (d.part >= 0) {
        const size_t prow = static_cast<size_t>(d.part) * 2 * kQ + t * kQ + row;
        const bool real = warp_row + lane < warp_end;
        if (real) p.part_ml[prow] = make_float2(m_run, l_run);
#pragma unroll 1
        for (int c = 0; c < HD / 32; ++c) {
          uint32_t r[32];
          __syncwarp();
          tmem_ld32(tO + 32 * c, r);
          if (real) {
            float4* d4 = reinterpret_cast<float4*>(p.part_o + prow * HD + 32 * c);
#pragma unroll
            for (int v = 0; v < 8; ++v)
              d4[v] = make_float4(__uint_as_float(r[4 * v]), __uint_as_float(r[4 * v + 1]),
                                  __uint_as_float(r[4 * v + 2]), __uint_as_float(r[4 * v + 3]));
          }
        }
      } else {
        const float inv = 1.0f / l_run;
        const int g = lane & 7;
#pragma unroll 1
        for (int c = 0; c < HD / 32; ++c) {
          uint32_t r[32];
          __syncwarp();
          tmem_ld32(tO + 32 * c, r);
          if (!(c & 1)) {  // the stage may still be on its way out
            if (lane == 0) tma_store_wait_read();
            __syncwarp();
          }
          // this lane's row of the stage: 64 columns, 16-byte group v at v ^ (row & 7)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            *reinterpret_cast<uint4*>(stage + lane * 128 + 16 * ((4 * (c & 1) + v) ^ (lane & 7))) = make_uint4(
                pack_bf16(__uint_as_float(r[8 * v]) * inv, __uint_as_float(r[8 * v + 1]) * inv),
                pack_bf16(__uint_as_float(r[8 * v + 2]) * inv, __uint_as_float(r[8 * v + 3]) * inv),
                pack_bf16(__uint_as_float(r[8 * v + 4]) * inv, __uint_as_float(r[8 * v + 5]) * inv),
                pack_bf16(__uint_as_float(r[8 * v + 6]) * inv, __uint_as_float(r[8 * v + 7]) * inv));
          if (!(c & 1)) continue;
          if (warp_row + 32 <= warp_end && p.tile == kQ) {
            // 32 rows of this sequence, whole queries: one tiled store, which this warp does not
            // wait for (an SM stores about 32 bytes a clock: 2000 clocks a unit)
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(&tmO, stage, 32 * (c - 1), d.h * p.pack, d.q0 + over_pack(p, warp_row));
              tma_store_commit();
            }
          } else {
            // the next rows are another sequence's: one store covers four rows
            // and 128 contiguous bytes of each
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int rr = 4 * k + (lane >> 3);
              if (warp_row + rr < warp_end)
                *reinterpret_cast<uint4*>(out_row<HD>(p, d.h, d.q0, warp_row + rr) + 32 * (c - 1) + 8 * g) =
                    *reinterpret_cast<const uint4*>(stage + rr * 128 + 16 * (g ^ (rr & 7)));
            }
            __syncwarp();
          }
        }
      }
    }
    if (lane == 0) tma_store_wait();  // also keeps the stage until it is read
  }
  if (!ok) atomicOr(p.flag, DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Merge the key-range parts of the split units: one warp per query row,
// O = sum_i O_i 2^(m_i - M) / sum_i l_i 2^(m_i - M) with M = max_i m_i.  Parts
// without a key (l = 0) hold no O.
template <int HD>
__global__ void __launch_bounds__(256) k_cross_combine(const __grid_constant__ CrossParams p) {
  const int lane = threadIdx.x & 31;
  const int rr = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int unit = blockIdx.y;
  const int h = unit / p.units_per_head;
  int b, q0, q1;
  unit_rows(p, unit - h * p.units_per_head, b, q0, q1);
  const int row = rr / kQ * p.tile + rr % kQ;  // of the unit
  if (rr % kQ >= p.tile || row >= (q1 - q0) * p.pack) return;
  const size_t part0 = static_cast<size_t>(blockIdx.y) * p.split;
  float M = -FLT_MAX;
  for (int i = 0; i < p.split; ++i) M = fmaxf(M, p.part_ml[(part0 + i) * 2 * kQ + rr].x);
  constexpr int kPer = HD / 32;
  float acc[kPer];
#pragma unroll
  for (int c = 0; c < kPer; ++c) acc[c] = 0.f;
  float L = 0.f;
  for (int i = 0; i < p.split; ++i) {
    const size_t prow = (part0 + i) * 2 * kQ + rr;
    const float2 ml = p.part_ml[prow];
    if (ml.y == 0.f) continue;
    const float wgt = ex2_approx(ml.x - M);
    L += ml.y * wgt;
    const float* po = p.part_o + prow * HD;
#pragma unroll
    for (int c = 0; c < kPer; ++c) acc[c] += po[lane + 32 * c] * wgt;
  }
  const float inv = L == 0.f ? 0.f : 1.0f / L;
  __nv_bfloat16* orow = out_row<HD>(p, h, q0, row);
#pragma unroll
  for (int c = 0; c < kPer; ++c) orow[lane + 32 * c] = __float2bfloat16_rn(acc[c] * inv);
}

template <int HD>
cudaError_t launch_hd(const Ctx& c, const hsa_cross_args& a, std::string* why) {
  const int D = c.cfg.D, H = c.cfg.H;
  const bool k1 = a.B == 1 || a.bs_k == 0, v1 = a.B == 1 || a.bs_v == 0;
  const uint64_t width = static_cast<uint64_t>(a.kv_heads) * HD;
  CrossParams p{};
  p.n = a.n;
  p.B = a.B;
  p.S = a.S;
  p.group = H / a.kv_heads;
  // Packed heads and key ranges per unit: the rounds of CTAs times the tiles of a
  // range, plus two tiles' time for a unit's own ends and six for the merge,
  // whichever is least.  Packing the query heads of a key head fills the tiles
  // of short sequences (16 sequences of one query, 40 heads of 8 x 128, 1000 keys: 59 us
  // with heads of their own, 18.7 with five a tile); where it saves no round, heads
  // of their own load less at once (100 queries, 24 heads of 4 x 128, 512 keys:
  // 12.7 us, 14.5 with two a tile).
  const int tiles = (a.S + kKV - 1) / kKV;
  constexpr int kMaxUnits = 0x3fffffff / kMaxSplitParts;
  int64_t best = INT64_MAX;
  for (int pack = 1; pack <= kMaxPack; ++pack) {
    if (p.group % pack != 0) continue;
    const int64_t units64 = (static_cast<int64_t>(a.n / (2 * (kQ / pack))) + a.B) * (H / pack);
    if (units64 > kMaxUnits) continue;
    const int units = static_cast<int>(units64);
    for (int sp = 1; sp <= tiles && sp <= kMaxSplitParts && (sp == 1 || units * sp <= kMaxAttnParts); ++sp) {
      const int rounds = (units * sp + c.num_sms - 1) / c.num_sms;
      const int64_t cost = static_cast<int64_t>(rounds) * ((tiles + sp - 1) / sp + 2) + (sp > 1 ? 6 : 0);
      if (cost >= best) continue;
      best = cost;
      p.units = units;
      p.units_per_head = units / (H / pack);
      p.pack = pack;
      p.split = sp;
    }
  }
  if (p.units == 0) {
    if (why) *why = "too many sequences";
    return cudaErrorInvalidValue;
  }
  p.tile_q = kQ / p.pack;
  p.tile = p.tile_q * p.pack;
  p.unit_q = 2 * p.tile_q;
  p.over_pack = static_cast<uint32_t>((65536 + p.pack - 1) / p.pack);
  while ((2 << p.unit_shift) < p.unit_q) ++p.unit_shift;
  const uint64_t scaled = 1ull << (32 + p.unit_shift);
  p.over_unit = static_cast<uint32_t>((scaled + p.unit_q - 1) / p.unit_q);
  const uint32_t heads = p.pack;  // Q and O as [queries][heads][columns]
  CUtensorMap tq, tk, tv, to;
  if (!make_tmap_bf16_3d(&tq, a.q, a.n, H, HD, HD, D, heads, why, p.tile_q)) return cudaErrorInvalidValue;
  if (!make_tmap_bf16_3d(&tk, a.k, k1 ? 1 : a.B, a.S, width, a.ld_k, k1 ? a.ld_k * a.S : a.bs_k, kKV, why))
    return cudaErrorInvalidValue;
  if (!make_tmap_bf16_3d(&tv, a.v, v1 ? 1 : a.B, a.S, width, a.ld_v, v1 ? a.ld_v * a.S : a.bs_v, kKV, why))
    return cudaErrorInvalidValue;
  if (!make_tmap_bf16_3d(&to, a.o, a.n, H, HD, HD, D, heads, why, 32 % heads == 0 ? 32 / heads : 1)) return cudaErrorInvalidValue;
  p.k_shared = k1;
  p.v_shared = v1;
  const double scale = a.scale != 0.f ? a.scale : 1.0 / sqrt(static_cast<double>(HD));
  p.scale_log2 = static_cast<float>(1.4426950408889634 * scale);
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.ld = D;
  p.q_start = a.q_start;
  p.kv_len = a.kv_len;
  p.kv_mask = a.kv_mask;
  p.flag = c.flag;
  constexpr int smem = CrossCfg<HD>::kSmem;
  static std::atomic<uint64_t> smem_set[2] = {};  // per device
  const bool mask = a.kv_mask != nullptr;
  {
    const cudaError_t e = mask ? ensure_smem_limit(k_cross<HD, true>, smem, c.device, smem_set[1])
                               : ensure_smem_limit(k_cross<HD, false>, smem, c.device, smem_set[0]);
    if (e != cudaSuccess) return e;
  }
  p.part_o = c.attn_part_o;
  p.part_ml = reinterpret_cast<float2*>(c.attn_part_ml);
  const int items = p.units * p.split;
  const unsigned grid = static_cast<unsigned>(items < c.num_sms ? items : c.num_sms);
  if (mask) k_cross<HD, true><<<grid, kThreads, smem, c.stream>>>(tq, tk, tv, to, p);
  else k_cross<HD, false><<<grid, kThreads, smem, c.stream>>>(tq, tk, tv, to, p);
  c.launches += 1;
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.split == 1) return e;
  k_cross_combine<HD><<<dim3(2 * kQ / 8, p.units), 256, 0, c.stream>>>(p);
  c.launches += 1;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cross_attention(const Ctx& c, const hsa_cross_args& a, std::string* why) {
  Timed timed(c, TC_ATTN, 4.0 * a.n * a.S * c.cfg.D);  // every key seen
  bool taken = false;
  const cudaError_t e = launch_cross_few(c, a, &taken);
  if (taken) return e;
  return c.cfg.D / c.cfg.H == 128 ? launch_hd<128>(c, a, why) : launch_hd<64>(c, a, why);
}

}  // namespace hsa
