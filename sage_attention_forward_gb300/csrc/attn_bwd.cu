// Attention backward, sm_103a: the gradients of Q, K and V from dO, with the probabilities
// formed again from the row statistics that the forward left (attn_lse.cu).
//
//   p_ij  = exp(scale * q_i . k_j - lse_i)   over the keys j < limit(i)  (attn_tiles.cuh)
//   delta_i = dO_i . o_i                     (= sum_j p_ij dp_ij)
//   dp_ij = dO_i . v_j
//   ds_ij = p_ij (dp_ij - delta_i)
//   dV_j  = sum_i p_ij dO_i,   dK_j = scale sum_i ds_ij q_i,   dQ_i = scale sum_j ds_ij k_j
//
// with the sums over i also over the Hq / Hkv query heads that share a key head.  A row that sees
// one key has p = 1 whatever its score, so its ds is 0; it is set so, and not left to the
// rounding of dp - delta.
//
// Two kernels, no atomics: every sum has one order.
//   dq_kernel     one item per (128 queries, query head): Q and dO stay, K and V stream by:
//                 S = Q K^T, dP = dO V^T, dQ += dS K, its key tiles last first.  It forms delta of its
//                 rows from dO, which it has, and O, and at the end again from the sums of their dS; it leaves
//                 -lse * log2 e and the better -delta in the workspace, padded to whole tiles (-inf and 0 there
//                 and for empty rows: their probabilities come out as 0).
//   dkdv_kernel   one item per (128 keys, key head): K and V stay in shared memory, Q and dO tiles
//                 stream by with those statistics.  The transposed scores S^T = K Q^T and
//                 dP^T = V dO^T leave P^T and dS^T in TMEM as the A operands of dV += P^T dO and
//                 dK += dS^T Q.
// (A kernel of its own for the statistics read dO once more: 48 us of 386 at 16896 queries on 512 keys.)
// Seven products of a tile pair against five if one kernel did both, but a dQ that several CTAs
// add into needs either atomics, whose order changes the result, or 64 KB of FP32 traffic a
// tile pair: at 2560 cycles a pair and 152 SMs that is 7 TB/s of reductions in L2.
//
// P is rounded to BF16 for dV, dS to BF16 for dK and dQ (relative 2^-8 at most each; the unrounded
// P forms dS); every sum is FP32.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attn_tiles.cuh"
#include "kernels.h"

namespace sa {
namespace {

using namespace tiles;

// Four warpgroups share a tile's elementwise work, 32 of its 128 columns each: with two, of 64,
// the tensor core waited on their latency (dK/dV 3408 cycles a tile pair against 2048 of products).
constexpr int kGroups = 4;
constexpr int kCols = kTile / kGroups;
constexpr int kWarpLoad = 4 * kGroups;
constexpr int kWarpMma = kWarpLoad + 1;   // and the next
constexpr int kWarpClear = kWarpMma + 2;
constexpr int kThreads = 32 * (kWarpClear + 1);
// Products before an item's last at which the load warp, itself two or three ahead of the tensor core, asks
// for the next item: early enough to hide the answer's way, and late, because an SM that has asked has to
// take what it got (asked for at the start of the item, 256 items of unequal length left the
// first SMs with a second long one: 409 us of a backward in place of 332).
constexpr int kAskAhead = 5;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kHot = 0.51f;        // (dq_kernel) a key with more of a row's probability is its only one, roundings and all
constexpr float kLeastSum = 1e-6f;   // (dq_kernel) of a row's probabilities in a tile, to be divided by

__device__ uint32_t g_err_bwd;
std::atomic<bool> g_launched{false};

__device__ __forceinline__ float u2f(uint32_t u) { return __uint_as_float(u); }

// ------------------------------------------------------------------ dK, dV
struct BwdParams {
  Mask mask;
  float c_log2;           // softmax_scale * log2 e
  float scale;            // softmax_scale
  float* neg_lse2;        // [B * Hq, Sq_pad]: written by dq_kernel, read by dkdv_kernel
  float* neg_delta;
  int Sq_pad;
  const float* lse;         // [B, Hq, Sq] (dq_kernel)
  const __nv_bfloat16* k;   // (dq_kernel) K, for the keys that take their row's rest
  long long k_str[3];
  __nv_bfloat16 *d0, *d1;   // dQ; or dK and dV
  long long s0[3], s1[3];   // their element strides (b, s, h)
  int H, group;             // heads of this grid (Hkv, or Hq), Hq / Hkv
  Div by_H, by_group;
  Order order;
  // dkdv_kernel: the parts that a key tile's products are divided into, each an item; with more than
  // one, their sums as FP32 [unit][part][dV, dK][32 pieces of four channels][128 keys][4]
  int parts;
  Div by_parts;
  float4* partial;
};

// Q(i) is held from S(i) to dK(i), most of two steps, and S(i+2) follows dK(i) closely: with two
// slots the products waited for Q.
constexpr int kQRing = 3, kDRing = 2;

struct __align__(1024) SmemKV {
  uint8_t k[kTileBytes];
  uint8_t v[kTileBytes];
  uint8_t q[kQRing][kTileBytes];
  uint8_t dout[kDRing][kTileBytes];
  alignas(16) float neg_lse2[2][kTile];
  alignas(16) float neg_delta[2][kTile];
  WorkRing work;
  uint64_t k_full, k_empty, v_full, v_empty;
  uint64_t q_full[kQRing], q_empty[kQRing];
  uint64_t d_full[kDRing], d_empty[kDRing];
  uint64_t r_full[2], r_empty[2];   // the row statistics
  uint64_t s_full, dp_full;
  uint64_t p_full[2], ds_full[2];   // queries [0, 64) and [64, 128) of P^T, dS^T stored in TMEM (two warpgroups each)
  uint64_t acc_done;
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t abort_flag;
};

// 128 keys of one key head (a unit), with the query tiles of the heads that share it.
struct UnitKV {
  int b, hk, key0, keys, first, n_q, n;   // n: products with a query tile, 0 when no query sees a key
};
__device__ __forceinline__ UnitKV unit_kv(const BwdParams& p, int index) {
  UnitKV i;
  int tile, head;
  Work w;
  w.index = index;
  work_place(p.order, w, tile, head);
  i.b = div_by(head, p.by_H);
  i.hk = head - i.b * p.H;
  i.key0 = tile * kTile;
  i.n_q = (p.mask.Sq + kTile - 1) / kTile;
  i.keys = key_count(p.mask, i.b);
  // causal: query i sees key j when j <= i + Sk - Sq, so the tile's first key starts the queries
  i.first = p.mask.causal ? max(i.key0 - (p.mask.Sk - p.mask.Sq), 0) / kTile : 0;
  i.n = i.key0 < i.keys ? max(i.n_q - i.first, 0) * p.group : 0;
  return i;
}
// Products of each part but the last of a unit with n (parts without any stay unwritten).
__device__ __forceinline__ int part_length(const BwdParams& p, int n) { return div_by(n + p.parts - 1, p.by_parts); }

// One item: a part of a unit, from query tile t of the h-th head that shares the keys on.
struct ItemKV : UnitKV {
  int t, h;
};
template <bool kParts>
__device__ __forceinline__ ItemKV item_kv(const BwdParams& p, const Work& w) {
  ItemKV i;
  const int unit = kParts ? div_by(w.index, p.by_parts) : w.index;
  static_cast<UnitKV&>(i) = unit_kv(p, unit);
  i.t = i.first;
  i.h = 0;
  if (kParts) {
    const int len = part_length(p, i.n), start = (w.index - unit * p.parts) * len;
    i.n = max(min(i.n - start, len), 0);
    if (i.n > 0) {
      i.h = start / (i.n_q - i.first);
      i.t = i.first + start % (i.n_q - i.first);
    }
  }
  return i;
}

// kParts: units in parts (the other form has not their code: with it the loop took 3 % longer).
template <bool kParts>
__global__ void __launch_bounds__(kThreads, 1)
    dkdv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_d,
                const BwdParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  SmemKV& sm = *reinterpret_cast<SmemKV*>(smem_raw);
  if (smem_misaligned(smem_raw, &g_err_bwd)) return;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);   // (known to be uniform)
  const int lane = threadIdx.x & 31;
  volatile uint32_t* abort_flag = &sm.abort_flag;
  uint32_t* err = &g_err_bwd;

  if (threadIdx.x == 0) {
    work_init(sm.work, kWarpLoad + 1);   // readers: softmax, MMA
    mbar_init(&sm.k_full, 1);
    mbar_init(&sm.k_empty, 1);
    mbar_init(&sm.v_full, 1);
    mbar_init(&sm.v_empty, 1);
    for (int s = 0; s < kQRing; ++s) {
      mbar_init(&sm.q_full[s], 1);
      mbar_init(&sm.q_empty[s], 1);
    }
    for (int s = 0; s < kDRing; ++s) {
      mbar_init(&sm.d_full[s], 1);
      mbar_init(&sm.d_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.r_full[s], 1);
      mbar_init(&sm.r_empty[s], kWarpLoad);
      mbar_init(&sm.p_full[s], 2 * kGroups);
      mbar_init(&sm.ds_full[s], 2 * kGroups);
    }
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.dp_full, 1);
    mbar_init(&sm.acc_done, 1);
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  griddep_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;   // all 512 columns are this CTA's: they start at 0
  const int off = p.mask.Sk - p.mask.Sq;

  if (warp == kWarpLoad) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      tma_prefetch_desc(&tm_d);
      int it = 0, items = 0, requests = 0, q_issued = 0, d_issued = 0, r_issued = 0, k_issued = 0, v_issued = 0;
      Work w = first_work();
      auto ask_next = [&]() -> bool {
        if (!work_request(sm.work, w.t + 1, abort_flag, err)) return false;
        ++requests;
        return true;
      };
      auto load_item = [&](const ItemKV& i) -> bool {
        if (items > 0 && !wait_sleep(&sm.k_empty, (items - 1) & 1, abort_flag, err, kErrTimeoutSync)) return false;
        mbar_arrive_expect_tx(&sm.k_full, kTileBytes);
        load_tile(sm.k, &tm_k, &sm.k_full, i.key0, i.hk, i.b);
        ++k_issued;
        int t = i.t, h = i.hk * p.group + i.h;
        const int ask = max(i.n - kAskAhead, 0);
        for (int j = 0; j < i.n; ++j, ++it) {
          if (j == ask && !ask_next()) return false;
          const int qs = it % kQRing, qu = it / kQRing, ds = it % kDRing, du = it / kDRing, rs = it & 1, ru = it >> 1;
          if (qu > 0 && !wait_sleep(&sm.q_empty[qs], (qu - 1) & 1, abort_flag, err, kErrTimeoutSync)) return false;
          mbar_arrive_expect_tx(&sm.q_full[qs], kTileBytes);
          if (!withheld(q_issued++)) load_tile(sm.q[qs], &tm_q, &sm.q_full[qs], t * kTile, h, i.b);
          if (j == 0) {
            if (items > 0 && !wait_sleep(&sm.v_empty, (items - 1) & 1, abort_flag, err, kErrTimeoutSync)) return false;
            mbar_arrive_expect_tx(&sm.v_full, kTileBytes);
            load_tile(sm.v, &tm_v, &sm.v_full, i.key0, i.hk, i.b);
            ++v_issued;
          }
          if (du > 0 && !wait_sleep(&sm.d_empty[ds], (du - 1) & 1, abort_flag, err, kErrTimeoutSync)) return false;
          mbar_arrive_expect_tx(&sm.d_full[ds], kTileBytes);
          load_tile(sm.dout[ds], &tm_d, &sm.d_full[ds], t * kTile, h, i.b);
          ++d_issued;
          if (ru > 0 && !wait_sleep(&sm.r_empty[rs], (ru - 1) & 1, abort_flag, err, kErrTimeoutSync)) return false;
          const long long at = ((long long)i.b * p.H * p.group + h) * p.Sq_pad + t * kTile;
          mbar_arrive_expect_tx(&sm.r_full[rs], 2 * kTile * 4);
          bulk_load(sm.neg_lse2[rs], p.neg_lse2 + at, kTile * 4, &sm.r_full[rs]);
          bulk_load(sm.neg_delta[rs], p.neg_delta + at, kTile * 4, &sm.r_full[rs]);
          ++r_issued;
          if (++t == i.n_q) {
            t = i.first;
            ++h;
          }
        }
        ++items;
        return true;
      };
      do {
        const ItemKV i = item_kv<kParts>(p, w);
        if (!(i.n > 0 ? load_item(i) : ask_next())) break;
      } while (work_next_load(sm.work, w, abort_flag, err));
      if (*abort_flag) {
        // nothing may land in this CTA's shared memory after it has gone
        work_teardown(sm.work, requests);
        if (k_issued) mbar_wait_teardown(&sm.k_full, (k_issued - 1) & 1);
        if (v_issued) mbar_wait_teardown(&sm.v_full, (v_issued - 1) & 1);
        for (int i = max(q_issued - kQRing, 0); i < q_issued; ++i)
          mbar_wait_teardown(&sm.q_full[i % kQRing], (i / kQRing) & 1);
        for (int i = max(d_issued - kDRing, 0); i < d_issued; ++i)
          mbar_wait_teardown(&sm.d_full[i % kDRing], (i / kDRing) & 1);
        for (int i = max(r_issued - 2, 0); i < r_issued; ++i) mbar_wait_teardown(&sm.r_full[i & 1], (i >> 1) & 1);
      }
    }
  } else if (warp == kWarpMma) {
    // The tensor core's order is dV(i) S(i+1) dK(i) dP(i+1), over the tile products i of all items:
    // S(i+1) overwrites P(i) and dP(i+1) dS(i) after the products that read them, and while the
    // softmax warps work on one of the two chains S -> P -> dV and dP -> dS -> dK the tensor core
    // works on the other.  (A warp for each chain let their products alternate: 10 % slower.)  An
    // item's first dV and dK overwrite the accumulators of the item before: the softmax warps
    // published that P and dS after they had read them.
    const bool leader = elect_one();
    constexpr uint32_t tS = 0, tDP = 128, tDV = 256, tDK = 384;
    const uint32_t dk = desc_k(sm.k), dv = desc_k(sm.v), dq = desc_k(sm.q[0]), dd = desc_k(sm.dout[0]);
    const uint32_t dq_mn = desc_mn(sm.q[0]), dd_mn = desc_mn(sm.dout[0]);
    int k_items = 0, v_items = 0;
    auto make = [&](const Work& w) { return item_kv<kParts>(p, w); };
    Walk<ItemKV, decltype(make)> walk(make);
    int f0 = walk.next(sm.work, lane, abort_flag, err);
    // (a step's ring slots are compile-time constants, and so are the distances of its descriptors)
    auto issue_s = [&](auto u_c, int i, int flags) -> bool {
      constexpr int slot = decltype(u_c)::value % kQRing;
      if ((flags & kFirst) && !wait_warp(&sm.k_full, k_items++ & 1, abort_flag, err, kErrTimeoutTma)) return false;
      if (!wait_warp(&sm.q_full[slot], (i / kQRing) & 1, abort_flag, err, kErrTimeoutTma)) return false;
      tc_fence_after();
      mma_tile_nt(tS, dk, dq + kDescTile * slot, leader);
      if (leader) mma_commit(&sm.s_full);
      if (leader && (flags & kLast)) mma_commit(&sm.k_empty);
      return true;
    };
    auto issue_dp = [&](auto u_c, int i, int flags) -> bool {
      constexpr int slot = decltype(u_c)::value % kDRing;
      if ((flags & kFirst) && !wait_warp(&sm.v_full, v_items++ & 1, abort_flag, err, kErrTimeoutTma)) return false;
      if (!wait_warp(&sm.d_full[slot], (i / kDRing) & 1, abort_flag, err, kErrTimeoutTma)) return false;
      tc_fence_after();
      mma_tile_nt(tDP, dv, dd + kDescTile * slot, leader);
      if (leader) mma_commit(&sm.dp_full);
      if (leader && (flags & kLast)) mma_commit(&sm.v_empty);
      return true;
    };
    // acc (+)= A B, A in kGroups pieces at columns a, a + kCols, ..., as the halves' barriers complete
    auto issue_acc = [&](uint32_t acc, uint32_t a, uint64_t* bars, uint32_t tile_mn, int i, bool first) -> bool {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (!wait_warp(&bars[half], i & 1, abort_flag, err, kErrTimeoutSync)) return false;
        tc_fence_after();
#pragma unroll
        for (int g = half * kGroups / 2; g < (half + 1) * kGroups / 2; ++g)
          mma_tile_part_nn<kCols>(acc, a + kCols * g, tile_mn, g, !first || g > 0, leader);
      }
      return true;
    };
    constexpr int kCopies = kQRing * kDRing;
    auto step = [&](auto u_c, int i) -> bool {
      constexpr int u = decltype(u_c)::value, qs = u % kQRing, ds = u % kDRing;
      const std::integral_constant<int, (u + 1) % kCopies> next_c;
      const bool last = f0 & kLast, first = f0 & kFirst;
      if (!last) f0 = walk.next(sm.work, lane, abort_flag, err);
      if (!issue_acc(tDV, tS, sm.p_full, dd_mn + kDescTile * ds, i, first)) return false;
      if (leader) mma_commit(&sm.d_empty[ds]);   // (dP(i) was issued before)
      if (!last && !issue_s(next_c, i + 1, f0)) return false;
      if (!issue_acc(tDK, tDP, sm.ds_full, dq_mn + kDescTile * qs, i, first)) return false;
      if (leader) mma_commit(&sm.q_empty[qs]);
      if (!last) return issue_dp(next_c, i + 1, f0);
      if (leader) mma_commit(&sm.acc_done);
      f0 = walk.next(sm.work, lane, abort_flag, err);
      return f0 == kEnd || (issue_s(next_c, i + 1, f0) && issue_dp(next_c, i + 1, f0));
    };
    const std::integral_constant<int, 0> c0;
    bool ok = f0 == kEnd || (issue_s(c0, 0, f0) && issue_dp(c0, 0, f0));
    for (int i = 0; ok && f0 != kEnd; i += kCopies) {
      ok = step(c0, i);
      if (ok && f0 != kEnd) ok = step(std::integral_constant<int, 1>(), i + 1);
      if (ok && f0 != kEnd) ok = step(std::integral_constant<int, 2>(), i + 2);
      if (ok && f0 != kEnd) ok = step(std::integral_constant<int, 3>(), i + 3);
      if (ok && f0 != kEnd) ok = step(std::integral_constant<int, 4>(), i + 4);
      if (ok && f0 != kEnd) ok = step(std::integral_constant<int, 5>(), i + 5);
    }
    static_assert(kCopies == 6, "six copies of the step");
    if (leader) mma_commit(&sm.drain);
    mbar_wait_teardown(&sm.drain, 0);
  } else if (warp < kWarpLoad) {
    // Warpgroup g takes the queries [32 g, 32 g + 32) of each tile.  A thread has eight of these
    // columns of four keys (rows lane / 4 + 8 r of its warp's 32), not 32 columns of one: the
    // statistics, which belong to the columns, are then 8 values a thread and not 32 (the
    // shared-memory reads of 32 took 420 cycles of the 1260 from a tile's S to its P).
    const int g = warp >> 2, wq = warp & 3;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + kCols * g, tDP = tS + 128;
    const int col = kCols * g + 2 * (lane & 3);   // the first of the thread's columns
    constexpr uint32_t kLow = 16u << 16;          // the lower 16 of the warp's 32 TMEM lanes
    bool ok = true;
    int it = 0, items = 0, turn = 0;
    do {
      {
        const ItemKV item = item_kv<kParts>(p, work_read(sm.work, turn));
        const int key = item.key0 + wq * 32 + (lane >> 2);   // and the keys 8, 16, 24 after it
        const int t_first = item.first, t_end = item.n_q;
        int t = item.t;
        for (int end = it + item.n; it != end; ++it) {
          const int slot = it & 1;
          // a tile on the diagonal: the thread's column 8 i + e sees its key r from
          // 8 i + e >= 8 r + c_min on.  Key 0's first query sees key 0 alone; its ds is 0.
          const int c_min = p.mask.causal ? key - off - t * kTile - col : -kTile;
          const bool diag = __any_sync(0xffffffffu, c_min + 24 > 0);
          float pr[2][16];
          ok = mbar_wait_warp<false>(&sm.r_full[slot], (it >> 1) & 1, abort_flag, err, kErrTimeoutTma) &&
               mbar_wait_warp<false>(&sm.s_full, it & 1, abort_flag, err, kErrTimeoutMma);
          if (!ok) break;
          tc_fence_after();
          {
            uint32_t a[2][16];
            tmem_ld_16x32(tS, a[0]);
            tmem_ld_16x32(tS + kLow, a[1]);
            float2 m[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) m[i] = *reinterpret_cast<const float2*>(&sm.neg_lse2[slot][col + 8 * i]);
            tmem_ld_wait();
            tmem_reg_fence16(a[0]);
            tmem_reg_fence16(a[1]);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int e = 4 * i + 2 * (r & 1);
                float x0, x1;
                ffma2(x0, x1, u2f(a[r >> 1][e]), u2f(a[r >> 1][e + 1]), p.c_log2, p.c_log2, m[i].x, m[i].y);
                pr[r >> 1][e] = ex2_approx(x0);
                pr[r >> 1][e + 1] = ex2_approx(x1);
              }
            if (diag) {
#pragma unroll
              for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                  float& x = pr[r >> 1][4 * (c >> 1) + 2 * (r & 1) + (c & 1)];
                  x = 8 * (c >> 1) + (c & 1) - 8 * r >= c_min ? x : 0.0f;
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t pk[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) pk[e] = pack_bf16x2(pr[h][2 * e], pr[h][2 * e + 1]);
              tmem_st_16x16(tS + h * kLow, pk);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_full[g >> 1]);
          }
          ok = mbar_wait_warp<false>(&sm.dp_full, it & 1, abort_flag, err, kErrTimeoutMma);
          if (!ok) break;
          tc_fence_after();
          {
            uint32_t a[2][16];
            tmem_ld_16x32(tDP, a[0]);
            tmem_ld_16x32(tDP + kLow, a[1]);
            float2 d[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = *reinterpret_cast<const float2*>(&sm.neg_delta[slot][col + 8 * i]);
            tmem_ld_wait();
            tmem_reg_fence16(a[0]);
            tmem_reg_fence16(a[1]);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int e = 4 * i + 2 * (r & 1);
                float x0, x1;
                fadd2(x0, x1, u2f(a[r >> 1][e]), u2f(a[r >> 1][e + 1]), d[i].x, d[i].y);
                fmul2(pr[r >> 1][e], pr[r >> 1][e + 1], pr[r >> 1][e], pr[r >> 1][e + 1], x0, x1);
              }
            if (diag) {
              const int c_min_ds = key == 0 ? c_min + 1 : c_min;
#pragma unroll
              for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                  float& x = pr[r >> 1][4 * (c >> 1) + 2 * (r & 1) + (c & 1)];
                  x = 8 * (c >> 1) + (c & 1) - 8 * r >= (r == 0 ? c_min_ds : c_min) ? x : 0.0f;
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t pk[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) pk[e] = pack_bf16x2(pr[h][2 * e], pr[h][2 * e + 1]);
              tmem_st_16x16(tDP + h * kLow, pk);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&sm.ds_full[g >> 1]);
              mbar_arrive(&sm.r_empty[slot]);
            }
          }
          if (++t == t_end) t = t_first;
        }
      }
      if (!ok) break;
      // warpgroups 0 and 1 store dV's channels, 2 and 3 dK's; keys that no query sees get zeros (their
      // rows hold what the padding made of them), and a key alone in its batch entry has dK = 0
      const ItemKV done = item_kv<kParts>(p, work_read(sm.work, turn));
      const int which = g / (kGroups / 2), ch = (g % (kGroups / 2)) * 64;
      const int row0 = done.key0 + wq * 32;
      const long long* str = which == 0 ? p.s1 : p.s0;
      const uint32_t acc = tmem + lane_off + 256 + 128 * which + ch;
      if (done.n > 0) {
        ok = mbar_wait_warp<false>(&sm.acc_done, items++ & 1, abort_flag, err, kErrTimeoutMma);
        if (!ok) break;
        tc_fence_after();
      }
      if (!kParts) {
        uint32_t out[32] = {};
        if (done.n > 0) {
          load_row_bf16<64>(acc, out, which == 0 ? 1.0f : p.scale);
          if (row0 + lane >= done.keys || (which == 1 && done.keys == 1)) {
#pragma unroll
            for (int e = 0; e < 32; ++e) out[e] = 0u;
          }
        }
        store_rows<64>((which == 0 ? p.d1 : p.d0) + (long long)done.b * str[0] + (long long)row0 * str[1] +
                           (long long)done.hk * str[2] + ch,
                       str[1], out, p.mask.Sk - row0, lane);
      } else if (done.n > 0) {
        // (a piece of four channels of a warp's rows is one contiguous store)
        float4* dst = p.partial + ((long long)work_read(sm.work, turn).index * 2 + which) * (32 * kTile) +
                      (ch / 4) * kTile + wq * 32 + lane;
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          uint32_t a[32];
          tmem_ld32(acc + 32 * cc, a);
          tmem_ld_wait();
          tmem_reg_fence(a);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[(8 * cc + e) * kTile] =
                make_float4(u2f(a[4 * e]), u2f(a[4 * e + 1]), u2f(a[4 * e + 2]), u2f(a[4 * e + 3]));
        }
      }
      tc_fence_before();
      work_release(sm.work, turn, lane);
    } while (work_wait(sm.work, ++turn, abort_flag, err));
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) {
    __syncwarp();
    tmem_dealloc(sm.tmem_base, 512);
  }
}

// The parts of a unit's dV and dK in their order, rounded once.  A thread has eight channels of a key.
constexpr int kJoinThreads = 256;
constexpr int kJoinBlocks = 2 * kTile * (128 / 8) / kJoinThreads;   // of a unit
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const BwdParams p) {
  griddep_wait();
  const int index = blockIdx.x / kJoinBlocks, at = (blockIdx.x % kJoinBlocks) * kJoinThreads + threadIdx.x;
  const UnitKV u = unit_kv(p, index);
  // four lanes have 32 channels of a key, a warp eight keys
  const int key = (at >> 2) % kTile, rest = (at >> 2) / kTile, c8 = (at & 3) + 4 * (rest & 3), which = rest >> 2;
  if (u.key0 + key >= p.mask.Sk) return;
  float sum[8] = {};
  if (u.n > 0 && u.key0 + key < u.keys && !(which == 1 && u.keys == 1)) {
    const int len = part_length(p, u.n);
    const float4* src = p.partial + ((long long)index * p.parts * 2 + which) * (32 * kTile) + 2 * c8 * kTile + key;
#pragma unroll 4
    for (int done = 0; done < u.n; done += len, src += 2 * 32 * kTile) {
      const float4 x = __ldcg(src), y = __ldcg(src + kTile);
      sum[0] += x.x;
      sum[1] += x.y;
      sum[2] += x.z;
      sum[3] += x.w;
      sum[4] += y.x;
      sum[5] += y.y;
      sum[6] += y.z;
      sum[7] += y.w;
    }
  }
  const float f = which == 0 ? 1.0f : p.scale;
  const long long* str = which == 0 ? p.s1 : p.s0;
  uint4 out;
  out.x = pack_bf16x2(sum[0] * f, sum[1] * f);
  out.y = pack_bf16x2(sum[2] * f, sum[3] * f);
  out.z = pack_bf16x2(sum[4] * f, sum[5] * f);
  out.w = pack_bf16x2(sum[6] * f, sum[7] * f);
  *reinterpret_cast<uint4*>((which == 0 ? p.d1 : p.d0) + (long long)u.b * str[0] + (long long)(u.key0 + key) * str[1] +
                            (long long)u.hk * str[2] + 8 * c8) = out;
}

// ------------------------------------------------------------------ dQ
constexpr int kKRing = 3, kVRing = 2;

struct __align__(1024) SmemQ {
  uint8_t q[kTileBytes];   // Q, then O
  uint8_t dout[kTileBytes];
  uint8_t k[kKRing][kTileBytes];
  uint8_t v[kVRing][kTileBytes];
  WorkRing work;
  uint64_t q_full, q_empty, o_full, o_empty, d_full, d_empty;
  uint64_t q_ready;      // Q in TMEM (every softmax warp's part)
  uint64_t k_full[kKRing], k_empty[kKRing], k_clear[kKRing];
  uint64_t v_full[kVRing], v_empty[kVRing];
  uint64_t s_full, s_free;     // S in TMEM; read by every softmax warp
  uint64_t dp_full;
  uint64_t ds_full, ds_free;   // dS stored in TMEM by every softmax warp; read by dQ's product
  float delta[kGroups][kTile];   // each warpgroup's part of the rows' sums
  int hot[kTile];                // each row's key with more than half of its probability
  uint64_t delta_full, rest_full;
  uint64_t acc_done;
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t abort_flag;
};

// One item: 128 queries of one query head, with the key tiles that they see.
struct ItemQ {
  int b, h, row0, keys, n;
};
__device__ __forceinline__ ItemQ item_q(const BwdParams& p, const Work& w) {
  ItemQ i;
  int tile, head;
  work_place(p.order, w, tile, head);
  i.b = div_by(head, p.by_H);
  i.h = head - i.b * p.H;
  // the last queries have the most keys when the mask is causal: they start first
  i.row0 = (p.mask.causal ? p.order.tiles - 1 - tile : tile) * kTile;
  i.keys = key_count(p.mask, i.b);
  i.n = (row_limit(p.mask, i.keys, min(i.row0 + kTile, p.mask.Sq) - 1) + kTile - 1) / kTile;
  return i;
}

__global__ void __launch_bounds__(kThreads, 1)
    dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
              const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_d,
              const __grid_constant__ CUtensorMap tm_o, const BwdParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  SmemQ& sm = *reinterpret_cast<SmemQ*>(smem_raw);
  if (smem_misaligned(smem_raw, &g_err_bwd)) return;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);   // (known to be uniform)
  const int lane = threadIdx.x & 31;
  volatile uint32_t* abort_flag = &sm.abort_flag;
  uint32_t* err = &g_err_bwd;

  if (threadIdx.x == 0) {
    work_init(sm.work, kWarpLoad + 2 + (p.mask.kv_len != nullptr ? 1 : 0));   // readers: softmax, MMA, clear
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, kWarpLoad);
    mbar_init(&sm.q_ready, kWarpLoad);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_empty, kWarpLoad);
    mbar_init(&sm.d_full, 1);
    mbar_init(&sm.d_empty, 1 + kWarpLoad);   // the last dP, and every softmax warp's part of delta
    for (int s = 0; s < kKRing; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], tile_releasers(p.mask));
      mbar_init(&sm.k_clear[s], 1);
    }
    for (int s = 0; s < kVRing; ++s) {
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.v_empty[s], 1);
    }
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.s_free, kWarpLoad);
    mbar_init(&sm.dp_full, 1);
    mbar_init(&sm.ds_full, kWarpLoad);
    mbar_init(&sm.ds_free, 1);
    mbar_init(&sm.delta_full, kWarpLoad);
    mbar_init(&sm.rest_full, kWarpLoad);
    mbar_init(&sm.acc_done, 1);
    mbar_init(&sm.drain, 2);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  // (a key of the tensor at all times: an lse that is not the forward's can make a row's sum look as if it had one)
  if (threadIdx.x < kTile) sm.hot[threadIdx.x] = 0;
  if (warp == kWarpMma) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  griddep_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // TMEM columns (all 512 are this CTA's: they start at 0); dS and Q take two values a column
  constexpr uint32_t tS = 0, tDP = 128, tDS = 256, tQ = 320, tDQ = 384;

  if (warp == kWarpLoad) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      tma_prefetch_desc(&tm_d);
      tma_prefetch_desc(&tm_o);
      int it = 0, requests = 0, k_issued = 0, v_issued = 0, q_issued = 0, o_issued = 0, d_issued = 0;
      // One place holds Q(t), from which the softmax warps copy it to TMEM, then O(t), of which they form delta,
      // then Q(t+1): it is loaded while item t runs.  So item t + 1 is looked up before the last two K and V tiles
      // of item t.
      auto load_q = [&](const ItemQ& i) -> bool {
        if (o_issued > 0 && !wait_sleep(&sm.o_empty, (o_issued - 1) & 1, abort_flag, err, kErrTimeoutSync)) return false;
        mbar_arrive_expect_tx(&sm.q_full, kTileBytes);
        load_tile(sm.q, &tm_q, &sm.q_full, i.row0, i.h, i.b);
        ++q_issued;
        return true;
      };
      auto load_o = [&](const ItemQ& i) -> bool {
        if (!wait_sleep(&sm.q_empty, o_issued & 1, abort_flag, err, kErrTimeoutSync)) return false;
        mbar_arrive_expect_tx(&sm.o_full, kTileBytes);
        load_tile(sm.q, &tm_o, &sm.o_full, i.row0, i.h, i.b);
        ++o_issued;
        return true;
      };
      auto load_kv = [&](const ItemQ& i, int j) -> bool {
        const int hk = div_by(i.h, p.by_group);
        {
          const int slot = it % kKRing, use = it / kKRing;
          if (use > 0 && !wait_sleep(&sm.k_empty[slot], (use - 1) & 1, abort_flag, err, kErrTimeoutSync)) return false;
          mbar_arrive_expect_tx(&sm.k_full[slot], kTileBytes);
          if (!withheld(k_issued++))
            load_tile(sm.k[slot], &tm_k, &sm.k_full[slot], (i.n - 1 - j) * kTile, hk, i.b);
        }
        if (j == 0) {
          if (d_issued > 0 && !wait_sleep(&sm.d_empty, (d_issued - 1) & 1, abort_flag, err, kErrTimeoutSync)) return false;
          mbar_arrive_expect_tx(&sm.d_full, kTileBytes);
          load_tile(sm.dout, &tm_d, &sm.d_full, i.row0, i.h, i.b);
          ++d_issued;
        }
        {
          const int slot = it % kVRing, use = it / kVRing;
          if (use > 0 && !wait_sleep(&sm.v_empty[slot], (use - 1) & 1, abort_flag, err, kErrTimeoutSync)) return false;
          mbar_arrive_expect_tx(&sm.v_full[slot], kTileBytes);
          load_tile(sm.v[slot], &tm_v, &sm.v_full[slot], (i.n - 1 - j) * kTile, hk, i.b);
          ++v_issued;
        }
        ++it;
        return j > 0 || load_o(i);
      };
      Work w = first_work();
      ItemQ item = item_q(p, w);
      bool ok = item.n == 0 || load_q(item), more = true;
      while (ok && more) {
        ItemQ next = item;
        const int ask = max(item.n - kAskAhead, 0), look = max(item.n - 2, min(item.n, 2));
        for (int j = 0; ok && j <= item.n; ++j) {
          if (j == ask) {
            ok = work_request(sm.work, w.t + 1, abort_flag, err);
            if (ok) ++requests;
          }
          if (ok && j == look && (more = work_next_load(sm.work, w, abort_flag, err))) {
            next = item_q(p, w);
            ok = next.n == 0 || load_q(next);
          }
          ok = ok && (j == item.n || load_kv(item, j));
        }
        item = next;
      }
      if (*abort_flag) {
        work_teardown(sm.work, requests);
        if (q_issued) mbar_wait_teardown(&sm.q_full, (q_issued - 1) & 1);
        if (o_issued) mbar_wait_teardown(&sm.o_full, (o_issued - 1) & 1);
        if (d_issued) mbar_wait_teardown(&sm.d_full, (d_issued - 1) & 1);
        for (int i = max(k_issued - kKRing, 0); i < k_issued; ++i)
          mbar_wait_teardown(&sm.k_full[i % kKRing], (i / kKRing) & 1);
        for (int i = max(v_issued - kVRing, 0); i < v_issued; ++i)
          mbar_wait_teardown(&sm.v_full[i % kVRing], (i / kVRing) & 1);
      }
    }
  } else if (warp == kWarpMma || warp == kWarpMma + 1) {
    // Two warps issue the products, over the tile products i of all items: one S(i+1) as soon as
    // the softmax warps have S(i) in registers, the other dP(i+1) and dQ(i) when dS(i) is there.  An
    // item's first dQ overwrites the accumulator of the item before: the softmax warps
    // published that dS after they had read it.
    const bool leader = elect_one();
    auto make = [&](const Work& w) { return item_q(p, w); };
    Walk<ItemQ, decltype(make)> walk(make);
    int items = 0;
    int f0 = walk.next(sm.work, lane, abort_flag, err);
    bool ok = true;
    if (warp == kWarpMma) {
      const uint32_t dk = desc_k(sm.k[0]);
      for (int i = 0; f0 != kEnd; ++i) {
        const int slot = i % kKRing;
        ok = (!(f0 & kFirst) || wait_warp(&sm.q_ready, items++ & 1, abort_flag, err, kErrTimeoutSync)) &&
             wait_warp(&sm.k_full[slot], (i / kKRing) & 1, abort_flag, err, kErrTimeoutTma) &&
             (i == 0 || wait_warp(&sm.s_free, (i - 1) & 1, abort_flag, err, kErrTimeoutSync));
        if (!ok) break;
        tc_fence_after();
        mma_tile_nt_ts(tS, tQ, dk + kDescTile * slot, leader);
        if (leader) mma_commit(&sm.s_full);
        f0 = walk.next(sm.work, lane, abort_flag, err);
      }
    } else {
      const uint32_t dd = desc_k(sm.dout), dv = desc_k(sm.v[0]), dk_mn = desc_mn(sm.k[0]);
      uint32_t cleared = 0;   // parity of each slot's clear barrier
      auto issue_dp = [&](int i, int flags) -> bool {
        const int slot = i % kVRing;
        if ((flags & kFirst) && !wait_warp(&sm.d_full, items++ & 1, abort_flag, err, kErrTimeoutTma)) return false;
        if (!wait_warp(&sm.v_full[slot], (i / kVRing) & 1, abort_flag, err, kErrTimeoutTma)) return false;
        tc_fence_after();
        mma_tile_nt(tDP, dd, dv + kDescTile * slot, leader);
        if (leader) mma_commit(&sm.dp_full);
        if (leader) mma_commit(&sm.v_empty[slot]);
        if (leader && (flags & kLast)) mma_commit(&sm.d_empty);
        return true;
      };
      ok = f0 == kEnd || issue_dp(0, f0);
      for (int i = 0; ok && f0 != kEnd; ++i) {
        const int slot = i % kKRing;
        const bool last = f0 & kLast, first = f0 & kFirst;
        if (first && last_rows(p.mask, walk.item.keys, walk.item.n) < kTile) {
          ok = wait_warp(&sm.k_clear[slot], (cleared >> slot) & 1, abort_flag, err, kErrTimeoutSync);
          cleared ^= 1u << slot;
        }
        if (!last) f0 = walk.next(sm.work, lane, abort_flag, err);
        ok = ok && wait_warp(&sm.ds_full, i & 1, abort_flag, err, kErrTimeoutSync) && (last || issue_dp(i + 1, f0));
        if (!ok) break;
        tc_fence_after();
        mma_tile_part_nn<kTile>(tDQ, tDS, dk_mn + kDescTile * slot, 0, !first, leader);
        if (leader) mma_commit(&sm.ds_free);
        if (leader) mma_commit(&sm.k_empty[slot]);   // (dS(i) followed S(i), the other reader of K(i))
        if (last) {
          if (leader) mma_commit(&sm.acc_done);
          f0 = walk.next(sm.work, lane, abort_flag, err);
          ok = f0 == kEnd || issue_dp(i + 1, f0);
        }
      }
    }
    if (leader) mma_commit(&sm.drain);
    mbar_wait_teardown(&sm.drain, 0);
  } else if (warp == kWarpClear) {
    if (p.mask.kv_len != nullptr)
      clear_warp<kKRing, true>(p.mask, [&](const Work& w) { return item_q(p, w); }, sm.work, sm.k, sm.k_full,
                               sm.k_empty, sm.k_clear, lane, abort_flag, err);
  } else if (warp < kWarpLoad) {
    // warpgroup g takes the keys [32 g, 32 g + 32) of each tile, a thread one query
    const int g = warp >> 2, wq = warp & 3;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    bool ok = true;
    int it = 0, turn = 0;
    uint32_t par = 0;   // parities: bit 0 of the items done that have keys, bit 1 of those with several tiles
    const int r = wq * 32 + lane;   // the thread's row of a tile
    // the warpgroup's 32 channels of the row in a tile (row r's 16-byte piece c of a half is at c ^ (r & 7))
    auto tile_row = [&](const uint8_t* tile, uint32_t (&x)[16]) {
      const uint8_t* src = tile + (g >> 1) * kHalfBytes + r * 128;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint4 v = *reinterpret_cast<const uint4*>(src + ((((g & 1) * 4 + c) ^ (r & 7)) << 4));
        x[4 * c] = v.x;
        x[4 * c + 1] = v.y;
        x[4 * c + 2] = v.z;
        x[4 * c + 3] = v.w;
      }
    };
    // Q from its tile in shared memory to TMEM: as the A operand from shared memory it would be read
    // again for every key tile, at the full rate of shared memory while S runs.
    auto begin_item = [&](uint32_t parity) -> bool {
      if (!mbar_wait_warp<false>(&sm.q_full, parity, abort_flag, err, kErrTimeoutTma)) return false;
      uint32_t x[16];
      tile_row(sm.q, x);
      tmem_st16(tQ + lane_off + 16 * g, x);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.q_empty);
        mbar_arrive(&sm.q_ready);
      }
      return true;
    };
    // -delta of the row from the warpgroups' parts.  (They are next written in the next item, whose S and O
    // no warp sees before all have begun it.)
    auto sum_parts = [&](float part, float& neg_delta) -> bool {
      sm.delta[g][r] = part;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.delta_full);
      if (!mbar_wait_warp<false>(&sm.delta_full, (par >> 1) & 1, abort_flag, err, kErrTimeoutSync)) return false;
      par ^= 2u;
      neg_delta = -((sm.delta[0][r] + sm.delta[1][r]) + (sm.delta[2][r] + sm.delta[3][r]));
      return true;
    };
    // The sums of the warpgroups' x and y, in columns of S that each has read (the next S is not
    // issued before all softmax warps have begun the next item).
    auto sum_rest = [&](float& x, float& y) -> bool {
      tmem_st2(tS + lane_off + kCols * g, __float_as_uint(x), __float_as_uint(y));
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.rest_full);
      if (!mbar_wait_warp<false>(&sm.rest_full, par & 1, abort_flag, err, kErrTimeoutSync)) return false;
      tc_fence_after();
      uint32_t v[kGroups][2];
#pragma unroll
      for (int i = 0; i < kGroups; ++i) tmem_ld2(tS + lane_off + kCols * i, v[i]);
      tmem_ld_wait();
      x = y = 0.0f;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        asm volatile("" : "+r"(v[i][0]), "+r"(v[i][1]));   // (not read before the wait)
        x += u2f(v[i][0]);
        y += u2f(v[i][1]);
      }
      tc_fence_before();
      return true;
    };
    // the warpgroup's part of delta, from O's tile and dO's
    auto find_part = [&](float& part) -> bool {
      if (!mbar_wait_warp<false>(&sm.d_full, par & 1, abort_flag, err, kErrTimeoutTma) ||
          !mbar_wait_warp<false>(&sm.o_full, par & 1, abort_flag, err, kErrTimeoutTma))
        return false;
      uint32_t x[16], y[16];
      tile_row(sm.dout, x);
      tile_row(sm.q, y);
      part = 0.0f;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        part = fmaf(u2f(y[c] << 16), u2f(x[c] << 16), part);
        part = fmaf(u2f(y[c] & 0xffff0000u), u2f(x[c] & 0xffff0000u), part);
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.d_empty);
        mbar_arrive(&sm.o_empty);
      }
      return true;
    };
    static_assert(kGroups == 4, "four parts of delta");
    {
      const ItemQ item = item_q(p, first_work());
      if (item.n > 0) ok = begin_item(0);
    }
    bool more = ok;
    while (more) {
      int n, valid;   // products left, and the keys that this row sees from the group's first of the tile on
      float nl = -INFINITY, nd = 0.0f;
      {
        const ItemQ item = item_q(p, work_read(sm.work, turn));
        const int row = item.row0 + r;
        n = item.n;
        const bool one_tile = n == 1;
        // a row that sees one key has ds = 0: as a row that sees none
        valid = row_limit(p.mask, item.keys, row);
        if (valid == 1) valid = 0;
        valid -= kCols * g + (n - 1) * kTile;   // (an item's key tiles come last first)
        const long long at = ((long long)item.b * p.H + item.h) * p.Sq_pad + row;
        if (n > 0) {
          const float lse =
              row < p.mask.Sq ? __ldg(p.lse + ((long long)item.b * p.H + item.h) * p.mask.Sq + row) : -INFINITY;
          float part;
          ok = find_part(part) && (one_tile || sum_parts(part, nd));
          if (lse == -INFINITY) nd = 0.0f;
          else nl = -lse * kLog2e;
          if (g == 0) p.neg_lse2[at] = nl;
        }
      }
      if (!ok) break;
      // A row of dS has the sum 0.  The rounding of its elements, of O in delta and of the P that O was formed with
      // leave it some other sum, by which a mean of the keys that is not 0 comes into dQ.  So the
      // item's last tile, the first 128 keys, all of which a row sees that sees any other tile, takes the delta that
      // makes the sum 0 with what has been rounded so far: delta + rest / sum p.  dQ's error, of its norm, at 1200
      // keys with a mean of 0, 0.5, 1 and 4 times their spread: 0.0024, 0.0028, 0.0037 and 0.0123 without this
      // and 0.0024, 0.0024, 0.0025 and 0.0033 with it (0.0017 is the rounding of dQ); with one tile, where delta itself
      // is formed so, and 2 keys 0.0045 and 0.0024.  It takes 2 to 4 % of the backward's time.
      // A key with more than half of a row's probability has most of that rest, and its dP - delta may be no larger than
      // O's rounding: where it is in another tile it takes 1 / (1 + sum p) of the rest, by itself at the item's end, as
      // a multiple of its K off dQ.  There is at most one such key in a row.  Where all the rest went to the first tile,
      // dQ was off by 0.17 and 0.07 of its norm with 260 and 1000 queries equal to keys, and by all of it where every
      // row has nearly all its probability on one key beyond the tile; so by 0.0020 to 0.0028 (at most 1 % of
      // the backward's time: 16896 queries on 512 keys 317 -> 320 us).
      float rest = 0.0f, better = 0.0f;   // better: with all of the row's p, whose sum is 1, -delta as sum p dp
      int hot = -1;   // that key: its warpgroup's, and from the last product on the row's
      // (a copy of each without the other's code: with it the loop took 1.5 % longer)
      auto product = [&](auto last_c) -> bool {
        constexpr bool kLast = decltype(last_c)::value;
        const bool partial = __any_sync(0xffffffffu, valid < kCols);
        float pr[kCols];
        ok = mbar_wait_warp<false>(&sm.s_full, it & 1, abort_flag, err, kErrTimeoutMma);
        if (!ok) return false;
        tc_fence_after();
        {
          uint32_t a[kCols];
          float top = 0.0f;
          if (kLast) tmem_ld32(tS + lane_off + kCols * g, a);
          else tmem_ld32_max(tS + lane_off + kCols * g, a, top);
          tmem_ld_wait();
          tmem_reg_fence(a);
          if (!kLast) asm volatile("" : "+f"(top));   // (not read before the wait)
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.s_free);
#pragma unroll
          for (int e = 0; e < kCols / 2; ++e) {
            float x0, x1;
            ffma2(x0, x1, u2f(a[2 * e]), u2f(a[2 * e + 1]), p.c_log2, p.c_log2, nl, nl);
            pr[2 * e] = ex2_approx(x0);
            pr[2 * e + 1] = ex2_approx(x1);
          }
          if (!kLast && fmaf(top, p.c_log2, nl) > -1.0f) {   // (top may be that of a key that the row does not see)
            int at = -1;
#pragma unroll
            for (int c = 0; c < kCols; ++c)
              if (c < valid && pr[c] > kHot) at = c;
            if (at >= 0) hot = (n - 1) * kTile + kCols * g + at;
          }
        }
        float sum = 0.0f;
        if (kLast) {
          float s0 = 0.0f, s1 = 0.0f;
          if (partial) {
#pragma unroll
            for (int c = 0; c < kCols; ++c) pr[c] = c < valid ? pr[c] : 0.0f;
          }
#pragma unroll
          for (int e = 0; e < kCols / 2; ++e) fadd2(s0, s1, s0, s1, pr[2 * e], pr[2 * e + 1]);
          sum = s0 + s1;
        }
        ok = mbar_wait_warp<false>(&sm.dp_full, it & 1, abort_flag, err, kErrTimeoutMma);
        if (!ok) return false;
        tc_fence_after();
        {
          uint32_t a[kCols], pk[kCols / 2];
          tmem_ld32(tDP + lane_off + kCols * g, a);
          tmem_ld_wait();
          tmem_reg_fence(a);
          if (kLast) {
            if (partial) {   // (dP of a key that is none may be anything)
#pragma unroll
              for (int c = 0; c < kCols; ++c) a[c] = c < valid ? a[c] : 0u;
            }
            float r0 = 0.0f, r1 = 0.0f;
#pragma unroll
            for (int e = 0; e < kCols / 2; ++e) {
              float x0, x1;
              fadd2(x0, x1, u2f(a[2 * e]), u2f(a[2 * e + 1]), nd, nd);
              ffma2(r0, r1, pr[2 * e], pr[2 * e + 1], x0, x1, r0, r1);
            }
            rest += r0 + r1;
            if (hot >= 0) {
              sm.hot[r] = hot;
              sum += 2.0f;   // (a row's sum is at most 1, but for its rounding)
            }
            ok = sum_rest(rest, sum);
            if (!ok) return false;
            if (sum > 1.5f) {
              sum -= 1.0f;
              hot = sm.hot[r];
            }
            better = nd - rest;
            rest = sum > kLeastSum ? rest / sum : 0.0f;
            nd -= rest;
          }
#pragma unroll
          for (int e = 0; e < kCols / 2; ++e) {
            float x0, x1;
            fadd2(x0, x1, u2f(a[2 * e]), u2f(a[2 * e + 1]), nd, nd);
            fmul2(pr[2 * e], pr[2 * e + 1], pr[2 * e], pr[2 * e + 1], x0, x1);
          }
          if (!kLast && partial) {
#pragma unroll
            for (int c = 0; c < kCols; ++c) pr[c] = c < valid ? pr[c] : 0.0f;
          }
#pragma unroll
          for (int e = 0; e < kCols / 2; ++e) pk[e] = pack_bf16x2(pr[2 * e], pr[2 * e + 1]);
          ok = it == 0 || mbar_wait_warp<false>(&sm.ds_free, (it - 1) & 1, abort_flag, err, kErrTimeoutMma);
          if (!ok) return false;
          tc_fence_after();
          tmem_st16(tDS + lane_off + 16 * g, pk);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.ds_full);
          if (!kLast) {
            float r0 = 0.0f, r1 = 0.0f;
#pragma unroll
            for (int e = 0; e < kCols / 2; ++e) fadd2(r0, r1, r0, r1, u2f(pk[e] << 16), u2f(pk[e] & 0xffff0000u));
            rest += r0 + r1;
          }
        }
        return true;
      };
      for (; ok && n > 1; --n, ++it, valid += kTile) ok = product(std::false_type());
      if (ok && n > 0) {
        ok = product(std::true_type());
        ++it;
      }
      if (!ok) break;
      // the next item's Q, so that its first S runs while this one's rows are stored
      const ItemQ item = item_q(p, work_read(sm.work, turn));
      if (g == 0 && item.n > 0)   // (for dkdv_kernel)
        p.neg_delta[((long long)item.b * p.H + item.h) * p.Sq_pad + item.row0 + r] = better;
      more = work_wait(sm.work, turn + 1, abort_flag, err);
      if (more) {
        const ItemQ next = item_q(p, work_read(sm.work, turn + 1));
        if (next.n > 0) ok = begin_item((par ^ (item.n > 0 ? 1u : 0u)) & 1);
        if (!ok) break;
      }
      // each warpgroup stores 32 of the rows' channels
      uint32_t out[16] = {};
      if (item.n > 0) {
        ok = mbar_wait_warp<false>(&sm.acc_done, par & 1, abort_flag, err, kErrTimeoutMma);
        if (!ok) break;
        par ^= 1u;
        tc_fence_after();
        if (!__any_sync(0xffffffffu, hot >= 0)) {
          load_row_bf16<32>(tDQ + lane_off + 32 * g, out, p.scale);
        } else {
          const uint4* k = nullptr;
          if (hot >= 0)
            k = reinterpret_cast<const uint4*>(p.k + (long long)item.b * p.k_str[0] + (long long)hot * p.k_str[1] +
                                               (long long)div_by(item.h, p.by_group) * p.k_str[2] + 32 * g);
#pragma unroll
          for (int c = 0; c < 4; ++c) {   // (8 channels at a time, for the registers)
            uint32_t a[8];
            tmem_ld8(tDQ + lane_off + 32 * g + 8 * c, a);
            const uint4 v = k != nullptr ? __ldg(k + c) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              asm volatile("" : "+r"(a[2 * e]), "+r"(a[2 * e + 1]));   // (not read before the wait)
              out[4 * c + e] = pack_bf16x2(fmaf(-rest, u2f(w[e] << 16), u2f(a[2 * e])) * p.scale,
                                           fmaf(-rest, u2f(w[e] & 0xffff0000u), u2f(a[2 * e + 1])) * p.scale);
            }
          }
        }
        tc_fence_before();
      }
      const int first = item.row0 + wq * 32;
      store_rows<32>(p.d0 + (long long)item.b * p.s0[0] + (long long)first * p.s0[1] + (long long)item.h * p.s0[2] +
                         32 * g,
                     p.s0[1], out, p.mask.Sq - first, lane);
      work_release(sm.work, turn, lane);
      ++turn;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) {
    __syncwarp();
    tmem_dealloc(sm.tmem_base, 512);
  }
}

constexpr int kSmemKV = (int)sizeof(SmemKV);
constexpr int kSmemQ = (int)sizeof(SmemQ);
static_assert(kSmemKV <= 232448 && kSmemQ <= 232448, "227 KB of shared memory per CTA");

// Parts of each unit of dK and dV: with fewer units than a few per SM, whole units leave SMs idle at the end.
// Times are in products of a tile pair (1.3 us): an item costs two besides its products (first loads and
// results), the parts' sums 0.027 each to write and read, the kernel that joins them two.  The
// products' own time is at least an SM's share of them all, and, as the longest items start
// first, k + 1 times the length of item 152 k: one SM has that many as long.  Backward with 1 part and
// with the parts chosen: 96 units of 132 products 352 and 312 us (3 parts); 16 of 64: 104 and 40 (9); 8 of 128:
// 185 and 44 (19); causal, 64 of up to 128: 212 and 109 (4); 256 of up to 128: 342, and 4 % more with 2, so 1.
constexpr int kSms = 152, kMostRounds = 8;
int kv_parts(const TrainArgs& a) {
  const int tiles = (a.Sk + kTile - 1) / kTile, n_q = (a.Sq + kTile - 1) / kTile, group = a.Hq / a.Hkv;
  const int off = a.Sk - a.Sq;
  const long long heads = (long long)a.B * a.Hkv, units = tiles * heads;
  if (units > kMostRounds * kSms / 2) return 1;
  // products of a unit of tile t: that many of the tiles of a head's queries see it
  auto length = [&](long long t) {
    const long long first = a.causal ? std::max(t * kTile - off, 0ll) / kTile : 0;
    return (double)group * (double)std::max(n_q - first, 0ll);
  };
  double total = 0;
  for (int t = 0; t < tiles; ++t) total += length(t) * (double)heads;
  int best = 1;
  double least = 0;
  for (int rounds = 0; rounds <= kMostRounds; ++rounds) {
    const long long parts = rounds == 0 ? 1 : std::min(rounds * kSms / units, (long long)length(0));
    if (rounds > 0 && parts <= best) continue;
    const long long items = units * parts;
    double products = total / kSms;
    int k = 0;
    for (; (long long)k * kSms < items; ++k)
      products = std::max(products, (k + 1) * std::ceil(length(k * kSms / (heads * parts)) / (double)parts));
    const double time = products + 2 * k + (parts > 1 ? 2 + 0.027 * (double)items : 0);
    if (rounds == 0 || time < least) {
      least = time;
      best = (int)parts;
    }
  }
  return best;
}

}  // namespace

static long long attn_bwd_padded_rows(long long Sq) { return (Sq + kTile - 1) / kTile * kTile; }

size_t attn_bwd_workspace(TrainArgs a) {
  const size_t rows = (size_t)2 * a.B * a.Hq * (size_t)attn_bwd_padded_rows(a.Sq) * sizeof(float);
  int parts = 1;
  for (a.causal = 0; a.causal < 2; ++a.causal) parts = std::max(parts, kv_parts(a));
  const size_t units = (size_t)((a.Sk + kTile - 1) / kTile) * a.B * a.Hkv;
  return rows + (parts > 1 ? units * parts * 2 * kTile * 128 * sizeof(float) : 0);
}

cudaError_t launch_attn_bwd_bf16(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                 const CUtensorMap& tm_d, const CUtensorMap& tm_o, const TrainArgs& a,
                                 const BwdTensors& t, float* workspace, cudaStream_t stream) {
  static ContextOnce attr_done;
  cudaError_t e = attr_done.run([] {
    cudaError_t r = cudaFuncSetAttribute(dkdv_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemKV);
    if (r != cudaSuccess) return r;
    r = cudaFuncSetAttribute(dkdv_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemKV);
    if (r != cudaSuccess) return r;
    return cudaFuncSetAttribute(dq_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemQ);
  });
  if (e != cudaSuccess) return e;
  const int Sq_pad = (int)attn_bwd_padded_rows(a.Sq);
  BwdParams p;
  p.mask = {a.kv_len, a.causal, a.Sq, a.Sk};
  p.c_log2 = a.c_log2;
  p.scale = a.scale;
  p.neg_lse2 = workspace;
  p.neg_delta = workspace + (long long)a.B * a.Hq * Sq_pad;
  p.Sq_pad = Sq_pad;
  p.group = a.Hq / a.Hkv;
  p.lse = t.lse;
  p.k = reinterpret_cast<const __nv_bfloat16*>(t.k);
  const int k_tiles = (a.Sk + kTile - 1) / kTile, q_tiles = Sq_pad / kTile;
  p.H = a.Hq;
  p.by_H = make_div(p.H);
  p.by_group = make_div(p.group);
  p.order = make_order(q_tiles, a.B * a.Hq, a.causal);
  p.d0 = reinterpret_cast<__nv_bfloat16*>(t.dq);
  p.d1 = nullptr;
  p.parts = 1;
  p.by_parts = make_div(1);
  p.partial = nullptr;
  for (int i = 0; i < 3; ++i) {
    p.k_str[i] = t.k_str[i];
    p.s0[i] = t.dq_str[i];
    p.s1[i] = 0;
  }
  g_launched.store(true, std::memory_order_relaxed);
  e = launch_dependent(dq_kernel, dim3((unsigned)p.order.items), kThreads, kSmemQ, stream, tm_q, tm_k, tm_v, tm_d,
                       tm_o, p);
  if (e != cudaSuccess) return e;
  p.H = a.Hkv;
  p.by_H = make_div(p.H);
  p.order = make_order(k_tiles, a.B * a.Hkv, a.causal);
  p.parts = kv_parts(a);
  p.by_parts = make_div(p.parts);
  p.partial = reinterpret_cast<float4*>(p.neg_delta + (long long)a.B * a.Hq * Sq_pad);
  p.d0 = reinterpret_cast<__nv_bfloat16*>(t.dk);
  p.d1 = reinterpret_cast<__nv_bfloat16*>(t.dv);
  for (int i = 0; i < 3; ++i) {
    p.s0[i] = t.dk_str[i];
    p.s1[i] = t.dv_str[i];
  }
  if (p.parts == 1)
    return launch_dependent(dkdv_kernel<false>, dim3((unsigned)p.order.items), kThreads, kSmemKV, stream, tm_q, tm_k,
                            tm_v, tm_d, p);
  e = launch_dependent(dkdv_kernel<true>, dim3((unsigned)(p.order.items * p.parts)), kThreads, kSmemKV, stream, tm_q,
                       tm_k, tm_v, tm_d, p);
  if (e != cudaSuccess) return e;
  return launch_dependent(join_kernel, dim3((unsigned)(p.order.items * kJoinBlocks)), kJoinThreads, 0, stream, p);
}

static const bool err_reader_added =
    add_err_reader([](uint32_t* out) { return read_and_clear_err(g_err_bwd, g_launched, out); });

}  // namespace sa
