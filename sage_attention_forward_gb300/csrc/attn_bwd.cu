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
// Three kernels, no atomics: every sum has one order.
//   rows_kernel   -lse * log2 e and -delta of each row, padded to whole tiles (-inf and 0 there,
//                 and for empty rows: their probabilities come out as 0).  Reads dO and O once.
//   dkdv_kernel   one CTA per (128 keys, key head): K and V stay in shared memory, Q and dO tiles
//                 stream by.  The transposed scores S^T = K Q^T and dP^T = V dO^T leave P^T and
//                 dS^T in TMEM as the A operands of dV += P^T dO and dK += dS^T Q.
//   dq_kernel     one CTA per (128 queries, query head): Q and dO stay, K and V stream by:
//                 S = Q K^T, dP = dO V^T, dQ += dS K.
// Seven products of a tile pair against five if one kernel did both, but a dQ that several CTAs
// add into needs either atomics, whose order changes the result, or 64 KB of FP32 traffic a
// tile pair: at 2560 cycles a pair and 152 SMs that is 7 TB/s of reductions in L2.
//
// P is rounded to BF16 for dV, dS to BF16 for dK and dQ (relative 2^-8 at most each; the unrounded
// P forms dS); every sum is FP32.
#include <cuda_runtime.h>

#include <type_traits>

#include "attn_tiles.cuh"
#include "kernels.h"

namespace sa {
namespace {

using namespace tiles;

constexpr int kThreads = 320;
constexpr int kWarpLoad = 8;
constexpr int kWarpMma = 9;
constexpr float kLog2e = 1.4426950408889634f;

__device__ uint32_t g_err_bwd;

__device__ __forceinline__ float u2f(uint32_t u) { return __uint_as_float(u); }

// ------------------------------------------------------------------ row statistics
struct RowsParams {
  const __nv_bfloat16* o;
  const __nv_bfloat16* dout;
  long long o_s[3], d_s[3];   // element strides (b, s, h)
  const float* lse;           // [B, Hq, Sq]
  float* neg_lse2;            // [B * Hq, Sq_pad]
  float* neg_delta;
  int Sq, Sq_pad, Hq;
  long long rows;             // B * Hq * Sq_pad
};

// Half a warp per row, 16 bytes of O and dO per thread.  Consecutive rows of a warp are
// consecutive heads of one token, which are neighbours in memory in the usual layout.
__global__ void __launch_bounds__(256) rows_kernel(const RowsParams p) {
  griddep_wait();
  const int sub = threadIdx.x & 15;
  const long long step = (long long)gridDim.x * 16;
  for (long long it = (long long)blockIdx.x * 16 + (threadIdx.x >> 4); it < p.rows; it += step) {
    const int h = (int)(it % p.Hq);
    const long long bs = it / p.Hq;
    const int s = (int)(bs % p.Sq_pad), b = (int)(bs / p.Sq_pad);
    const long long out = ((long long)b * p.Hq + h) * p.Sq_pad + s;
    float nl = -INFINITY, nd = 0.0f;
    if (s < p.Sq) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(p.o + b * p.o_s[0] + s * p.o_s[1] + h * p.o_s[2]) + sub);
      const uint4 y = __ldg(reinterpret_cast<const uint4*>(p.dout + b * p.d_s[0] + s * p.d_s[1] + h * p.d_s[2]) + sub);
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
      float a = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a = fmaf(u2f(xs[e] << 16), u2f(ys[e] << 16), a);
        a = fmaf(u2f(xs[e] & 0xffff0000u), u2f(ys[e] & 0xffff0000u), a);
      }
      const uint32_t half = 0xffffu << (threadIdx.x & 16);   // a row's 16 threads are in step with one another
#pragma unroll
      for (int d = 8; d >= 1; d >>= 1) a += __shfl_xor_sync(half, a, d);
      const float lse = __ldg(p.lse + ((long long)b * p.Hq + h) * p.Sq + s);
      if (lse != -INFINITY) {
        nl = -lse * kLog2e;
        nd = -a;
      }
    }
    if (sub == 0) {
      p.neg_lse2[out] = nl;
      p.neg_delta[out] = nd;
    }
  }
}

// ------------------------------------------------------------------ dK, dV
struct BwdParams {
  Mask mask;
  float c_log2;           // softmax_scale * log2 e
  float scale;            // softmax_scale
  const float* neg_lse2;  // [B * Hq, Sq_pad]
  const float* neg_delta;
  int Sq_pad;
  __nv_bfloat16 *d0, *d1;   // dQ; or dK and dV
  long long s0[3], s1[3];   // their element strides (b, s, h)
  int H, group, BH;         // heads of this grid (Hkv, or Hq), Hq / Hkv, B * H
};

struct __align__(1024) SmemKV {
  uint8_t k[kTileBytes];
  uint8_t v[kTileBytes];
  uint8_t q[2][kTileBytes];
  uint8_t dout[2][kTileBytes];
  alignas(16) float neg_lse2[2][kTile];
  alignas(16) float neg_delta[2][kTile];
  uint64_t kv_full;
  uint64_t q_full[2], q_empty[2];   // Q with the row statistics
  uint64_t d_full[2], d_empty[2];   // dO
  uint64_t s_full, dp_full;
  uint64_t p_full[2], ds_full[2];   // queries [0, 64) and [64, 128) of P^T, dS^T stored in TMEM
  uint64_t done;
  uint32_t tmem_base;
  uint32_t abort_flag;
};

__global__ void __launch_bounds__(kThreads, 1)
    dkdv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_d,
                const BwdParams p) {
  extern __shared__ uint8_t smem_raw[];
  SmemKV& sm = *reinterpret_cast<SmemKV*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int bh = (int)(blockIdx.y + gridDim.y * blockIdx.z);
  if (bh >= p.BH) return;   // the last grid.z slice may run past B * Hkv
  const int key0 = blockIdx.x * kTile;
  volatile uint32_t* abort_flag = &sm.abort_flag;
  uint32_t* err = &g_err_bwd;

  if (threadIdx.x == 0) {
    mbar_init(&sm.kv_full, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.q_full[s], 1);
      mbar_init(&sm.q_empty[s], 1);
      mbar_init(&sm.d_full[s], 1);
      mbar_init(&sm.d_empty[s], 1);
      mbar_init(&sm.p_full[s], 4);
      mbar_init(&sm.ds_full[s], 4);
    }
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.dp_full, 1);
    mbar_init(&sm.done, 1);
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
  const uint32_t tmem = sm.tmem_base;
  const int b = bh / p.H, hk = bh % p.H;
  const int keys = key_count(p.mask, b);
  const int off = p.mask.Sk - p.mask.Sq;
  const int n_q = (p.mask.Sq + kTile - 1) / kTile;
  // causal: query i sees key j when j <= i + off, so the tile's first key starts the queries
  const int first = p.mask.causal ? max(key0 - off, 0) / kTile : 0;
  const int per_head = key0 < keys ? max(n_q - first, 0) : 0;
  const int n = per_head * p.group;

  if (warp == kWarpLoad) {
    if (lane == 0 && n > 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_d);
      mbar_arrive_expect_tx(&sm.kv_full, 2 * kTileBytes);
      load_tile(sm.k, &tm_k, &sm.kv_full, key0, hk, b);
      load_tile(sm.v, &tm_v, &sm.kv_full, key0, hk, b);
      int q_issued = 0, d_issued = 0, t = first, h = hk * p.group;
      for (int j = 0; j < n; ++j) {
        const int slot = j & 1, use = j >> 1;
        if (use > 0 && !mbar_wait<true>(&sm.q_empty[slot], (use - 1) & 1, abort_flag, err, kErrTimeoutSync)) break;
        const long long at = ((long long)b * p.H * p.group + h) * p.Sq_pad + t * kTile;
        mbar_arrive_expect_tx(&sm.q_full[slot], kTileBytes + 2 * kTile * 4);
        load_tile(sm.q[slot], &tm_q, &sm.q_full[slot], t * kTile, h, b);
        bulk_load(sm.neg_lse2[slot], p.neg_lse2 + at, kTile * 4, &sm.q_full[slot]);
        bulk_load(sm.neg_delta[slot], p.neg_delta + at, kTile * 4, &sm.q_full[slot]);
        q_issued = j + 1;
        if (use > 0 && !mbar_wait<true>(&sm.d_empty[slot], (use - 1) & 1, abort_flag, err, kErrTimeoutSync)) break;
        mbar_arrive_expect_tx(&sm.d_full[slot], kTileBytes);
        load_tile(sm.dout[slot], &tm_d, &sm.d_full[slot], t * kTile, h, b);
        d_issued = j + 1;
        if (++t == n_q) {
          t = first;
          ++h;
        }
      }
      if (*abort_flag) {
        mbar_wait_teardown(&sm.kv_full, 0);
        for (int it = max(q_issued - 2, 0); it < q_issued; ++it) mbar_wait_teardown(&sm.q_full[it & 1], (it >> 1) & 1);
        for (int it = max(d_issued - 2, 0); it < d_issued; ++it) mbar_wait_teardown(&sm.d_full[it & 1], (it >> 1) & 1);
      }
    }
  } else if (warp == kWarpMma) {
    if (n > 0) {
      // the tensor core's order: dV(j) S(j+1) dK(j) dP(j+1).  S(j+1) overwrites P(j) and dP(j+1)
      // dS(j) after the products that read them, and while the softmax warps work on one of
      // the two chains S -> P -> dV and dP -> dS -> dK the tensor core works on the other.
      const bool leader = elect_one();
      const uint32_t tS = tmem, tDP = tmem + 128, tDV = tmem + 256, tDK = tmem + 384;
      auto issue_s = [&](int j) -> bool {
        if (!mbar_wait_warp<false>(&sm.q_full[j & 1], (j >> 1) & 1, abort_flag, err, kErrTimeoutTma)) return false;
        tc_fence_after();
        mma_tile_nt(tS, sm.k, sm.q[j & 1], leader);
        if (leader) mma_commit(&sm.s_full);
        return true;
      };
      auto issue_dp = [&](int j) -> bool {
        if (!mbar_wait_warp<false>(&sm.d_full[j & 1], (j >> 1) & 1, abort_flag, err, kErrTimeoutTma)) return false;
        tc_fence_after();
        mma_tile_nt(tDP, sm.v, sm.dout[j & 1], leader);
        if (leader) mma_commit(&sm.dp_full);
        return true;
      };
      // acc += A B, A the two halves at columns a and a + 64, as their barriers complete
      auto issue_acc = [&](uint32_t acc, uint32_t a, uint64_t* bars, const uint8_t* tile, int j) -> bool {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!mbar_wait_warp<false>(&bars[half], j & 1, abort_flag, err, kErrTimeoutSync)) return false;
          tc_fence_after();
          mma_tile_half_nn(acc, a + 64 * half, tile, half, j > 0 || half > 0, leader);
        }
        return true;
      };
      bool ok = mbar_wait_warp<false>(&sm.kv_full, 0, abort_flag, err, kErrTimeoutTma) && issue_s(0) && issue_dp(0);
      for (int j = 0; j < n && ok; ++j) {
        const int slot = j & 1;
        ok = issue_acc(tDV, tS, sm.p_full, sm.dout[slot], j);
        if (!ok) break;
        if (leader) mma_commit(&sm.d_empty[slot]);   // (dP(j) was issued before)
        if (j + 1 < n && !issue_s(j + 1)) break;
        ok = issue_acc(tDK, tDP, sm.ds_full, sm.q[slot], j);
        if (!ok) break;
        if (leader) mma_commit(&sm.q_empty[slot]);
        if (j + 1 < n && !issue_dp(j + 1)) break;
      }
      if (leader) mma_commit(&sm.done);
      mbar_wait_teardown(&sm.done, 0);
    }
  } else {
    // warpgroup `half` takes the queries [64 * half, 64 * half + 64) of each tile, a thread one key
    const int half = warp >> 2, wq = warp & 3;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + 64 * half, tDP = tS + 128;
    const int key = key0 + wq * 32 + lane;
    bool ok = true;
    int t = first;
    for (int j = 0; j < n; ++j) {
      const int slot = j & 1;
      // a tile on the diagonal: column c (query 128 t + 64 half + c) sees this key from c_min on.
      // Key 0's first query sees key 0 alone; its ds is 0.
      const int c_min = p.mask.causal ? key - off - (t * kTile + 64 * half) : 0;
      const bool diag = p.mask.causal && key0 + kTile - 1 - off > t * kTile;   // uniform over the CTA
      const int c_min_ds = key == 0 ? c_min + 1 : c_min;
      float pr[64];
      if (!mbar_wait_warp<false>(&sm.s_full, j & 1, abort_flag, err, kErrTimeoutMma)) { ok = false; break; }
      tc_fence_after();
      // (the MMA warp waited for this tile's Q and statistics, but their bytes are visible to a
      // thread only through its own wait)
      if (!mbar_wait_warp<false>(&sm.q_full[slot], (j >> 1) & 1, abort_flag, err, kErrTimeoutTma)) { ok = false; break; }
      {
        uint32_t a[2][32];
        tmem_ld64(tS, a[0], a[1]);
        uint32_t pk[32];
        const float4* nl = reinterpret_cast<const float4*>(&sm.neg_lse2[slot][64 * half]);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float4 m = nl[e];
          const uint32_t* s = &a[e >> 3][4 * (e & 7)];
          float x0, x1, x2, x3;
          ffma2(x0, x1, u2f(s[0]), u2f(s[1]), p.c_log2, p.c_log2, m.x, m.y);
          ffma2(x2, x3, u2f(s[2]), u2f(s[3]), p.c_log2, p.c_log2, m.z, m.w);
          pr[4 * e] = ex2_approx(x0);
          pr[4 * e + 1] = ex2_approx(x1);
          pr[4 * e + 2] = ex2_approx(x2);
          pr[4 * e + 3] = ex2_approx(x3);
        }
        if (diag) {
#pragma unroll
          for (int c = 0; c < 64; ++c) pr[c] = c >= c_min ? pr[c] : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) pk[e] = pack_bf16x2(pr[2 * e], pr[2 * e + 1]);
        tmem_st32(tS, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[half]);
      }
      if (!mbar_wait_warp<false>(&sm.dp_full, j & 1, abort_flag, err, kErrTimeoutMma)) { ok = false; break; }
      tc_fence_after();
      {
        uint32_t a[2][32];
        tmem_ld64(tDP, a[0], a[1]);
        uint32_t pk[32];
        const float4* nd = reinterpret_cast<const float4*>(&sm.neg_delta[slot][64 * half]);
        float ds[64];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float4 d = nd[e];
          const uint32_t* s = &a[e >> 3][4 * (e & 7)];
          float x0, x1, x2, x3;
          fadd2(x0, x1, u2f(s[0]), u2f(s[1]), d.x, d.y);
          fadd2(x2, x3, u2f(s[2]), u2f(s[3]), d.z, d.w);
          fmul2(ds[4 * e], ds[4 * e + 1], pr[4 * e], pr[4 * e + 1], x0, x1);
          fmul2(ds[4 * e + 2], ds[4 * e + 3], pr[4 * e + 2], pr[4 * e + 3], x2, x3);
        }
        if (diag) {
#pragma unroll
          for (int c = 0; c < 64; ++c) ds[c] = c >= c_min_ds ? ds[c] : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) pk[e] = pack_bf16x2(ds[2 * e], ds[2 * e + 1]);
        tmem_st32(tDP, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.ds_full[half]);
      }
      if (++t == n_q) t = first;
    }
    // warpgroup 0 stores dV, warpgroup 1 dK; keys that no query sees get zeros (their rows hold
    // what the padding made of them), and a key alone in its batch entry has dK = 0
    __nv_bfloat16* dst = half == 0 ? p.d1 + (long long)b * p.s1[0] + (long long)key * p.s1[1] + (long long)hk * p.s1[2]
                                   : p.d0 + (long long)b * p.s0[0] + (long long)key * p.s0[1] + (long long)hk * p.s0[2];
    const bool store = key < p.mask.Sk;
    const bool zero = n == 0 || key >= keys || (half == 1 && keys == 1);
    if (n > 0) {
      ok = ok && mbar_wait_warp<true>(&sm.done, 0, abort_flag, err, kErrTimeoutMma);
      if (ok) {
        tc_fence_after();
        store_row_bf16(tmem + lane_off + 256 + 128 * half, dst, half == 0 ? 1.0f : p.scale, store && !zero);
      }
    }
    if (ok && store && zero) store_row_zero(dst);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ dQ
constexpr int kKRing = 3, kVRing = 2;

struct __align__(1024) SmemQ {
  uint8_t q[kTileBytes];
  uint8_t dout[kTileBytes];
  uint8_t k[kKRing][kTileBytes];
  uint8_t v[kVRing][kTileBytes];
  uint64_t q_full, d_full;
  uint64_t k_full[kKRing], k_empty[kKRing];
  uint64_t v_full[kVRing], v_empty[kVRing];
  uint64_t s_full[2], dp_full;
  uint64_t ds_full[2];   // keys [0, 64) and [64, 128) of dS stored in TMEM
  uint64_t done;
  uint32_t tmem_base;
  uint32_t abort_flag;
};

__global__ void __launch_bounds__(kThreads, 1)
    dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
              const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_d, const BwdParams p) {
  extern __shared__ uint8_t smem_raw[];
  SmemQ& sm = *reinterpret_cast<SmemQ*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int bh = (int)(blockIdx.y + gridDim.y * blockIdx.z);
  if (bh >= p.BH) return;   // the last grid.z slice may run past B * Hq
  const int qb = p.mask.causal ? (int)(gridDim.x - 1 - blockIdx.x) : (int)blockIdx.x;
  const int row0 = qb * kTile;
  volatile uint32_t* abort_flag = &sm.abort_flag;
  uint32_t* err = &g_err_bwd;

  if (threadIdx.x == 0) {
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.d_full, 1);
    for (int s = 0; s < kKRing; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 1);
    }
    for (int s = 0; s < kVRing; ++s) {
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.s_full[s], 1);
      mbar_init(&sm.ds_full[s], 4);
    }
    mbar_init(&sm.dp_full, 1);
    mbar_init(&sm.done, 1);
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
  const uint32_t tmem = sm.tmem_base;
  const int b = bh / p.H, h = bh % p.H, hk = h / p.group;
  const int keys = key_count(p.mask, b);
  const int last_row = min(row0 + kTile, p.mask.Sq) - 1;
  const int n = (row_limit(p.mask, keys, last_row) + kTile - 1) / kTile;

  if (warp == kWarpLoad) {
    if (lane == 0 && n > 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      mbar_arrive_expect_tx(&sm.q_full, kTileBytes);
      load_tile(sm.q, &tm_q, &sm.q_full, row0, h, b);
      mbar_arrive_expect_tx(&sm.d_full, kTileBytes);
      load_tile(sm.dout, &tm_d, &sm.d_full, row0, h, b);
      int k_issued = 0, v_issued = 0;
      for (int j = 0; j < n; ++j) {
        {
          const int slot = j % kKRing, use = j / kKRing;
          if (use > 0 && !mbar_wait<true>(&sm.k_empty[slot], (use - 1) & 1, abort_flag, err, kErrTimeoutSync)) break;
          mbar_arrive_expect_tx(&sm.k_full[slot], kTileBytes);
          load_tile(sm.k[slot], &tm_k, &sm.k_full[slot], j * kTile, hk, b);
          k_issued = j + 1;
        }
        {
          const int slot = j % kVRing, use = j / kVRing;
          if (use > 0 && !mbar_wait<true>(&sm.v_empty[slot], (use - 1) & 1, abort_flag, err, kErrTimeoutSync)) break;
          mbar_arrive_expect_tx(&sm.v_full[slot], kTileBytes);
          load_tile(sm.v[slot], &tm_v, &sm.v_full[slot], j * kTile, hk, b);
          v_issued = j + 1;
        }
      }
      if (*abort_flag) {
        mbar_wait_teardown(&sm.q_full, 0);
        mbar_wait_teardown(&sm.d_full, 0);
        for (int it = max(k_issued - kKRing, 0); it < k_issued; ++it)
          mbar_wait_teardown(&sm.k_full[it % kKRing], (it / kKRing) & 1);
        for (int it = max(v_issued - kVRing, 0); it < v_issued; ++it)
          mbar_wait_teardown(&sm.v_full[it % kVRing], (it / kVRing) & 1);
      }
    }
  } else if (warp == kWarpMma) {
    if (n > 0) {
      // S is formed two tiles ahead in two TMEM buffers; dS(j) takes S(j)'s place.  The tensor core's
      // order is dP(j+1) dQ(j) S(j+2): the softmax warps have S(j+1) in hand meanwhile.
      const bool leader = elect_one();
      const uint32_t tDP = tmem + 256, tDQ = tmem + 384;
      auto issue_s = [&](int j) -> bool {
        const int slot = j % kKRing;
        if (!mbar_wait_warp<false>(&sm.k_full[slot], (j / kKRing) & 1, abort_flag, err, kErrTimeoutTma)) return false;
        if (keys < p.mask.Sk && (j + 1) * kTile > keys) clear_rows(sm.k[slot], keys - j * kTile, lane);
        tc_fence_after();
        mma_tile_nt(tmem + 128 * (j & 1), sm.q, sm.k[slot], leader);
        if (leader) mma_commit(&sm.s_full[j & 1]);
        return true;
      };
      auto issue_dp = [&](int j) -> bool {
        const int slot = j % kVRing;
        if (!mbar_wait_warp<false>(&sm.v_full[slot], (j / kVRing) & 1, abort_flag, err, kErrTimeoutTma)) return false;
        tc_fence_after();
        mma_tile_nt(tDP, sm.dout, sm.v[slot], leader);
        if (leader) mma_commit(&sm.dp_full);
        if (leader) mma_commit(&sm.v_empty[slot]);
        return true;
      };
      bool ok = mbar_wait_warp<false>(&sm.q_full, 0, abort_flag, err, kErrTimeoutTma) && issue_s(0) &&
                mbar_wait_warp<false>(&sm.d_full, 0, abort_flag, err, kErrTimeoutTma) && issue_dp(0) &&
                (n < 2 || issue_s(1));
      for (int j = 0; j < n && ok; ++j) {
        ok = mbar_wait_warp<false>(&sm.ds_full[0], j & 1, abort_flag, err, kErrTimeoutSync) &&
             mbar_wait_warp<false>(&sm.ds_full[1], j & 1, abort_flag, err, kErrTimeoutSync) &&
             (j + 1 >= n || issue_dp(j + 1));
        if (!ok) break;
        tc_fence_after();
        const int slot = j % kKRing;
#pragma unroll
        for (int half = 0; half < 2; ++half)
          mma_tile_half_nn(tDQ, tmem + 128 * (j & 1) + 64 * half, sm.k[slot], half, j > 0 || half > 0, leader);
        if (leader) mma_commit(&sm.k_empty[slot]);
        ok = j + 2 >= n || issue_s(j + 2);
      }
      if (leader) mma_commit(&sm.done);
      mbar_wait_teardown(&sm.done, 0);
    }
  } else {
    // warpgroup `half` takes the keys [64 * half, 64 * half + 64) of each tile, a thread one query
    const int half = warp >> 2, wq = warp & 3;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + 64 * half, tDP = tS + 256;
    const int row = row0 + wq * 32 + lane;
    // a row that sees one key has ds = 0: as a row that sees none
    int limit = row_limit(p.mask, keys, row);
    if (limit == 1) limit = 0;
    int whole = row_limit(p.mask, keys, row0 + wq * 32);
    if (whole == 1) whole = 0;
    // (rows past Sq have their statistics in the padding)
    const float nl = __ldg(p.neg_lse2 + (long long)bh * p.Sq_pad + row);
    const float nd = __ldg(p.neg_delta + (long long)bh * p.Sq_pad + row);
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const bool partial = whole < (j + 1) * kTile;              // warp-uniform
      const int valid = limit - j * kTile - 64 * half;           // this row sees the half's keys [0, valid)
      const uint32_t tSj = tS + 128 * (j & 1);
      float pr[64];
      if (!mbar_wait_warp<false>(&sm.s_full[j & 1], (j >> 1) & 1, abort_flag, err, kErrTimeoutMma)) { ok = false; break; }
      tc_fence_after();
      {
        uint32_t a[2][32];
        tmem_ld64(tSj, a[0], a[1]);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const uint32_t* s = &a[e >> 4][2 * (e & 15)];
          float x0, x1;
          ffma2(x0, x1, u2f(s[0]), u2f(s[1]), p.c_log2, p.c_log2, nl, nl);
          pr[2 * e] = ex2_approx(x0);
          pr[2 * e + 1] = ex2_approx(x1);
        }
      }
      if (!mbar_wait_warp<false>(&sm.dp_full, j & 1, abort_flag, err, kErrTimeoutMma)) { ok = false; break; }
      tc_fence_after();
      {
        uint32_t a[2][32];
        tmem_ld64(tDP, a[0], a[1]);
        float ds[64];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const uint32_t* s = &a[e >> 4][2 * (e & 15)];
          float x0, x1;
          fadd2(x0, x1, u2f(s[0]), u2f(s[1]), nd, nd);
          fmul2(ds[2 * e], ds[2 * e + 1], pr[2 * e], pr[2 * e + 1], x0, x1);
        }
        if (partial) {
#pragma unroll
          for (int c = 0; c < 64; ++c) ds[c] = c < valid ? ds[c] : 0.0f;
        }
        uint32_t pk[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) pk[e] = pack_bf16x2(ds[2 * e], ds[2 * e + 1]);
        tmem_st32(tSj, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.ds_full[half]);
      }
    }
    // each warpgroup stores 64 of the row's channels
    __nv_bfloat16* dst = p.d0 + (long long)b * p.s0[0] + (long long)row * p.s0[1] + (long long)h * p.s0[2] + 64 * half;
    const bool store = row < p.mask.Sq;
    if (n == 0) {
      if (store) store_row_zero<64>(dst);
    } else if (ok && mbar_wait_warp<true>(&sm.done, 0, abort_flag, err, kErrTimeoutMma)) {
      tc_fence_after();
      store_row_bf16<64>(tmem + lane_off + 384 + 64 * half, dst, p.scale, store);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

constexpr int kSmemKV = (int)sizeof(SmemKV) + 1024;
constexpr int kSmemQ = (int)sizeof(SmemQ) + 1024;
static_assert(kSmemKV <= 232448 && kSmemQ <= 232448, "227 KB of shared memory per CTA");

}  // namespace

long long attn_bwd_padded_rows(long long Sq) { return (Sq + kTile - 1) / kTile * kTile; }

cudaError_t launch_attn_bwd_bf16(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                 const CUtensorMap& tm_d, const TrainArgs& a, const BwdTensors& t, float* workspace,
                                 cudaStream_t stream) {
  static ContextOnce attr_done;
  cudaError_t e = attr_done.run([] {
    cudaError_t r = cudaFuncSetAttribute(dkdv_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemKV);
    if (r != cudaSuccess) return r;
    return cudaFuncSetAttribute(dq_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemQ);
  });
  if (e != cudaSuccess) return e;
  const int Sq_pad = (int)attn_bwd_padded_rows(a.Sq);
  RowsParams r;
  r.o = reinterpret_cast<const __nv_bfloat16*>(t.o);
  r.dout = reinterpret_cast<const __nv_bfloat16*>(t.dout);
  for (int i = 0; i < 3; ++i) {
    r.o_s[i] = t.o_str[i];
    r.d_s[i] = t.dout_str[i];
  }
  r.lse = t.lse;
  r.neg_lse2 = workspace;
  r.rows = (long long)a.B * a.Hq * Sq_pad;
  r.neg_delta = workspace + r.rows;
  r.Sq = a.Sq;
  r.Sq_pad = Sq_pad;
  r.Hq = a.Hq;
  long long blocks = (r.rows + 15) / 16;
  const long long cap = (long long)device_sm_count() * 16;
  if (blocks > cap) blocks = cap;
  e = launch_dependent(rows_kernel, dim3((unsigned)blocks), 256, 0, stream, r);
  if (e != cudaSuccess) return e;

  BwdParams p;
  p.mask = {a.kv_len, a.causal, a.Sq, a.Sk};
  p.c_log2 = a.c_log2;
  p.scale = a.scale;
  p.neg_lse2 = r.neg_lse2;
  p.neg_delta = r.neg_delta;
  p.Sq_pad = Sq_pad;
  p.group = a.Hq / a.Hkv;
  p.H = a.Hkv;
  p.BH = a.B * a.Hkv;
  p.d0 = reinterpret_cast<__nv_bfloat16*>(t.dk);
  p.d1 = reinterpret_cast<__nv_bfloat16*>(t.dv);
  for (int i = 0; i < 3; ++i) {
    p.s0[i] = t.dk_str[i];
    p.s1[i] = t.dv_str[i];
  }
  e = launch_dependent(dkdv_kernel, heads_grid((a.Sk + kTile - 1) / kTile, p.BH), kThreads, kSmemKV, stream, tm_q,
                       tm_k, tm_v, tm_d, p);
  if (e != cudaSuccess) return e;
  p.H = a.Hq;
  p.BH = a.B * a.Hq;
  p.d0 = reinterpret_cast<__nv_bfloat16*>(t.dq);
  p.d1 = nullptr;
  for (int i = 0; i < 3; ++i) p.s0[i] = t.dq_str[i];
  return launch_dependent(dq_kernel, heads_grid((a.Sq + kTile - 1) / kTile, p.BH), kThreads, kSmemQ, stream, tm_q,
                          tm_k, tm_v, tm_d, p);
}

cudaError_t read_and_clear_err_bwd(uint32_t* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_err_bwd, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_err_bwd, &zero, sizeof(uint32_t));
}

}  // namespace sa
