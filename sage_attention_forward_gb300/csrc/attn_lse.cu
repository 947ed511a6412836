// Attention forward for training, sm_103a: O and each row's log-sum-exp, which is what a
// backward pass needs to form the probabilities again.
//
//   s_ij = scale * q_i . k_j            over the keys j < limit(i)  (attn_tiles.cuh)
//   lse_i = log sum_j exp(s_ij)         natural logarithm; -inf for an empty row
//   o_i  = sum_j exp(s_ij - lse_i) v_j  0 for an empty row
//
// Query head h reads the keys and values of head h / (Hq / Hkv).
//
// The pipeline is the BF16 forward's (attn_fwd.cu): one CTA = two 128-row Q tiles of one
// query head, a TMA warp, an MMA warp and two softmax warpgroups of one thread per row, online
// softmax in base 2 against a reference maximum that moves only when it is passed by kTau.
// What differs: the number of key tiles is the CTA's own (causal rows stop at the diagonal; the
// CTAs with the most tiles start first), a tile that a warp's rows do not all see whole takes the
// masked copy of the softmax, and the rows of V past the last key are cleared in shared memory.
#include <cuda_runtime.h>

#include <type_traits>

#include "attn_tiles.cuh"
#include "kernels.h"

namespace sa {
namespace {

using namespace tiles;

constexpr int kNQ = 2;
constexpr int kStages = 2;
constexpr int kThreads = 320;
constexpr int kWarpLoad = 8;
constexpr int kWarpMma = 9;
constexpr float kTau = 64.0f;   // as the BF16 forward: p <= 2^64 stays far inside BF16's and FP32's range
constexpr float kLn2 = 0.6931471805599453f;

struct __align__(1024) Smem {
  uint8_t q[kNQ][kTileBytes];
  uint8_t k[kStages][kTileBytes];
  uint8_t v[kStages][kTileBytes];
  uint64_t q_full;
  uint64_t k_full[kStages], k_empty[kStages];
  uint64_t v_full[kStages], v_empty[kStages];
  uint64_t s_full[kNQ];
  uint64_t p_full[kNQ][2];   // P_i keys [0, 64) and [64, 128) stored in TMEM
  uint64_t o_done[kNQ];
  uint64_t mma_drain;
  uint32_t tmem_base;
  uint32_t abort_flag;
};

__device__ uint32_t g_err_lse;

struct Params {
  Mask mask;
  float c_log2;   // softmax_scale * log2 e
  __nv_bfloat16* o;
  long long o_sb, o_ss, o_sh;
  float* lse;     // [B, Hq, Sq]
  int Hq, group, BH;
};

__device__ __forceinline__ float u2f(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ uint32_t f2u(float f) { return __float_as_uint(f); }

__global__ void __launch_bounds__(kThreads, 1)
    lse_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int bh = (int)(blockIdx.y + gridDim.y * blockIdx.z);
  if (bh >= p.BH) return;   // the last grid.z slice may run past B * Hq
  // the last query block has the most keys when the mask is causal: it starts first
  const int qb = p.mask.causal ? (int)(gridDim.x - 1 - blockIdx.x) : (int)blockIdx.x;
  const int q_row0 = qb * (kNQ * kTile);
  volatile uint32_t* abort_flag = &sm.abort_flag;
  uint32_t* err = &g_err_lse;

  if (threadIdx.x == 0) {
    mbar_init(&sm.q_full, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 1);
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.v_empty[s], 1);
    }
    for (int i = 0; i < kNQ; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i][0], 4);
      mbar_init(&sm.p_full[i][1], 4);
      mbar_init(&sm.o_done[i], 1);
    }
    mbar_init(&sm.mma_drain, 1);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  griddep_wait();   // kv_len and the tensors may come from the kernel before this one
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const int b = bh / p.Hq, h = bh % p.Hq, hk = h / p.group;
  const int keys = key_count(p.mask, b);
  const int last_row = min(q_row0 + kNQ * kTile, p.mask.Sq) - 1;
  const int n = (row_limit(p.mask, keys, last_row) + kTile - 1) / kTile;   // key tiles; 0: no row sees a key

  if (warp == kWarpLoad) {
    if (lane == 0 && n > 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      mbar_arrive_expect_tx(&sm.q_full, kNQ * kTileBytes);
      for (int i = 0; i < kNQ; ++i) load_tile(sm.q[i], &tm_q, &sm.q_full, q_row0 + i * kTile, h, b);
      int k_issued = 0, v_issued = 0;
      for (int j = 0; j < n; ++j) {
        const int slot = j % kStages, use = j / kStages;
        if (use > 0 && !mbar_wait<true>(&sm.k_empty[slot], (use - 1) & 1, abort_flag, err, kErrTimeoutSync)) break;
        mbar_arrive_expect_tx(&sm.k_full[slot], kTileBytes);
        load_tile(sm.k[slot], &tm_k, &sm.k_full[slot], j * kTile, hk, b);
        k_issued = j + 1;
        if (use > 0 && !mbar_wait<true>(&sm.v_empty[slot], (use - 1) & 1, abort_flag, err, kErrTimeoutSync)) break;
        mbar_arrive_expect_tx(&sm.v_full[slot], kTileBytes);
        load_tile(sm.v[slot], &tm_v, &sm.v_full[slot], j * kTile, hk, b);
        v_issued = j + 1;
      }
      if (*abort_flag) {
        mbar_wait_teardown(&sm.q_full, 0);
        for (int it = max(k_issued - kStages, 0); it < k_issued; ++it)
          mbar_wait_teardown(&sm.k_full[it % kStages], (it / kStages) & 1);
        for (int it = max(v_issued - kStages, 0); it < v_issued; ++it)
          mbar_wait_teardown(&sm.v_full[it % kStages], (it / kStages) & 1);
      }
    }
  } else if (warp == kWarpMma) {
    if (n > 0) {
      const bool leader = elect_one();
      auto tS = [&](int i) { return tmem + 128u * (uint32_t)i; };
      auto tO = [&](int i) { return tmem + 256u + 128u * (uint32_t)i; };
      auto issue_pv = [&](int i, int slot, int j) -> bool {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!mbar_wait_warp<false>(&sm.p_full[i][half], j & 1, abort_flag, err, kErrTimeoutSync)) return false;
          tc_fence_after();
          mma_tile_half_nn(tO(i), tS(i) + 32 * half, sm.v[slot], half, j > 0 || half > 0, leader);
        }
        if (leader) mma_commit(&sm.o_done[i]);
        return true;
      };
      auto wait_k = [&](int t, int slot) -> bool {
        return mbar_wait_warp<false>(&sm.k_full[slot], (t / kStages) & 1, abort_flag, err, kErrTimeoutTma);
      };
      bool ok = mbar_wait_warp<false>(&sm.q_full, 0, abort_flag, err, kErrTimeoutTma) && wait_k(0, 0);
      if (ok) {
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < kNQ; ++i) {
          mma_tile_nt(tS(i), sm.q[i], sm.k[0], leader);
          if (leader) mma_commit(&sm.s_full[i]);
        }
        if (leader) mma_commit(&sm.k_empty[0]);
      }
      for (int j0 = 0; j0 < n && ok; j0 += kStages) {
#pragma unroll
        for (int u = 0; u < kStages; ++u) {
          const int j = j0 + u;
          if (j >= n || !ok) break;
          const int slotV = u, slotK = (u + 1) % kStages;
          const bool more = (j + 1 < n);
          ok = mbar_wait_warp<false>(&sm.v_full[slotV], (j / kStages) & 1, abort_flag, err, kErrTimeoutTma);
          if (!ok) break;
          if (keys < p.mask.Sk && (j + 1) * kTile > keys) clear_rows(sm.v[slotV], keys - j * kTile, lane);
#pragma unroll
          for (int i = 0; i < kNQ; ++i) {
            ok = issue_pv(i, slotV, j) && (!more || i > 0 || wait_k(j + 1, slotK));
            if (!ok) break;
            if (leader && i == kNQ - 1) mma_commit(&sm.v_empty[slotV]);
            if (more) {
              tc_fence_after();
              mma_tile_nt(tS(i), sm.q[i], sm.k[slotK], leader);
              if (leader) mma_commit(&sm.s_full[i]);
              if (leader && i == kNQ - 1) mma_commit(&sm.k_empty[slotK]);
            }
          }
        }
      }
      if (leader) mma_commit(&sm.mma_drain);
      mbar_wait_teardown(&sm.mma_drain, 0);
    }
  } else {
    const int i = warp >> 2, wq = warp & 3;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + 128u * i;
    const uint32_t tO = tmem + lane_off + 256u + 128u * i;
    const int grow = q_row0 + i * kTile + wq * 32 + lane;
    const int limit = row_limit(p.mask, keys, grow);
    // keys below this are seen by every row of the warp (limits grow with the row)
    const int whole = row_limit(p.mask, keys, q_row0 + i * kTile + wq * 32);
    const float f = p.c_log2;
    float m_used = -INFINITY, l = 0.0f;
    bool ok = true;

    for (int j = 0; j < n; ++j) {
      if (!mbar_wait_warp<false>(&sm.s_full[i], j & 1, abort_flag, err, kErrTimeoutMma)) { ok = false; break; }
      tc_fence_after();
      uint32_t s[128];
      uint32_t(&s0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&s[0]);
      uint32_t(&s1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&s[32]);
      uint32_t(&s2)[32] = *reinterpret_cast<uint32_t(*)[32]>(&s[64]);
      uint32_t(&s3)[32] = *reinterpret_cast<uint32_t(*)[32]>(&s[96]);
      const bool partial = whole < (j + 1) * kTile;   // warp-uniform
      const int valid = limit - j * kTile;            // this row sees the tile's keys [0, valid)
      float r0, r1, r2, r3;
      tmem_ld32_max(tS + 0, s0, r0);
      tmem_ld32_max(tS + 32, s1, r1);
      tmem_ld_wait();
      tmem_reg_fence(s0);
      tmem_reg_fence(s1);
      tmem_reg_fence2f(r0, r1);
      tmem_ld32_max(tS + 64, s2, r2);
      tmem_ld32_max(tS + 96, s3, r3);
      tmem_ld_wait();
      tmem_reg_fence(s2);
      tmem_reg_fence(s3);
      tmem_reg_fence2f(r2, r3);
      float m_cand;
      if (!partial) {
        m_cand = fmaxf(fmaxf(r0, r1), fmaxf(r2, r3)) * f;   // f >= 0
      } else {
#pragma unroll
        for (int e = 0; e < 128; ++e)
          if (e >= valid) s[e] = f2u(-INFINITY);
        m_cand = fmaxf(fmaxf(max32(&s[0]), max32(&s[32])), fmaxf(max32(&s[64]), max32(&s[96])));
        m_cand = m_cand == -INFINITY ? -INFINITY : m_cand * f;   // (0 * -inf is NaN)
      }
      const bool need = m_cand > m_used + kTau;
      const float sc = need ? ex2_approx(m_used - m_cand) : 1.0f;
      if (need) {
        l *= sc;
        m_used = m_cand;
      }
      float rs0 = 0.0f, rs1 = 0.0f;
      auto p_section = [&](auto masked) {
        constexpr bool kMasked = decltype(masked)::value;
#pragma unroll
        for (int blk = 0; blk < 4; ++blk) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int c0 = 32 * blk + 2 * e;
            float x0, x1;
            ffma2(x0, x1, u2f(s[c0]), u2f(s[c0 + 1]), f, f, -m_used, -m_used);
            float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            if (kMasked) {
              p0 = c0 < valid ? p0 : 0.0f;
              p1 = c0 + 1 < valid ? p1 : 0.0f;
            }
            fadd2(rs0, rs1, rs0, rs1, p0, p1);
            pk[e] = pack_bf16x2(p0, p1);
          }
          tmem_st16(tS + 16 * blk, pk);
          if (blk & 1) {
            if (blk == 1 && j > 0 && __any_sync(0xffffffffu, need)) {
              // O_i must hold P_{j-1} V_{j-1} before it is rescaled, and be rescaled before
              // the first half of P_j V_j accumulates into it
              if (mbar_wait_warp<true>(&sm.o_done[i], (j - 1) & 1, abort_flag, err, kErrTimeoutMma)) {
                tc_fence_after();
                uint32_t oa[16], ob[16];
                tmem_ld16(tO, oa);
                tmem_ld_wait();
                tmem_reg_fence16(oa);
#pragma unroll
                for (int c2 = 0; c2 < 8; c2 += 2) {
                  tmem_ld16(tO + 16 * (c2 + 1), ob);
#pragma unroll
                  for (int e = 0; e < 16; ++e) oa[e] = f2u(u2f(oa[e]) * sc);
                  tmem_st16(tO + 16 * c2, oa);
                  tmem_ld_wait();
                  tmem_reg_fence16(ob);
                  if (c2 + 2 < 8) tmem_ld16(tO + 16 * (c2 + 2), oa);
#pragma unroll
                  for (int e = 0; e < 16; ++e) ob[e] = f2u(u2f(ob[e]) * sc);
                  tmem_st16(tO + 16 * (c2 + 1), ob);
                  if (c2 + 2 < 8) {
                    tmem_ld_wait();
                    tmem_reg_fence16(oa);
                  }
                }
              } else {
                ok = false;
              }
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(&sm.p_full[i][blk >> 1]);
          }
        }
      };
      if (partial) p_section(std::true_type{});
      else p_section(std::false_type{});
      if (!ok) break;
      l += rs0 + rs1;
    }

    const bool store = grow < p.mask.Sq;
    __nv_bfloat16* dst = p.o + (long long)b * p.o_sb + (long long)grow * p.o_ss + (long long)h * p.o_sh;
    float* lse = p.lse + (long long)bh * p.mask.Sq + grow;
    if (n == 0) {
      if (store) {
        store_row_zero(dst);
        *lse = -INFINITY;
      }
    } else if (ok && mbar_wait_warp<true>(&sm.o_done[i], (n - 1) & 1, abort_flag, err, kErrTimeoutMma)) {
      tc_fence_after();
      // an empty row next to others: its probabilities, and so its O and l, are zeros
      store_row_bf16(tO, dst, limit > 0 ? 1.0f / l : 0.0f, store);
      if (store) *lse = limit > 0 ? kLn2 * (m_used + log2f(l)) : -INFINITY;
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

constexpr int kSmemBytes = (int)sizeof(Smem) + 1024;

}  // namespace

cudaError_t launch_attn_fwd_bf16_lse(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                     const TrainArgs& a, void* o, const long long o_str[3], float* lse,
                                     cudaStream_t stream) {
  static ContextOnce attr_done;
  cudaError_t e = attr_done.run([] {
    return cudaFuncSetAttribute(lse_fwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  });
  if (e != cudaSuccess) return e;
  Params p;
  p.mask = {a.kv_len, a.causal, a.Sq, a.Sk};
  p.c_log2 = a.c_log2;
  p.o = reinterpret_cast<__nv_bfloat16*>(o);
  p.o_sb = o_str[0];
  p.o_ss = o_str[1];
  p.o_sh = o_str[2];
  p.lse = lse;
  p.Hq = a.Hq;
  p.group = a.Hq / a.Hkv;
  p.BH = a.B * a.Hq;
  return launch_dependent(lse_fwd_kernel, heads_grid((a.Sq + kNQ * kTile - 1) / (kNQ * kTile), p.BH), kThreads,
                          kSmemBytes, stream, tm_q, tm_k, tm_v, p);
}

cudaError_t read_and_clear_err_lse(uint32_t* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_err_lse, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  const uint32_t zero = 0;
  return cudaMemcpyToSymbol(g_err_lse, &zero, sizeof(uint32_t));
}

}  // namespace sa
