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
constexpr int kWarpLoad = 8;
constexpr int kWarpMma = 9;
constexpr int kWarpClear = 10;
constexpr int kThreads = 352;
constexpr float kTau = 64.0f;   // as the BF16 forward: p <= 2^64 stays far inside BF16's and FP32's range
constexpr float kLn2 = 0.6931471805599453f;

struct __align__(1024) Smem {
  uint8_t q[kNQ][kTileBytes];
  uint8_t k[kStages][kTileBytes];
  uint8_t v[kStages][kTileBytes];
  uint8_t out[kWarpLoad][32 * 128];   // each softmax warp's 32 rows of O, 64 channels at a time
  WorkRing work;
  uint64_t q_full, q_empty;
  uint64_t k_full[kStages], k_empty[kStages];
  uint64_t v_full[kStages], v_empty[kStages], v_clear[kStages];
  uint64_t s_full[kNQ];
  uint64_t p_full[kNQ][2];   // P_i keys [0, 64) and [64, 128) stored in TMEM
  uint64_t o_done[kNQ];
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t abort_flag;
};

// Key tiles before an item's last at which the load warp asks for the next item: early enough to hide the
// answer's way, and late, because an SM that has asked has to take what it got.
constexpr int kAskAhead = 4;

__device__ uint32_t g_err_lse;
std::atomic<bool> g_launched{false};

struct Params {
  Mask mask;
  float c_log2;   // softmax_scale * log2 e
  float* lse;     // [B, Hq, Sq]
  int Hq, group;
  Div by_Hq, by_group;
  Order order;
};

__device__ __forceinline__ float u2f(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ uint32_t f2u(float f) { return __float_as_uint(f); }

// One item: two 128-row query tiles of one head, with the key tiles that they see.
struct Item {
  int b, h, row0, keys, n;   // n: key tiles; 0 when no row sees a key
};
__device__ __forceinline__ Item item_of(const Params& p, const Work& w) {
  Item i;
  int tile, head;
  work_place(p.order, w, tile, head);
  i.b = div_by(head, p.by_Hq);
  i.h = head - i.b * p.Hq;
  // the last queries have the most keys when the mask is causal: they start first
  i.row0 = (p.mask.causal ? p.order.tiles - 1 - tile : tile) * (kNQ * kTile);
  i.keys = key_count(p.mask, i.b);
  i.n = (row_limit(p.mask, i.keys, min(i.row0 + kNQ * kTile, p.mask.Sq) - 1) + kTile - 1) / kTile;
  return i;
}

__global__ void __launch_bounds__(kThreads, 1)
    lse_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);   // (known to be uniform)
  const int lane = threadIdx.x & 31;
  volatile uint32_t* abort_flag = &sm.abort_flag;
  uint32_t* err = &g_err_lse;

  if (threadIdx.x == 0) {
    work_init(sm.work, kWarpLoad + 1 + (p.mask.kv_len != nullptr ? 1 : 0));   // readers: softmax, MMA, clear
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 1);
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.v_empty[s], tile_releasers(p.mask));
      mbar_init(&sm.v_clear[s], 1);
    }
    for (int i = 0; i < kNQ; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i][0], 4);
      mbar_init(&sm.p_full[i][1], 4);
      mbar_init(&sm.o_done[i], 1);
    }
    mbar_init(&sm.drain, 1);
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
  constexpr uint32_t tmem = 0;   // all 512 columns are this CTA's: they start at 0

  if (warp == kWarpLoad) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      tma_prefetch_desc(&tm_o);
      int it = 0, items = 0, requests = 0, q_issued = 0, k_issued = 0, v_issued = 0;
      Work w = first_work();
      auto ask_next = [&]() -> bool {
        if (!work_request(sm.work, w.t + 1, abort_flag, err)) return false;
        ++requests;
        return true;
      };
      auto load_k = [&](const Item& i, int j, int hk) -> bool {
        const int at = it + j, slot = at % kStages, use = at / kStages;
        if (use > 0 && !wait_sleep(&sm.k_empty[slot], (use - 1) & 1, abort_flag, err, kErrTimeoutSync)) return false;
        mbar_arrive_expect_tx(&sm.k_full[slot], kTileBytes);
        load_tile(sm.k[slot], &tm_k, &sm.k_full[slot], j * kTile, hk, i.b);
        ++k_issued;
        return true;
      };
      auto load_item = [&](const Item& i) -> bool {
        const int hk = div_by(i.h, p.by_group);
        // (the first K has a free place before Q has: with Q first, at 4 key tiles an item, 51.4 us in place of 48.5)
        if (!load_k(i, 0, hk)) return false;
        if (items > 0 && !wait_sleep(&sm.q_empty, (items - 1) & 1, abort_flag, err, kErrTimeoutSync)) return false;
        mbar_arrive_expect_tx(&sm.q_full, kNQ * kTileBytes);
        for (int q = 0; q < kNQ; ++q) load_tile(sm.q[q], &tm_q, &sm.q_full, i.row0 + q * kTile, i.h, i.b);
        ++q_issued;
        const int ask = max(i.n - kAskAhead, 0);
        for (int j = 0; j < i.n; ++j) {
          if (j == ask && !ask_next()) return false;
          const int slot = (it + j) % kStages, use = (it + j) / kStages;
          if (use > 0 && !wait_sleep(&sm.v_empty[slot], (use - 1) & 1, abort_flag, err, kErrTimeoutSync)) return false;
          mbar_arrive_expect_tx(&sm.v_full[slot], kTileBytes);
          if (!withheld(v_issued++)) load_tile(sm.v[slot], &tm_v, &sm.v_full[slot], j * kTile, hk, i.b);
          if (j + 1 < i.n && !load_k(i, j + 1, hk)) return false;
        }
        it += i.n;
        ++items;
        return true;
      };
      do {
        const Item i = item_of(p, w);
        if (!(i.n > 0 ? load_item(i) : ask_next())) break;
      } while (work_next_load(sm.work, w, abort_flag, err));
      if (*abort_flag) {
        // nothing may land in this CTA's shared memory after it has gone
        work_teardown(sm.work, requests);
        if (q_issued) mbar_wait_teardown(&sm.q_full, (q_issued - 1) & 1);
        for (int i = max(k_issued - kStages, 0); i < k_issued; ++i)
          mbar_wait_teardown(&sm.k_full[i % kStages], (i / kStages) & 1);
        for (int i = max(v_issued - kStages, 0); i < v_issued; ++i)
          mbar_wait_teardown(&sm.v_full[i % kStages], (i / kStages) & 1);
      }
    }
  } else if (warp == kWarpMma) {
    // Over the key tiles i of all items: P_0 V(i), S_0(i+1), P_1 V(i), S_1(i+1), in this order: while
    // one Q tile's softmax runs the tensor core works on the other.  (A warp for each tile let their
    // products alternate, both S came late together, and a step took 3400 cycles instead of 2700.)
    // S_q(i+1) overwrites P_q(i) after the product that reads it.  An item's first P V overwrites the
    // O of the item before: the softmax warps published that P after they had read it.
    const bool leader = elect_one();
    const uint32_t dq = desc_k(sm.q[0]), dk = desc_k(sm.k[0]), dv = desc_mn(sm.v[0]);
    int q_items = 0;
    uint32_t cleared = 0;   // parity of each slot's clear barrier
    auto make = [&](const Work& w) { return item_of(p, w); };
    Walk<Item, decltype(make)> walk(make);
    int f0 = walk.next(sm.work, lane, abort_flag, err);
    // (a step's ring slots are compile-time constants, and so are the distances of its descriptors)
    auto wait_qk = [&](auto slot_c, int i, int flags) -> bool {
      constexpr int slot = decltype(slot_c)::value;
      if ((flags & kFirst) && !wait_warp(&sm.q_full, q_items++ & 1, abort_flag, err, kErrTimeoutTma)) return false;
      return wait_warp(&sm.k_full[slot], (i / kStages) & 1, abort_flag, err, kErrTimeoutTma);
    };
    auto issue_s = [&](auto slot_c, auto q_c, int flags) {
      constexpr int slot = decltype(slot_c)::value, q = decltype(q_c)::value;
      tc_fence_after();
      mma_tile_nt(tmem + 128 * q, dq + kDescTile * q, dk + kDescTile * slot, leader);
      if (leader) mma_commit(&sm.s_full[q]);
      if (leader && q == kNQ - 1) mma_commit(&sm.k_empty[slot]);
      if (leader && q == kNQ - 1 && (flags & kLast)) mma_commit(&sm.q_empty);
    };
    auto issue_pv = [&](auto slot_c, auto q_c, int i, bool first) -> bool {
      constexpr int slot = decltype(slot_c)::value, q = decltype(q_c)::value;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (!wait_warp(&sm.p_full[q][half], i & 1, abort_flag, err, kErrTimeoutSync)) return false;
        tc_fence_after();
        mma_tile_part_nn<64>(tmem + 256 + 128 * q, tmem + 128 * q + 32 * half, dv + kDescTile * slot, half,
                             !first || half > 0, leader);
      }
      if (leader) mma_commit(&sm.o_done[q]);
      return true;
    };
    const std::integral_constant<int, 0> c0;
    const std::integral_constant<int, 1> c1;
    auto step = [&](auto slot_c, auto next_c, int i) -> bool {
      constexpr int slot = decltype(slot_c)::value;
      const bool last = f0 & kLast, first = f0 & kFirst;
      const bool clear = last && last_rows(p.mask, walk.item.keys, walk.item.n) < kTile;
      if (!last) f0 = walk.next(sm.work, lane, abort_flag, err);
      if (!wait_warp(&sm.v_full[slot], (i / kStages) & 1, abort_flag, err, kErrTimeoutTma)) return false;
      if (clear) {
        if (!wait_warp(&sm.v_clear[slot], (cleared >> slot) & 1, abort_flag, err, kErrTimeoutSync)) return false;
        cleared ^= 1u << slot;
      }
      if (!issue_pv(slot_c, c0, i, first)) return false;
      if (!last) {
        if (!wait_qk(next_c, i + 1, f0)) return false;
        issue_s(next_c, c0, f0);
      }
      if (!issue_pv(slot_c, c1, i, first)) return false;
      if (leader) mma_commit(&sm.v_empty[slot]);
      if (last) {
        f0 = walk.next(sm.work, lane, abort_flag, err);
        if (f0 == kEnd) return true;
        if (!wait_qk(next_c, i + 1, f0)) return false;
        issue_s(next_c, c0, f0);
      }
      issue_s(next_c, c1, f0);
      return true;
    };
    static_assert(kStages == 2, "two copies of the step");
    bool ok = f0 == kEnd || wait_qk(c0, 0, f0);
    if (ok && f0 != kEnd) {
      issue_s(c0, c0, f0);
      issue_s(c0, c1, f0);
    }
    for (int i = 0; ok && f0 != kEnd; i += 2) {
      ok = step(c0, c1, i);
      if (ok && f0 != kEnd) ok = step(c1, c0, i + 1);
    }
    if (leader) mma_commit(&sm.drain);
    mbar_wait_teardown(&sm.drain, 0);
  } else if (warp == kWarpClear) {
    if (p.mask.kv_len != nullptr)
      clear_warp<kStages, false>(p.mask, [&](const Work& w) { return item_of(p, w); }, sm.work, sm.v, sm.v_full,
                                 sm.v_empty, sm.v_clear, lane, abort_flag, err);
  } else if (warp < kWarpLoad) {
    const int i = warp >> 2, wq = warp & 3;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + 128u * i;
    const uint32_t tO = tmem + lane_off + 256u + 128u * i;
    const float f = p.c_log2;
    bool ok = true;
    int it = 0, turn = 0;
    do {
      int n;
      int valid;   // what is left of the keys that this row sees
      {
        const Item item = item_of(p, work_read(sm.work, turn));
        n = item.n;
        valid = row_limit(p.mask, item.keys, item.row0 + i * kTile + wq * 32 + lane);
      }
      float m_used = -INFINITY, l = 0.0f;

      for (; n > 0; --n, ++it, valid -= kTile) {
        if (!mbar_wait_warp<false>(&sm.s_full[i], it & 1, abort_flag, err, kErrTimeoutMma)) { ok = false; break; }
        tc_fence_after();
        uint32_t s[128];
        uint32_t(&s0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&s[0]);
        uint32_t(&s1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&s[32]);
        uint32_t(&s2)[32] = *reinterpret_cast<uint32_t(*)[32]>(&s[64]);
        uint32_t(&s3)[32] = *reinterpret_cast<uint32_t(*)[32]>(&s[96]);
        const bool partial = __any_sync(0xffffffffu, valid < kTile);
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
        // (until a row's first key its O is zeros, or the item before's)
        const bool scale = need && m_used > -INFINITY;
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
              if (blk == 1 && __any_sync(0xffffffffu, scale)) {
                // O_i must hold P_{j-1} V_{j-1} before it is rescaled, and be rescaled before
                // the first half of P_j V_j accumulates into it
                if (mbar_wait_warp<true>(&sm.o_done[i], (it - 1) & 1, abort_flag, err, kErrTimeoutMma)) {
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

      if (!ok) break;
      const Item item = item_of(p, work_read(sm.work, turn));
      const int row = item.row0 + i * kTile + wq * 32 + lane;
      const bool some = row_limit(p.mask, item.keys, row) > 0;
      if (item.n > 0) {
        ok = mbar_wait_warp<true>(&sm.o_done[i], (it - 1) & 1, abort_flag, err, kErrTimeoutMma);
        if (!ok) break;
        tc_fence_after();
      }
      const int row0 = row - lane;
      // Through shared memory and TMA (16-byte piece c of row r at c ^ (r & 7)): stored from registers,
      // pieces exchanged between lanes for whole rows, O took 3600 cycles of an item.
      uint8_t* stage = sm.out[warp] + lane * 128;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t out[32] = {};
        // (an empty row next to others: its probabilities, and so its O and l, are zeros)
        if (item.n > 0) load_row_bf16<64>(tO + 64 * half, out, some ? 1.0f / l : 0.0f);
        if (lane == 0) bulk_wait_read();
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(stage + ((c ^ (lane & 7)) << 4)) =
              make_uint4(out[4 * c], out[4 * c + 1], out[4 * c + 2], out[4 * c + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && row0 < p.mask.Sq) tma_store_4d(&tm_o, sm.out[warp], 64 * half, row0, item.h, item.b);
      }
      tc_fence_before();
      if (row < p.mask.Sq)
        p.lse[((long long)item.b * p.Hq + item.h) * p.mask.Sq + row] = some ? kLn2 * (m_used + log2f(l)) : -INFINITY;
      work_release(sm.work, turn, lane);
    } while (work_wait(sm.work, ++turn, abort_flag, err));
    if (lane == 0) bulk_wait();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) {
    __syncwarp();
    tmem_dealloc(sm.tmem_base, 512);
  }
}

constexpr int kSmemBytes = (int)sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 232448, "227 KB of shared memory per CTA");

}  // namespace

cudaError_t launch_attn_fwd_bf16_lse(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                     const CUtensorMap& tm_o, const TrainArgs& a, float* lse, cudaStream_t stream) {
  static ContextOnce attr_done;
  cudaError_t e = attr_done.run([] {
    return cudaFuncSetAttribute(lse_fwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  });
  if (e != cudaSuccess) return e;
  Params p;
  p.mask = {a.kv_len, a.causal, a.Sq, a.Sk};
  p.c_log2 = a.c_log2;
  p.lse = lse;
  p.Hq = a.Hq;
  p.group = a.Hq / a.Hkv;
  p.by_Hq = make_div(a.Hq);
  p.by_group = make_div(p.group);
  p.order = make_order((a.Sq + kNQ * kTile - 1) / (kNQ * kTile), a.B * a.Hq, a.causal);
  g_launched.store(true, std::memory_order_relaxed);
  return launch_dependent(lse_fwd_kernel, dim3((unsigned)p.order.items), kThreads, kSmemBytes, stream, tm_q, tm_k, tm_v,
                          tm_o, p);
}

static const bool err_reader_added =
    add_err_reader([](uint32_t* out) { return read_and_clear_err(g_err_lse, g_launched, out); });

}  // namespace sa
