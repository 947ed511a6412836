// What the training attention kernels (attn_lse.cu, attn_bwd.cu) share: 128 x 128 BF16
// tiles in shared memory, the products on them, and the masks.
//
// A query i of batch entry b sees the keys j < limit(i),
//   limit(i) = min(kv_len[b], causal ? i + 1 + (Sk - Sq) : Sk),
// which may be zero or negative: that row is empty.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace sa {
namespace tiles {

constexpr int kTile = 128;                          // rows of a tile, and its channels
constexpr int kTileBytes = kTile * kTile * 2;       // BF16, two [128 rows][64 channels] halves, 128-byte swizzle
constexpr int kHalfBytes = kTileBytes / 2;

struct Mask {
  const int* kv_len;   // [B] keys per batch entry (clamped to [0, Sk]), or nullptr: Sk
  int causal;
  int Sq, Sk;
};

__device__ __forceinline__ int key_count(const Mask& m, int b) {
  return m.kv_len == nullptr ? m.Sk : min(max(__ldg(m.kv_len + b), 0), m.Sk);
}
// limit(i), clamped below at 0
__device__ __forceinline__ int row_limit(const Mask& m, int keys, int i) {
  return m.causal ? max(min(keys, i + 1 + (m.Sk - m.Sq)), 0) : keys;
}

// The MMA and load warps wait through these: the slow path of a bounded wait is a call, which keeps
// their loops within the instruction cache (inlined at every wait, and with the loops unrolled by
// their rings, dQ took 2880 cycles a tile pair instead of 2320).
static __device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag,
                                              uint32_t* err_word, uint32_t err) {
  return mbar_wait<false>(bar, parity, abort_flag, err_word, err);
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag,
                                          uint32_t* err_word, uint32_t err) {
  bool ok = mbar_try_wait<false>(bar, parity);
  if (!ok) ok = wait_slow(bar, parity, abort_flag, err_word, err);
  return __all_sync(0xffffffffu, ok);
}
// One thread of the load warp, whose waits may sleep on their barriers.
static __device__ __noinline__ bool wait_one(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag,
                                             uint32_t* err_word, uint32_t err) {
  return mbar_wait<true>(bar, parity, abort_flag, err_word, err);
}

// ------------------------------------------------------------------ work
// The kernels launch one CTA per work item and run as many as there are SMs: a CTA that has the
// answer takes over an item whose CTA has not started, so that barriers, TMEM and descriptors are
// set up once, and the next item's loads and first products run under the last one's end
// (a CTA of its own costs about 14 K cycles outside its main loop).  Items start in grid order.
// The load warp asks for item t + 1 when it starts item t; every warp reads the answers in turn.
constexpr int kWorkSlots = 4;
struct WorkRing {
  alignas(16) uint4 answer[kWorkSlots];
  uint64_t full[kWorkSlots], empty[kWorkSlots];
};
struct Work {
  int x, head;   // the item's place in the grid (heads_grid)
  int t;         // how many came before it in this CTA
};
__device__ __forceinline__ Work first_work() { return {(int)blockIdx.x, (int)(blockIdx.y + gridDim.y * blockIdx.z), 0}; }
__device__ __forceinline__ bool work_answer(const uint4* answer, Work& w) {
  uint32_t x = 0, y = 0, z = 0;
  if (!clc_answer(answer, x, y, z)) return false;
  w.x = (int)x;
  w.head = (int)(y + gridDim.y * z);
  return true;
}
__device__ __forceinline__ void work_init(WorkRing& r, int reader_warps) {
  for (int s = 0; s < kWorkSlots; ++s) {
    mbar_init(&r.full[s], 1);
    mbar_init(&r.empty[s], reader_warps);
  }
}
// One thread of the load warp: ask for the item after w.
__device__ __forceinline__ bool work_request(WorkRing& r, const Work& w, volatile uint32_t* abort_flag, uint32_t* err) {
  const int s = w.t % kWorkSlots, use = w.t / kWorkSlots;
  if (use > 0 && !wait_one(&r.empty[s], (use - 1) & 1, abort_flag, err, kErrTimeoutSync)) return false;
  mbar_arrive_expect_tx(&r.full[s], 16);
  clc_try_cancel(&r.answer[s], &r.full[s]);
  return true;
}
// The same thread: the answer, w becomes it; false at the end (or after an abort).
__device__ __forceinline__ bool work_next_load(WorkRing& r, Work& w, volatile uint32_t* abort_flag, uint32_t* err) {
  const int s = w.t % kWorkSlots, use = w.t / kWorkSlots;
  ++w.t;
  return wait_one(&r.full[s], use & 1, abort_flag, err, kErrTimeoutSync) &&
         work_answer(&r.answer[s], w);
}
// A whole reader warp: waits for the answer for item t > 0; whether there is such an item.
__device__ __forceinline__ bool work_wait(WorkRing& r, int t, volatile uint32_t* abort_flag, uint32_t* err) {
  const int s = (t - 1) % kWorkSlots, use = (t - 1) / kWorkSlots;
  Work w;
  return mbar_wait_warp<false>(&r.full[s], use & 1, abort_flag, err, kErrTimeoutSync) && work_answer(&r.answer[s], w);
}
// Item t, after work_wait.  A warp short of registers reads it again rather than keep it.
__device__ __forceinline__ Work work_read(WorkRing& r, int t) {
  Work w = first_work();
  if (t > 0) work_answer(&r.answer[(t - 1) % kWorkSlots], w);
  w.t = t;
  return w;
}
// The warp is done with item t's answer.
__device__ __forceinline__ void work_release(WorkRing& r, int t, int lane) {
  if (t == 0) return;
  fence_proxy_async_smem();   // the slot is next written by the async proxy
  __syncwarp();
  if (lane == 0) mbar_arrive(&r.empty[(t - 1) % kWorkSlots]);
}
// All three: w becomes the next item.
__device__ __forceinline__ bool work_next(WorkRing& r, Work& w, int lane, volatile uint32_t* abort_flag, uint32_t* err) {
  if (!work_wait(r, w.t + 1, abort_flag, err)) return false;
  w = work_read(r, w.t + 1);
  work_release(r, w.t, lane);
  return true;
}
// After an abort: the request after item w, if it was made, has landed.
__device__ __forceinline__ void work_teardown(WorkRing& r, int requests) {
  if (requests > 0) mbar_wait_teardown(&r.full[(requests - 1) % kWorkSlots], ((requests - 1) / kWorkSlots) & 1);
}

// Whether work_wait(r, t) would return at once (the same for the whole warp).
__device__ __forceinline__ bool work_ready(WorkRing& r, int t) {
  const int s = (t - 1) % kWorkSlots, use = (t - 1) / kWorkSlots;
  return __all_sync(0xffffffffu, mbar_try_wait<false>(&r.full[s], use & 1));
}

// The MMA warp's walk over the tile products of all items, each known before it is issued.
// An item's last product must be issued whole before the warp waits for another item: the softmax
// warps hold their place in the ring until their item's end, so that a walk over several empty
// items would otherwise wait for an answer that is not asked for before they get on.
enum : int { kUnknown = -1, kEnd = 0, kValid = 1, kFirst = 2, kLast = 4 };
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }   // the same for the whole warp, and known to be
template <class Item, class Make>
struct Walk {
  Work w;
  Item item;   // the item of the latest product
  int j;       // that product's number within it, from 1
  Make make;
  __device__ __forceinline__ explicit Walk(Make m) : w(first_work()), item(m(w)), j(0), make(m) { settle(); }
  // (tcgen05.mma takes its descriptors from uniform registers: what the loop turns on must be uniform)
  __device__ __forceinline__ void settle() {
    item.n = uniform(item.n);
    item.keys = uniform(item.keys);
  }
  // The next product's flags; kEnd after the last.  With wait = false an answer that is not there
  // yet, or a next item without products, is kUnknown.
  __device__ __forceinline__ int next(bool wait, WorkRing& r, int lane, volatile uint32_t* abort_flag, uint32_t* err) {
    while (j == item.n) {
      if (!wait && !work_ready(r, w.t + 1)) return kUnknown;
      if (!work_next(r, w, lane, abort_flag, err)) return kEnd;
      item = make(w);
      settle();
      j = 0;
      if (!wait && item.n == 0) return kUnknown;
    }
    ++j;
    return kValid | (j == 1 ? kFirst : 0) | (j == item.n ? kLast : 0);
  }
};

// One 128-row tile of a BF16 [B, S, H, 128] tensor; rows past S read as 0.
__device__ __forceinline__ void load_tile(uint8_t* dst, const void* tmap, uint64_t* bar, int row, int h, int b) {
  tma_load_4d(dst, tmap, bar, 0, row, h, b);
  tma_load_4d(dst + kHalfBytes, tmap, bar, 64, row, h, b);
}

// A tile's rows [first, 128) set to zero by one warp, for the tensor core: rows past a batch
// entry's last key meet probabilities of zero in the products, but hold whatever the caller's
// padding holds, and 0 * NaN is NaN.  (The swizzle permutes a row's 16-byte pieces within the
// row, so whole rows are contiguous.)  Call after the tile has landed.
__device__ __forceinline__ void clear_rows(uint8_t* tile, int first, int lane) {
  for (int at = first * 128 + lane * 16; at < kHalfBytes; at += 32 * 16) {
    *reinterpret_cast<uint4*>(tile + at) = make_uint4(0u, 0u, 0u, 0u);
    *reinterpret_cast<uint4*>(tile + kHalfBytes + at) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// The low word of a tile's shared-memory descriptor (the high word is the same for all): the rows
// read as K-major, or as MN-major (channels; its two 64-channel halves are lbo apart).  Tile t of an
// array is kDescTile * t further.
constexpr uint32_t kDescTile = kTileBytes >> 4;
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);   // smem_desc_sw128's: 1024-byte groups of 8 rows
__device__ __forceinline__ uint32_t desc_k(const uint8_t* tile) { return ((smem_u32(tile) >> 4) & 0x3FFFu) | ((16u >> 4) << 16); }
__device__ __forceinline__ uint32_t desc_mn(const uint8_t* tile) {
  return ((smem_u32(tile) >> 4) & 0x3FFFu) | ((uint32_t)(kHalfBytes >> 4) << 16);
}
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) { return ((uint64_t)kDescHi << 32) | lo; }

// D = A B^T over the 128 channels of two tiles in shared memory (scores, and dO V^T).
__device__ __forceinline__ void mma_tile_nt(uint32_t d, uint32_t a_desc_k, uint32_t b_desc_k, bool leader) {
  constexpr uint32_t idesc = idesc_f32acc(kFmtBF16, kFmtBF16, false, false, kTile, kTile);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint32_t off = ((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4;
    if (leader) mma_f16_ss(d, desc_of(a_desc_k + off), desc_of(b_desc_k + off), idesc, kk > 0 ? 1u : 0u);
  }
}

// The same with A, BF16, in 64 columns of TMEM from `a`.
__device__ __forceinline__ void mma_tile_nt_ts(uint32_t d, uint32_t a, uint32_t b_desc_k, bool leader) {
  constexpr uint32_t idesc = idesc_f32acc(kFmtBF16, kFmtBF16, false, false, kTile, kTile);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint32_t off = ((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4;
    if (leader) mma_f16_ts(d, a + kk * 8, desc_of(b_desc_k + off), idesc, kk > 0 ? 1u : 0u);
  }
}

// D (+)= A B for `kRows` of the 128 summed rows of B, from row kRows * part on: A is BF16 in TMEM,
// kRows / 2 columns from `a` (two values each).
template <int kRows>
__device__ __forceinline__ void mma_tile_part_nn(uint32_t d, uint32_t a, uint32_t b_desc_mn, int part, bool accumulate,
                                                 bool leader) {
  constexpr uint32_t idesc = idesc_f32acc(kFmtBF16, kFmtBF16, false, true, kTile, kTile);
#pragma unroll
  for (int k = 0; k < kRows / 16; ++k) {
    const uint32_t off = ((kRows / 16 * part + k) * 2048) >> 4;
    if (leader) mma_f16_ts(d, a + k * 8, desc_of(b_desc_mn + off), idesc, (accumulate || k > 0) ? 1u : 0u);
  }
}

// kN accumulators of this thread's lane, times `factor`, as packed BF16.
template <int kN>
__device__ __forceinline__ void load_row_bf16(uint32_t taddr, uint32_t (&w)[kN / 2], float factor) {
#pragma unroll
  for (int cc = 0; cc < kN / 32; ++cc) {
    uint32_t o[32];
    tmem_ld32(taddr + 32 * cc, o);
    tmem_ld_wait();
    tmem_reg_fence(o);
#pragma unroll
    for (int e = 0; e < 16; ++e)
      w[16 * cc + e] = pack_bf16x2(__uint_as_float(o[2 * e]) * factor, __uint_as_float(o[2 * e + 1]) * factor);
  }
}
// The rows of a warp's 32 lanes, kN packed BF16 channels each, to global memory: the 16-byte pieces
// change lanes (a transposition within groups of kN / 8 lanes) so that each store covers whole
// rows' pieces next to one another.  One row per lane touched 32 cache lines a store, and
// took 7000 cycles for a 128 x 256 result.
// base: the first row's channels; rows: how many of the 32 to store.
template <int kN>
__device__ __forceinline__ void store_rows(__nv_bfloat16* base, long long row_stride, uint32_t (&w)[kN / 2], int rows,
                                           int lane) {
  constexpr int kPieces = kN / 8;
#pragma unroll
  for (int bit = 1; bit < kPieces; bit <<= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if (i & bit) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t &x = w[4 * i + e], &y = w[4 * (i | bit) + e];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? x : y, bit);
        if (up) x = got;
        else y = got;
      }
    }
  }
  const int first = lane & ~(kPieces - 1);
  uint4* dst = reinterpret_cast<uint4*>(base + first * row_stride) + (lane & (kPieces - 1));
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
    if (first + i < rows)
      *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(dst) + i * row_stride) =
          make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

}  // namespace tiles
}  // namespace sa
