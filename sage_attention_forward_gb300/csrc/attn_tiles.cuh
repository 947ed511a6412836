// What the training attention kernels (attn_lse.cu, attn_bwd.cu) share: 128 x 128 BF16
// tiles in shared memory, the products on them, and the masks.
//
// A query i of batch entry b sees the keys j < limit(i),
//   limit(i) = min(kv_len[b], causal ? i + 1 + (Sk - Sq) : Sk),
// which may be zero or negative: that row is empty.
#pragma once

#include <cstdint>

#include "kernels.h"
#include "ptx_train.cuh"

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

// The bounded waits of the load warp's thread, which may sleep on its barriers, and of the MMA warps,
// which wait as a whole.  The slow path is a call, so that the loops that wait stay small.
static __device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag,
                                              uint32_t* err_word, uint32_t err) {
  return mbar_wait<false>(bar, parity, abort_flag, err_word, err);
}
static __device__ __noinline__ bool wait_sleep(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag,
                                               uint32_t* err_word, uint32_t err) {
  return mbar_wait<true>(bar, parity, abort_flag, err_word, err);
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag,
                                          uint32_t* err_word, uint32_t err) {
  bool ok = mbar_try_wait<false>(bar, parity);
  if (!ok) ok = wait_slow(bar, parity, abort_flag, err_word, err);
  return __all_sync(0xffffffffu, ok);
}

// The tiles' 128-byte swizzle wants them on 1024-byte boundaries.  Dynamic shared memory declared so
// starts on one; should it not, the kernel says so and does nothing (there is no room to move up in).
__device__ __forceinline__ bool smem_misaligned(const uint8_t* smem, uint32_t* err_word) {
  if ((smem_u32(smem) & 1023u) == 0) return false;
  if (threadIdx.x == 0) atomicOr(err_word, kErrSmemBase);
  return true;
}

// ------------------------------------------------------------------ work
// The kernels launch one CTA per work item and run as many as there are SMs: a CTA that has the
// answer takes over an item whose CTA has not started, so that barriers, TMEM and descriptors are
// set up once, and the next item's loads and first products run under the last one's end
// (a CTA of its own costs about 14 K cycles outside its main loop).  Items start in grid order.
// The load warp asks for the next item ahead of time; every warp reads the answers in turn.
constexpr int kWorkSlots = 4;
struct WorkRing {
  alignas(16) uint4 answer[kWorkSlots];
  uint64_t full[kWorkSlots], empty[kWorkSlots];
};
struct Work {
  int index;   // the item's place in the grid
  int t;       // how many came before it in this CTA
};
__device__ __forceinline__ Work first_work() { return {(int)blockIdx.x, 0}; }
__device__ __forceinline__ bool work_answer(const uint4* answer, Work& w) {
  uint32_t x = 0, y = 0, z = 0;
  if (!clc_answer(answer, x, y, z)) return false;
  w.index = (int)x;
  return true;
}
// (by products: five divisions of each role at each item took about 1000 cycles)
__device__ __forceinline__ void work_place(const Order& o, const Work& w, int& tile, int& head) {
  const int g = div_by(w.index, o.by_group), first = g * o.group, at = w.index - g * (int)o.by_group.d;
  const bool rest = first + o.group > o.heads;
  tile = div_by(at, rest ? o.by_rest : o.by_heads);
  head = first + at - tile * (int)(rest ? o.by_rest.d : o.by_heads.d);
}
__device__ __forceinline__ void work_init(WorkRing& r, int reader_warps) {
  for (int s = 0; s < kWorkSlots; ++s) {
    mbar_init(&r.full[s], 1);
    mbar_init(&r.empty[s], reader_warps);
  }
}
// The load warp's thread: ask for item t > 0 (and for no other before that one's answer has been read).
__device__ __forceinline__ bool work_request(WorkRing& r, int t, volatile uint32_t* abort_flag, uint32_t* err) {
  const int s = (t - 1) % kWorkSlots, use = (t - 1) / kWorkSlots;
  if (use > 0 && !wait_sleep(&r.empty[s], (use - 1) & 1, abort_flag, err, kErrTimeoutSync)) return false;
  mbar_arrive_expect_tx(&r.full[s], 16);
  clc_try_cancel(&r.answer[s], &r.full[s]);
  return true;
}
// Item t, once its answer is there.  A warp short of registers reads it again rather than keep it.
__device__ __forceinline__ Work work_read(WorkRing& r, int t) {
  Work w = first_work();
  if (t > 0) work_answer(&r.answer[(t - 1) % kWorkSlots], w);
  w.t = t;
  return w;
}
// The same thread: w becomes the next item; false at the end (or after an abort).
__device__ __forceinline__ bool work_next_load(WorkRing& r, Work& w, volatile uint32_t* abort_flag, uint32_t* err) {
  const int s = w.t % kWorkSlots, use = w.t / kWorkSlots;
  ++w.t;
  return wait_sleep(&r.full[s], use & 1, abort_flag, err, kErrTimeoutSync) && work_answer(&r.answer[s], w);
}
// A whole warp: waits for the answer for item t > 0; whether there is such an item.
__device__ __forceinline__ bool work_wait(WorkRing& r, int t, volatile uint32_t* abort_flag, uint32_t* err) {
  const int s = (t - 1) % kWorkSlots, use = (t - 1) / kWorkSlots;
  Work w;
  return mbar_wait_warp<false>(&r.full[s], use & 1, abort_flag, err, kErrTimeoutSync) && work_answer(&r.answer[s], w);
}
// The warp is done with item t's answer.
__device__ __forceinline__ void work_release(WorkRing& r, int t, int lane) {
  if (t == 0) return;
  fence_proxy_async_smem();   // the slot is next written by the async proxy
  __syncwarp();
  if (lane == 0) mbar_arrive(&r.empty[(t - 1) % kWorkSlots]);
}
// After an abort: the last request has landed.
__device__ __forceinline__ void work_teardown(WorkRing& r, int requests) {
  if (requests > 0) mbar_wait_teardown(&r.full[(requests - 1) % kWorkSlots], ((requests - 1) / kWorkSlots) & 1);
}

// An MMA warp's walk over the tile products of all items.  It waits for an item's answer only
// after it has issued all of the item before: the softmax warps hold their place in the ring until
// their item's end, and further answers are not asked for until they get on.
enum : int { kEnd = 0, kValid = 1, kFirst = 2, kLast = 4 };
template <class Item, class Make>
struct Walk {
  Work w;
  Item item;   // the item of the latest product
  int j;       // that product's number within it, from 1
  Make make;
  __device__ __forceinline__ explicit Walk(Make m) : w(first_work()), item(m(w)), j(0), make(m) { settle(); }
  // (tcgen05.mma takes its operands from uniform registers: what the loop turns on is made uniform)
  __device__ __forceinline__ void settle() {
    item.n = __shfl_sync(0xffffffffu, item.n, 0);
    item.keys = __shfl_sync(0xffffffffu, item.keys, 0);
  }
  // the next product's flags; kEnd after the last
  __device__ __forceinline__ int next(WorkRing& r, int lane, volatile uint32_t* abort_flag, uint32_t* err) {
    while (j == item.n) {
      if (!work_wait(r, w.t + 1, abort_flag, err)) return kEnd;
      w = work_read(r, w.t + 1);
      work_release(r, w.t, lane);
      item = make(w);
      settle();
      j = 0;
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

// Rows past a batch entry's last key meet probabilities of zero in the products that sum over the
// keys, but hold whatever the caller's padding holds, and 0 * NaN is NaN: in the tile where an item's
// keys end they are set to zero in shared memory.  That is one warp's work: it waits for every
// tile of the ring in turn, clears where it has to, and tells the MMA threads by the slot's barrier.  A slot is
// loaded again only when this warp, too, is done with it: a turn of the ring behind the products, it would take
// another tile's phase for its own.
// (The swizzle permutes a row's 16-byte pieces within the row, so whole rows are contiguous.)
// How many of the rows of an item's last tile are keys; kTile: nothing to clear.
__device__ __forceinline__ int last_rows(const Mask& m, int keys, int n) {
  return keys < m.Sk && n * kTile > keys ? keys - (n - 1) * kTile : kTile;
}
// Arrivals that empty a slot of the ring whose tiles are cleared: the products', and the clearing warp's.
__device__ __forceinline__ int tile_releasers(const Mask& m) { return m.kv_len != nullptr ? 2 : 1; }
__device__ __forceinline__ void clear_rows(uint8_t* tile, int first, int lane) {
  for (int at = first * 128 + lane * 16; at < kHalfBytes; at += 32 * 16) {
    *reinterpret_cast<uint4*>(tile + at) = make_uint4(0u, 0u, 0u, 0u);
    *reinterpret_cast<uint4*>(tile + kHalfBytes + at) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncwarp();
}
// kFirst: an item's first tile is the one where its keys end, and not its last.
template <int kRing, bool kFirst, class Make>
__device__ __forceinline__ void clear_warp(const Mask& m, Make make, WorkRing& work, uint8_t (*tiles)[kTileBytes],
                                           uint64_t* full, uint64_t* empty, uint64_t* cleared, int lane,
                                           volatile uint32_t* abort_flag, uint32_t* err) {
  int it = 0, turn = 0;
  do {
    const auto item = make(work_read(work, turn));
    work_release(work, turn, lane);
    for (int begin = it, end = it + item.n; it != end; ++it) {
      const int slot = it % kRing;
      if (!mbar_wait_warp<true>(&full[slot], (it / kRing) & 1, abort_flag, err, kErrTimeoutTma)) return;
      const int rows = (kFirst ? it == begin : it + 1 == end) ? last_rows(m, item.keys, item.n) : kTile;
      if (rows < kTile) {
        clear_rows(tiles[slot], rows, lane);
        if (lane == 0) mbar_arrive(&cleared[slot]);
      }
      if (lane == 0) mbar_arrive(&empty[slot]);
    }
  } while (work_wait(work, ++turn, abort_flag, err));
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

// The products are issued by one lane of a warp that runs the loop as a whole: its descriptors and
// loop state are then uniform.  (Issued from a branch that one thread takes, each product took the
// forward 115 cycles instead of 80.)
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
