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

// D = A B^T over the 128 channels of two tiles in shared memory (scores, and dO V^T).
__device__ __forceinline__ void mma_tile_nt(uint32_t d, const uint8_t* a, const uint8_t* b, bool leader) {
  constexpr uint32_t idesc = idesc_f32acc(kFmtBF16, kFmtBF16, false, false, kTile, kTile);
  const uint64_t ad = smem_desc_sw128(smem_u32(a), 16, 1024), bd = smem_desc_sw128(smem_u32(b), 16, 1024);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint32_t off = ((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4;
    if (leader) mma_f16_ss(d, ad + off, bd + off, idesc, kk > 0 ? 1u : 0u);
  }
}

// D (+)= A B for 64 of the 128 summed rows of B: A is BF16 in TMEM, 32 columns from `a` (two
// values each); B is the tile's rows [64 * half, 64 * half + 64).
__device__ __forceinline__ void mma_tile_half_nn(uint32_t d, uint32_t a, const uint8_t* b, int half, bool accumulate,
                                                 bool leader) {
  constexpr uint32_t idesc = idesc_f32acc(kFmtBF16, kFmtBF16, false, true, kTile, kTile);
  const uint64_t bd = smem_desc_sw128(smem_u32(b), kHalfBytes, 1024);
#pragma unroll
  for (int k4 = 0; k4 < 4; ++k4) {
    const uint32_t off = ((4 * half + k4) * 2048) >> 4;
    if (leader) mma_f16_ts(d, a + k4 * 8, bd + off, idesc, (accumulate || k4 > 0) ? 1u : 0u);
  }
}

// 64 TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&a)[32], uint32_t (&b)[32]) {
  tmem_ld32(taddr, a);
  tmem_ld32(taddr + 32, b);
  tmem_ld_wait();
  tmem_reg_fence(a);
  tmem_reg_fence(b);
}

// kN accumulators of this thread's lane, times `factor`, as BF16 to dst.
template <int kN = 128>
__device__ __forceinline__ void store_row_bf16(uint32_t taddr, __nv_bfloat16* dst, float factor, bool store) {
#pragma unroll
  for (int cc = 0; cc < kN / 32; ++cc) {
    uint32_t o[32];
    tmem_ld32(taddr + 32 * cc, o);
    tmem_ld_wait();
    tmem_reg_fence(o);
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e)
      w[e] = pack_bf16x2(__uint_as_float(o[2 * e]) * factor, __uint_as_float(o[2 * e + 1]) * factor);
    if (store) {
      uint4* d4 = reinterpret_cast<uint4*>(dst + 32 * cc);
#pragma unroll
      for (int v = 0; v < 4; ++v) d4[v] = make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
    }
  }
}
template <int kN = 128>
__device__ __forceinline__ void store_row_zero(__nv_bfloat16* dst) {
  uint4* d4 = reinterpret_cast<uint4*>(dst);
#pragma unroll
  for (int v = 0; v < kN / 8; ++v) d4[v] = make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace tiles
}  // namespace sa
