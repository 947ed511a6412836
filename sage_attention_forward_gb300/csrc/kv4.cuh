// The K/V cache in 4 bits: its layout, and a walk's arithmetic.
//
// A record holds 16 tokens of one key head: K's codes, V's codes and the scales, 2304 bytes, 4.5 bits a value.  Records are
// stored as mma.m16n8k16 reads them (kv4_attn.cu), so that a warp takes a record with 16-byte accesses and no lane needs
// another's bytes:
//   [0, 1024)     K, 64 bytes a token: word (4 t + g) has channels 32 g + 8 t + i at bits 4 i (t, g = 0..3, i = 0..7)
//   [1024, 2048)  V, token j at 512 (j / 8) + 16 (4 r + j % 8 / 2) + 8 (j % 2) for r = 0..7: two words, halves of 16 bits by
//                 group g, channel 32 g + 4 r + i at bits 4 i of its half (i = 0..3)
//   [2048, 2304)  16 bytes a token: BF16 scales of K's four groups, then of V's
// A code is a value plus 8; it stands for (code - 8) scale.
#pragma once

#include <cuda_bf16.h>

#include "kernels.h"

namespace sa {

constexpr int kKvTile = 16;              // tokens of a record
constexpr int kKvRecord = 2304;
constexpr int kKvV = 1024, kKvScales = 2048;

// The pages of a request's tokens.
struct KvPages {
  unsigned char* cache;                  // [num_pages][heads][tiles][kKvRecord]
  const int* table;                      // [B][max_pages], rows table_str apart
  long long table_str;
  int num_pages, max_pages, heads;
  Div tiles;                             // records of a page and head
};
inline KvPages kv4_pages(const Kv4Args& a) {
  KvPages p;
  p.cache = reinterpret_cast<unsigned char*>(a.cache);
  p.table = a.table;
  p.table_str = a.table_str;
  p.num_pages = a.num_pages;
  p.max_pages = a.max_pages;
  p.heads = a.Hkv;
  p.tiles = make_div(a.page_size / kKvTile);
  return p;
}
// The page of a request's tile, or -1 where there is none.
__device__ __forceinline__ int kv_page(const KvPages& p, int b, int tile) {
  const int at = div_by(tile, p.tiles);
  if (at >= p.max_pages) return -1;
  const int page = __ldg(p.table + b * p.table_str + at);
  return page >= 0 && page < p.num_pages ? page : -1;
}
__device__ __forceinline__ unsigned char* kv_record(const KvPages& p, int page, int head, int tile) {
  const int in_page = tile - div_by(tile, p.tiles) * (int)p.tiles.d;
  return p.cache + (((long long)page * p.heads + head) * (int)p.tiles.d + in_page) * kKvRecord;
}

}  // namespace sa
