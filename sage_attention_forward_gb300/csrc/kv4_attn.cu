// Attention over a K/V cache in 4 bits, sm_103a: O = softmax(scale q K^T) V for one or a few queries of each request.
//
// Bound by memory: 144 bytes of cache a token and key head, read once for all queries that share the head.
//
// Products.  Keys (and V's channels) are the rows of mma.m16n8k16, the queries of a key head (tokens x heads that share it) its
// columns, so that each code is unpacked once for all of them.  Codes become operands without a conversion: four bits put into
// the mantissa of a constant are the value constant + code.
//   S^T = sum_g scale_K[key, g] (codes_g q_g)        FP16, two products for each 32 channels, scaled in FP32
//   O^T[group g] = sum_j codes (p_j scale_V[j, g])   FP16; P is scaled for each group in FP32, then rounded once
// K's codes are 256 + c and 16 + c (one shift and one masked insert for two values); what the constants and the codes' bias add,
// 264 q and 24 q summed over the channels, is taken off, formed by a product of the same operands.  (FP32 rounds the sums beside
// those parts: scores came out within 5 10^-7 rms, 4 10^-6 at most, of sum |q k|; exactly for queries of 8 whole bits.)  V's are 1024 + c and 64 + c
// where they stand, from which 1032 and 72 are subtracted, exactly: sums over many keys may be small beside their parts.
// Q becomes FP16 with its row's largest magnitude in [1, 2): its own 8 bits stay (what is below 2^-14 of that magnitude is off
// by up to 2^-25 of it).  P scale_V becomes FP16 with the largest scale of its group that the warp has met in [2^6, 2^7): a power
// of two that follows, and O's channels with it, as a row's reference maximum does.  (What is below 2^-14 then is off by up to
// 2^-25: by 2^-31 of the group's largest scale.)
// (e4m3 operands would need only masks, but mma.sync has no e4m3 on this machine: it came to 19 instructions a product.)
//
// Work.  The records of all requests and heads are one line of work, cut into items of equal length, found from the lengths on
// the device, so that ragged batches are balanced and a graph serves any lengths.  A warp takes an item, through its own ring
// of cp.async copies and with a softmax of its own.  Where an item holds a request's head only in part, its piece goes to the
// workspace, and a second kernel joins a head's pieces in order.  (All warps of an SM are one CTA's: of three CTAs of four warps
// the first was served first and ended at 152 us, the last at 207.  Two and six shorter items a warp: 8 x 131072 tokens 210 and
// 231 us in place of 205, an item's start and end taking 5 us.)
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kv4.cuh"
#include "pieces.cuh"

namespace sa {
namespace {

constexpr int kHeld = 6;            // records of a warp's ring
constexpr int kLeast = 2;           // records of an item, at least
constexpr int kStart = 4;           // what a segment's start and end cost beside its records, in records
constexpr int kCtas = 152;
constexpr float kSlack = 8.0f;      // a row's reference maximum is raised when one passes it by more (log2 units)
constexpr float kNone = -1.5e38f;    // a row's maximum before its first key (finite: differences of two are no NaN)
constexpr float kPart = 0x1p-30f;   // O's sums are taken times this: those of many keys of V's largest values stay finite
constexpr int kDim = 128;

struct AttnParams {
  KvPages pages;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  const int* kv_len;
  long long q_str[3], o_str[3];
  int B, S, Hq, rows;               // rows: queries of a key head, S * G
  int row_tiles, segments;          // segments: row tiles of a request over all its key heads
  int capacity;                     // tokens that a table row can hold
  Div G, by_row_tiles, by_segments;
  int causal;
  float c_log2;
  int ctas;
  // workspace
  int2* head;                       // [request][segment]: first item, pieces (1: complete)
  float* part_o;                    // pieces, [item][2][rows of a tile]
  float2* part_ml;
};

// 16 bytes at src, or zeros (size = 0: nothing is read); where `on` is false nothing is written
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t size, bool on = true) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\t@p cp.async.cg.shared.global [%0], [%1], 16, %2;\n\t}" ::"r"(dst), "l"(src),
      "r"(size), "r"((uint32_t)on)
      : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit values, a row to four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// V: four codes of each of two tokens, 4 bits each in halves of x, as FP16 pairs of code - 8.  low, high: FP16 1024 and 64
// twice, in registers (an instruction takes one constant).
__device__ __forceinline__ void v_pairs(uint32_t x, uint32_t low, uint32_t high, uint32_t (&a)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t y = i == 0 ? x : x >> 8;
    asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xEA;" : "=r"(a[2 * i]) : "r"(y), "r"(low));        // (y & mask) | 1024
    asm("lop3.b32 %0, %1, 0x00f000f0, %2, 0xEA;" : "=r"(a[2 * i + 1]) : "r"(y), "r"(high));
    asm("add.rn.f16x2 %0, %0, %1;" : "+r"(a[2 * i]) : "r"(0xe408e408u));                      // - 1032
    asm("add.rn.f16x2 %0, %0, %1;" : "+r"(a[2 * i + 1]) : "r"(0xd480d480u));                  // - 72
  }
}
// The larger magnitude of each half (its sign is of no use).
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// K: eight codes as FP16 pairs (i, i + 4): 256 + c for i = 0 and 2, 16 + c for i = 1 and 3.  wide, near: FP16 256 and 16 twice.
__device__ __forceinline__ void k_pairs(uint32_t w, uint32_t wide, uint32_t near, uint32_t (&a)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = i == 0 ? w << 2 : w >> 6;
    asm("lop3.b32 %0, %1, 0x003c003c, %2, 0xEA;" : "=r"(a[2 * i]) : "r"(x), "r"(wide));
    asm("lop3.b32 %0, %1, 0x03c003c0, %2, 0xEA;" : "=r"(a[2 * i + 1]) : "r"(x), "r"(near));
  }
}
__device__ __forceinline__ void scales_of(uint32_t w, float& a, float& b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}

__device__ __forceinline__ int tokens_of(const AttnParams& p, int b) { return min(max(__ldg(p.kv_len + b), 0), p.capacity); }

// One CTA an SM, of as many warps as the registers allow.
constexpr int warps(int rows) { return rows == 4 ? 12 : rows == 8 ? 11 : 8; }
// Records that a warp works on at a time: two, whose products do not wait for one another (8 x 131072 tokens, three CTAs of four
// warps: one at a time 257 us, two 243); one where the registers do not reach for two.
constexpr int together(int rows) { return rows <= 8 ? 2 : 1; }
constexpr int kRing = kHeld * kKvRecord;   // shared memory of a warp

// kRows: queries that an item's records are read for, 4, 8 or 16.  Four of them are the even columns of a product's eight, so
// that every lane has scores of one.
template <int kRows>
__global__ void __launch_bounds__(32 * warps(kRows), 1) kv4_attn_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kWarps = warps(kRows), kThreads = 32 * kWarps;
  constexpr int kCols = (kRows + 7) / 8;                   // columns of eight
  constexpr int kEach = kRows == 4 ? 1 : 2;                // queries of a lane and column
  constexpr int kPair = together(kRows), kStages = kHeld / kPair;
  // V's scales times their power of two: as they are loaded, or where they are used (8 x 131072 tokens, one query token of 32 and of
  // 64 heads on 8, and 8 x 65536 tokens, four of 32: loaded 193, 244, 189 us; used 199, 237, 183)
  constexpr bool kEarly = kRows == 4;
  auto early = [](uint32_t x, uint32_t d) { return kEarly ? mul_bf16x2(x, d) : x; };
  auto late = [](uint32_t x, uint32_t d) { return kEarly ? x : mul_bf16x2(x, d); };
  extern __shared__ __align__(16) unsigned char rings[];
  __shared__ long long warp_sums[kWarps];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, t = lane & 3;

  // the line's length, and an item's
  auto work_of = [&](int b) {
    const int n = b < p.B ? (tokens_of(p, b) + kKvTile - 1) / kKvTile : 0;
    return n > 0 ? (long long)(n + kStart) * p.segments : 0ll;
  };
  long long total = 0;
  for (int b = threadIdx.x; b < p.B; b += kThreads) total += work_of(b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) warp_sums[warp] = total;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += warp_sums[w];
  const long long most = (long long)p.ctas * kWarps;
  const long long share = max((long long)kLeast, (total + most - 1) / most);
  // requests without a key: nobody's work
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (tokens_of(p, b) != 0) continue;
    for (long long i = threadIdx.x; i < (long long)p.S * p.Hq * (kDim / 8); i += kThreads) {
      const long long row = i / (kDim / 8);
      const int s = (int)(row / p.Hq), h = (int)(row - (long long)s * p.Hq);
      *reinterpret_cast<uint4*>(p.o + b * p.o_str[0] + s * p.o_str[1] + h * p.o_str[2] + (int)(i % (kDim / 8)) * 8) =
          make_uint4(0u, 0u, 0u, 0u);
      if (i % (kDim / 8) == 0) p.lse[((long long)b * p.Hq + h) * p.S + s] = -INFINITY;
    }
  }

  // The warp's place in the line: request b starts at `before`
  int b = 0;
  const int item = blockIdx.x + warp * p.ctas;   // (few items: one for each CTA)
  long long before = 0, at = item * share;
  const long long stop = min(at + share, total);
  // A segment's records: the item's are [first, last)
  int len, tiles, seg, head, row0, first, last;
  long long seg_start;
  unsigned char* const mine = rings + warp * kRing;
  uint32_t there;                                   // bit of a place in the ring: its record has a page
  int to_load, left, next;                          // left: records of the current page; next: the page after it
  bool paged;
  const unsigned char* from;
  auto load = [&](int slot) {
#pragma unroll
    for (int j = 0; j < kPair; ++j) {
      if (left == 0) {
        paged = to_load < last && next >= 0;
        left = (int)p.pages.tiles.d - (to_load - div_by(to_load, p.pages.tiles) * (int)p.pages.tiles.d);
        if (paged) from = kv_record(p.pages, next, head, to_load) + lane * 16;
        if (to_load + left < last) next = kv_page(p.pages, b, to_load + left);
      }
      const bool held = paged && to_load < last;
      const int place = slot * kPair + j;
      const uint32_t into = smem_u32(mine) + place * kKvRecord + lane * 16;
      there = (there & ~(1u << place)) | (uint32_t)held << place;
#pragma unroll
      for (int i = 0; i < 5; ++i) cp_async16(into + i * 512, from + i * 512, held ? 16u : 0u, i < 4 || lane < 16);
      from += kKvRecord;
      ++to_load;
      --left;
    }
    cp_async_commit();
  };
  // Finds the next segment of the item and starts to load its records; false at its end.
  auto begin = [&]() -> bool {
    for (;;) {
      if (at >= stop) return false;
      // the request that `at` is in: 32 looked at together
      long long work = work_of(b + lane), end = work;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end += up;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, at < before + end);
      const int step = past != 0 ? __ffs((int)past) - 1 : 31;
      work = __shfl_sync(0xffffffffu, work, step);
      before += __shfl_sync(0xffffffffu, end, step) - (past != 0 ? work : 0);
      b += past != 0 ? step : 32;
      if (past == 0) {
        if (b >= p.B) return false;   // (lengths that changed under way)
        continue;
      }
      len = tokens_of(p, b);
      tiles = (len + kKvTile - 1) / kKvTile;
      seg = (int)((at - before) / (tiles + kStart));
      seg_start = before + (long long)seg * (tiles + kStart) + kStart;
      first = (int)max(0ll, at - seg_start);
      last = (int)min((long long)tiles, stop - seg_start);
      at = seg_start + last;
      if (last > first) break;   // (else the item ends before the segment's first record)
    }
    head = div_by(seg, p.by_row_tiles);
    row0 = (seg - head * p.row_tiles) * kRows;
    there = 0;
    to_load = first;
    left = 0;
    paged = false;
    from = p.pages.cache;
    next = first < last ? kv_page(p.pages, b, first) : -1;
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) load(i);
    return true;
  };
  bool more = begin();
  while (more) {
    // queries
    uint32_t qf[kCols][4][4];
    float off[kCols][kEach][4], factor[kCols][kEach];
    int limit[kCols][kEach], all = len;   // keys before `all` are seen by every query of the tile
#pragma unroll
    for (int n = 0; n < kCols; ++n) {
      const int row = kRows == 4 ? row0 + r / 2 : row0 + 8 * n + r;
      const int s = div_by(row, p.G), g0 = row - s * (int)p.G.d;
      uint4 raw[4] = {};
      if (row < p.rows && (kRows != 4 || r % 2 == 0)) {
        const uint4* const src = reinterpret_cast<const uint4*>(p.q + b * p.q_str[0] + s * p.q_str[1] +
                                                                (long long)(head * (int)p.G.d + g0) * p.q_str[2]);
#pragma unroll
        for (int g = 0; g < 4; ++g) raw[g] = __ldg(src + 4 * g + t);
      }
      float top = 0.0f;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float x[8];
        unpack<__nv_bfloat16>(raw[g], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = min(max((int)(__float_as_uint(top) >> 23), 27), 253);
      const float down = __uint_as_float((uint32_t)(254 - e) << 23);
      const float up = __uint_as_float((uint32_t)e << 23) * p.c_log2;
#pragma unroll
      for (int c = 0; c < kEach; ++c) factor[n][c] = __shfl_sync(0xffffffffu, up, 4 * (2 * t + c));
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float x[8];
        unpack<__nv_bfloat16>(raw[g], x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 h = __floats2half2_rn(x[i] * down, x[i + 4] * down);
          qf[n][g][i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        float d[4] = {};
        mma_f16(d, 0xdc20dc20u, 0xdc20dc20u, 0xce00ce00u, 0xce00ce00u, qf[n][g][0], qf[n][g][1]);   // -264, -24
        mma_f16(d, 0xdc20dc20u, 0xdc20dc20u, 0xce00ce00u, 0xce00ce00u, qf[n][g][2], qf[n][g][3]);
#pragma unroll
        for (int c = 0; c < kEach; ++c) off[n][c][g] = d[c];
      }
#pragma unroll
      for (int c = 0; c < kEach; ++c) {
        const int tok = div_by(row0 + 8 * n + kEach * t + c, p.G);
        limit[n][c] = p.causal ? min(len, len - p.S + tok + 1) : len;
      }
    }
    if (p.causal) all = max(0, min(len, len - p.S + div_by(row0, p.G) + 1));

    // [group][pair of channel rows][column]; kRows = 4: columns 2 t and 2 t + 1 are query t with the scales of an even
    // and of an odd group, one of which counts
    float acc[4][2][kCols][4] = {};
    float m[kCols][kEach], l[kCols][kEach];
#pragma unroll
    for (int n = 0; n < kCols; ++n)
#pragma unroll
      for (int c = 0; c < kEach; ++c) {
        m[n][c] = kNone;
        l[n][c] = 0.0f;
      }

    uint32_t low, high, wide, near;
    asm volatile("mov.b32 %0, 0x64006400;\n\tmov.b32 %1, 0x54005400;" : "=r"(low), "=r"(high));
    asm volatile("mov.b32 %0, 0x5c005c00;\n\tmov.b32 %1, 0x4c004c00;" : "=r"(wide), "=r"(near));
    // BF16 pairs of groups (0, 1) and (2, 3) of V: powers of two, 2^100 at most, that bring the scales met so far below 2^7
    uint32_t down[2] = {0x71807180u, 0x71807180u};
    int slot = 0;
#pragma unroll 1
    for (int tile = first; tile < last; tile += kPair) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      const uint32_t held = there >> (slot * kPair);
      const unsigned char* const recs = mine + slot * kPair * kKvRecord;
      load(slot == 0 ? kStages - 1 : slot - 1);   // (read by all lanes before the warp was last together)
      slot = slot + 1 == kStages ? 0 : slot + 1;

      // scores of keys r and r + 8 (h) of each record
      float sc[kCols][kEach][2 * kPair] = {};
      uint32_t vs[2 * kPair][2];   // BF16 scales of V's groups (0, 1) and (2, 3)
#pragma unroll
      for (int j = 0; j < kPair; ++j) {
        const unsigned char* const rec = recs + j * kKvRecord;
        const uint4 k0 = *reinterpret_cast<const uint4*>(rec + lane * 16);
        const uint4 k1 = *reinterpret_cast<const uint4*>(rec + 512 + lane * 16);
        const uint4 s0 = *reinterpret_cast<const uint4*>(rec + kKvScales + r * 16);
        const uint4 s1 = *reinterpret_cast<const uint4*>(rec + kKvScales + 128 + r * 16);
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
        float ks[2][4];
        scales_of(s0.x, ks[0][0], ks[0][1]);
        scales_of(s0.y, ks[0][2], ks[0][3]);
        scales_of(s1.x, ks[1][0], ks[1][1]);
        scales_of(s1.y, ks[1][2], ks[1][3]);
        vs[2 * j][0] = early(s0.z, down[0]);
        vs[2 * j][1] = early(s0.w, down[1]);
        vs[2 * j + 1][0] = early(s1.z, down[0]);
        vs[2 * j + 1][1] = early(s1.w, down[1]);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t a[4], c[4];
          k_pairs(w0[g], wide, near, a);
          k_pairs(w1[g], wide, near, c);
#pragma unroll
          for (int n = 0; n < kCols; ++n) {
            float d[4] = {};
            mma_f16(d, a[0], c[0], a[1], c[1], qf[n][g][0], qf[n][g][1]);
            mma_f16(d, a[2], c[2], a[3], c[3], qf[n][g][2], qf[n][g][3]);
#pragma unroll
            for (int e = 0; e < kEach; ++e)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                sc[n][e][2 * j + h] = fmaf(ks[h][g], d[2 * h + e] + off[n][e][g], sc[n][e][2 * j + h]);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int e = 0; e < kEach; ++e)
#pragma unroll
          for (int i = 0; i < 2 * kPair; ++i) sc[n][e][i] *= factor[n][e];
      // keys that a query does not see; a record without a page has none
      constexpr uint32_t kBoth = (1u << kPair) - 1;
      if ((tile + kPair) * kKvTile > all || (held & kBoth) != kBoth) {
#pragma unroll
        for (int i = 0; i < 2 * kPair; ++i) {
          const int key = tile * kKvTile + r + 8 * i;
          const bool none = !((held >> (i / 2)) & 1);
#pragma unroll
          for (int n = 0; n < kCols; ++n)
#pragma unroll
            for (int e = 0; e < kEach; ++e)
              if (none || key >= limit[n][e]) sc[n][e][i] = -INFINITY;
          // what a token that is not there holds as scales may be anything
          if (none || key >= len) vs[i][0] = vs[i][1] = 0u;
        }
      }
      bool raise = false;
      float most[kCols][kEach];
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          most[n][e] = fmaxf(sc[n][e][0], sc[n][e][1]);
#pragma unroll
          for (int i = 2; i < 2 * kPair; i += 2) most[n][e] = fmax3(most[n][e], sc[n][e][i], sc[n][e][i + 1]);
          raise = raise || most[n][e] > m[n][e] + kSlack;
        }
      uint32_t top[2] = {vs[0][0], vs[0][1]};
#pragma unroll
      for (int i = 1; i < 2 * kPair; ++i)
#pragma unroll
        for (int w = 0; w < 2; ++w) top[w] = larger(top[w], vs[i][w]);
      const uint32_t top_v = larger(late(top[0], down[0]), late(top[1], down[1]));
      raise = raise || (((top_v & 0x7fff7fffu) + 0x3d003d00u) & 0x80008000u) != 0;   // one is 2^7 or more (BF16 0x4300)
      if (__any_sync(0xffffffffu, raise)) {
        float change[4];
        if (kEarly) {   // the scales again, as the record has them, and each group's largest
          top[0] = top[1] = 0u;
#pragma unroll
          for (int i = 0; i < 2 * kPair; ++i) {
            const uint2 two = *reinterpret_cast<const uint2*>(recs + i / 2 * kKvRecord + kKvScales + i % 2 * 128 + r * 16 + 8);
            const bool seen = ((held >> (i / 2)) & 1) && tile * kKvTile + r + 8 * i < len;
            vs[i][0] = seen ? two.x : 0u;
            vs[i][1] = seen ? two.y : 0u;
#pragma unroll
            for (int w = 0; w < 2; ++w) top[w] = larger(top[w], vs[i][w]);
          }
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          uint32_t pair = 0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // 2^(6 - e) for scales below 2^(e + 1); BF16's exponent field is bits 7 to 14
            const uint32_t field = __reduce_max_sync(0xffffffffu, top[w] >> (16 * h + 7) & 0xffu);
            const uint32_t was = down[w] >> (16 * h + 7) & 0xffu, now = min(was, 260 - field);
            pair |= now << (16 * h + 7);
            change[2 * w + h] = __uint_as_float(now << 23) * __uint_as_float((254 - was) << 23);
          }
          down[w] = pair;
#pragma unroll
          for (int i = 0; i < 2 * kPair; ++i) vs[i][w] = early(vs[i][w], pair);
        }
#pragma unroll
        for (int n = 0; n < kCols; ++n)
#pragma unroll
          for (int e = 0; e < kEach; ++e) {
            float top = fmaxf(most[n][e], m[n][e]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float shrink = ex2_approx(m[n][e] - top);
            m[n][e] = top;
            l[n][e] *= shrink;
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (kEach == 1 || (i & 1) == e) acc[g][u][n][i] *= shrink * change[g];
          }
      }
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int e = 0; e < kEach; ++e)
#pragma unroll
          for (int i = 0; i < 2 * kPair; ++i) {
            sc[n][e][i] = ex2_approx(sc[n][e][i] - m[n][e]);
            l[n][e] += sc[n][e][i];
          }
#pragma unroll
      for (int j = 0; j < kPair; ++j) {
        const unsigned char* const rec = recs + j * kKvRecord;
        const uint4 v0 = *reinterpret_cast<const uint4*>(rec + kKvV + lane * 16);
        const uint4 v1 = *reinterpret_cast<const uint4*>(rec + kKvV + 512 + lane * 16);
        float v[2][4];
        scales_of(vs[2 * j][0], v[0][0], v[0][1]);
        scales_of(vs[2 * j][1], v[0][2], v[0][3]);
        scales_of(vs[2 * j + 1][0], v[1][0], v[1][1]);
        scales_of(vs[2 * j + 1][1], v[1][2], v[1][3]);
        if constexpr (!kEarly) {
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            float d[2];
            scales_of(down[w], d[0], d[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              v[h][2 * w] *= d[0];
              v[h][2 * w + 1] *= d[1];
            }
          }
        }
        uint32_t p0[kCols], p1[kCols];   // B operands: keys 0 to 7 and 8 to 15
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint32_t a0 = g < 2 ? v0.x : v0.y, c0 = g < 2 ? v0.z : v0.w, a1 = g < 2 ? v1.x : v1.y, c1 = g < 2 ? v1.z : v1.w;
          uint32_t x[4], y[4];
          v_pairs(__byte_perm(a0, c0, g & 1 ? 0x7632 : 0x5410), low, high, x);
          v_pairs(__byte_perm(a1, c1, g & 1 ? 0x7632 : 0x5410), low, high, y);
          if (kEach == 2 || g % 2 == 0) {
#pragma unroll
            for (int n = 0; n < kCols; ++n) {
              const int g2 = kEach == 1 ? g + 1 : g, i = 2 * j;
              p0[n] = transpose8(pack_f16x2(sc[n][0][i] * v[0][g], sc[n][kEach - 1][i] * v[0][g2]));
              p1[n] = transpose8(pack_f16x2(sc[n][0][i + 1] * v[1][g], sc[n][kEach - 1][i + 1] * v[1][g2]));
            }
          }
#pragma unroll
          for (int n = 0; n < kCols; ++n) {
            mma_f16(acc[g][0][n], x[0], x[1], y[0], y[1], p0[n], p1[n]);
            mma_f16(acc[g][1][n], x[2], x[3], y[2], y[3], p0[n], p1[n]);
          }
        }
      }
    }
    cp_async_wait<0>();
    __syncwarp();

    // the next segment's records are on their way while this one's results leave
    const int done_b = b, done_head = head, done_row0 = row0;
    const bool starts = first == 0, complete = starts && last == tiles;
    if (starts && lane == 0) {
      const long long end = (seg_start + tiles - 1) / share;   // the segment's last item
      p.head[(long long)b * p.segments + seg] = make_int2(item, (int)(end - item) + 1);
    }
    more = begin();
    float up[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) up[g] = __uint_as_float((254 - (down[g / 2] >> (16 * (g % 2) + 7) & 0xffu)) << 23) * kPart;
#pragma unroll
    for (int n = 0; n < kCols; ++n)
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], o);
        const int in_tile = 8 * n + kEach * t + e, row = done_row0 + in_tile;
        if (row >= p.rows) continue;
        float4 v[4];   // of channels 32 g + 4 r and the next three
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int c = kEach == 1 ? g & 1 : e;
          v[g] = make_float4(acc[g][0][n][c] * up[g], acc[g][0][n][2 + c] * up[g], acc[g][1][n][c] * up[g],
                             acc[g][1][n][2 + c] * up[g]);
        }
        if (!complete) {
          const long long piece = (2ll * item + starts) * kRows + in_tile;
#pragma unroll
          for (int g = 0; g < 4; ++g) reinterpret_cast<float4*>(p.part_o + piece * kDim)[8 * g + r] = v[g];
          if (r == 0) p.part_ml[piece] = make_float2(m[n][e], l[n][e]);
          continue;
        }
        const int s = div_by(row, p.G), h = done_head * (int)p.G.d + row - s * (int)p.G.d;
        const float inv = l[n][e] == 0.0f ? 0.0f : 1.0f / (l[n][e] * kPart);   // (a NaN stays one, here and in lse)
        uint2* const o = reinterpret_cast<uint2*>(p.o + done_b * p.o_str[0] + s * p.o_str[1] + h * p.o_str[2]);
#pragma unroll
        for (int g = 0; g < 4; ++g)
          o[8 * g + r] = make_uint2(pack_bf16x2(v[g].x * inv, v[g].y * inv), pack_bf16x2(v[g].z * inv, v[g].w * inv));
        if (r == 0)
          p.lse[((long long)done_b * p.Hq + h) * p.S + s] =
              l[n][e] == 0.0f ? -INFINITY : (m[n][e] + log2f(l[n][e])) * 0.6931471805599453f;
      }
  }
}

// A row of a segment in several items: its pieces, in order.
template <int kRows>
__global__ void __launch_bounds__(256) kv4_join_kernel(const __grid_constant__ AttnParams p) {
  __shared__ float4 sums[8][32];
  __shared__ float2 mls[8];
  griddep_wait();
  const int b = div_by((int)blockIdx.x, p.by_segments), seg = (int)blockIdx.x - b * p.segments;
  if (tokens_of(p, b) == 0) return;
  const int2 what = p.head[blockIdx.x];   // first item, pieces
  if (what.y <= 1) return;
  const int head = div_by(seg, p.by_row_tiles), row0 = (seg - head * p.row_tiles) * kRows;
  const int row = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (row0 + row >= p.rows) return;
  // (the first item's piece is its second: it may have another segment's end before)
  auto place = [&](int i) { return (2ll * (what.x + i) + (i == 0)) * kRows + row; };
  float m = kNone, l = 0.0f;
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  constexpr int kTogether = 4;
  for (int i0 = warp; i0 < what.y; i0 += 8 * kTogether) {
    float2 ml[kTogether];
    float4 v[kTogether];
#pragma unroll
    for (int u = 0; u < kTogether; ++u) {
      const int i = i0 + 8 * u;
      ml[u] = i < what.y ? p.part_ml[place(i)] : make_float2(kNone, 0.0f);
      v[u] = i < what.y ? reinterpret_cast<const float4*>(p.part_o + place(i) * kDim)[lane] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll
    for (int u = 0; u < kTogether; ++u) {
      const float top = fmaxf(m, ml[u].x), fm = ex2_approx(m - top), f = ex2_approx(ml[u].x - top);
      m = top;
      l = fmaf(l, fm, f * ml[u].y);
      sum = make_float4(fmaf(sum.x, fm, f * v[u].x), fmaf(sum.y, fm, f * v[u].y), fmaf(sum.z, fm, f * v[u].z),
                        fmaf(sum.w, fm, f * v[u].w));
    }
  }
  sums[warp][lane] = sum;
  if (lane == 0) mls[warp] = make_float2(m, l);
  __syncthreads();
  if (warp != 0) return;
  m = kNone;
  l = 0.0f;
  sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int w = 0; w < 8; ++w) m = fmaxf(m, mls[w].x);
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const float f = ex2_approx(mls[w].x - m);
    const float4 v = sums[w][lane];
    l = fmaf(f, mls[w].y, l);
    sum = make_float4(fmaf(f, v.x, sum.x), fmaf(f, v.y, sum.y), fmaf(f, v.z, sum.z), fmaf(f, v.w, sum.w));
  }
  const int s = div_by(row0 + row, p.G), h = head * (int)p.G.d + row0 + row - s * (int)p.G.d;
  const float inv = l == 0.0f ? 0.0f : 1.0f / (l * kPart);
  reinterpret_cast<uint2*>(p.o + b * p.o_str[0] + s * p.o_str[1] + h * p.o_str[2])[lane] =
      make_uint2(pack_bf16x2(sum.x * inv, sum.y * inv), pack_bf16x2(sum.z * inv, sum.w * inv));
  if (lane == 0)
    p.lse[((long long)b * p.Hq + h) * p.S + s] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Queries of a segment, tiles of them, and CTAs.
struct Grid {
  int rows, row_tiles, ctas;
  size_t segments, items;   // of all requests
};
Grid grid_of(int B, int S, int Hq, int Hkv, int max_pages, int page_size) {
  Grid g;
  const long long rows = (long long)S * (Hq / Hkv);
  g.rows = rows <= 4 ? 4 : rows <= 8 ? 8 : 16;
  g.row_tiles = (int)((rows + g.rows - 1) / g.rows);
  g.segments = (size_t)B * Hkv * g.row_tiles;
  // no more CTAs than the cache could give items to
  const double most = ((double)max_pages * (page_size / kKvTile) + kStart) * (double)g.segments / kLeast + 1.0;
  g.ctas = most < kCtas ? (int)most : kCtas;
  g.items = (size_t)g.ctas * warps(g.rows);
  return g;
}

template <int kRows>
cudaError_t launch_both(const AttnParams& p, const Grid& g, cudaStream_t stream) {
  constexpr int kShared = warps(kRows) * kRing;
  static ContextOnce attr_done;
  cudaError_t e = attr_done.run([] {
    return cudaFuncSetAttribute(kv4_attn_kernel<kRows>, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared);
  });
  if (e == cudaSuccess)
    e = launch_dependent(kv4_attn_kernel<kRows>, dim3((unsigned)g.ctas), 32 * warps(kRows), kShared, stream, p);
  if (e != cudaSuccess) return e;
  return launch_dependent(kv4_join_kernel<kRows>, dim3((unsigned)g.segments, kRows), 256, 0, stream, p);
}

}  // namespace

size_t attn_kv4_workspace(int B, int S, int Hq, int Hkv, int max_pages, int page_size) {
  const Grid g = grid_of(B, S, Hq, Hkv, max_pages, page_size);
  return (g.segments * sizeof(int2) + 15) / 16 * 16 + g.items * 2 * g.rows * (kDim * sizeof(float) + sizeof(float2));
}

cudaError_t launch_attn_kv4(const Kv4Args& a, void* workspace, cudaStream_t stream) {
  const Grid g = grid_of(a.B, a.S, a.Hq, a.Hkv, a.max_pages, a.page_size);
  AttnParams p;
  p.pages = kv4_pages(a);
  p.q = reinterpret_cast<const __nv_bfloat16*>(a.q);
  p.o = reinterpret_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.kv_len = a.kv_len;
  for (int i = 0; i < 3; ++i) {
    p.q_str[i] = a.q_str[i];
    p.o_str[i] = a.o_str[i];
  }
  p.B = a.B;
  p.S = a.S;
  p.Hq = a.Hq;
  p.rows = a.S * (a.Hq / a.Hkv);
  p.row_tiles = g.row_tiles;
  p.segments = g.row_tiles * a.Hkv;
  const long long capacity = (long long)a.max_pages * a.page_size;
  p.capacity = a.num_pages > 0 ? (int)capacity : 0;   // (at most 2^30)
  p.G = make_div(a.Hq / a.Hkv);
  p.by_row_tiles = make_div(g.row_tiles);
  p.causal = a.causal;
  p.c_log2 = a.c_log2;
  p.by_segments = make_div(p.segments);
  p.ctas = g.ctas;
  p.head = reinterpret_cast<int2*>(workspace);
  p.part_o = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + (g.segments * sizeof(int2) + 15) / 16 * 16);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + g.items * 2 * g.rows * kDim);
  switch (g.rows) {
    case 4: return launch_both<4>(p, g, stream);
    case 8: return launch_both<8>(p, g, stream);
    default: return launch_both<16>(p, g, stream);
  }
}

}  // namespace sa
