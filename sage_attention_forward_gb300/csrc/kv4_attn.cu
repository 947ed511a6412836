// Attention over a K/V cache in 4 bits, sm_103a: O = softmax(scale q K^T) V for one or a few queries of each request.
//
// Bound by memory: 144 bytes of cache a token and key head, read once for all queries that share the head.
//
// Products.  Keys (and V's channels) are the rows of mma.m16n8k16, the queries of a key head (tokens x heads that share it)
// its columns, eight at a time: with few queries no part of a product is empty.  Codes become matrix operands without a
// conversion: four bits put into the mantissa of a constant are the value constant + code (FP16 256 + c and 16 + c for K, BF16
// 16 + c for V; one shift and one masked insert for two values).  What the constants add is taken off exactly: for K the
// accumulators start at -(constant + 8) q summed over the channels, a product of the same operands; for V a product with
// rows of 24s gives 24 sum p for each group of channels.
//   S^T = sum_g scale_K[key, g] (codes_g q_g)        four products of 32 channels, scaled in FP32
//   O^T[group g] = sum_j codes (p_j scale_V[j, g])   P is scaled for each group in FP32, then rounded to BF16 once
// Q becomes FP16 with its row's largest magnitude in [1, 2): its own 8 bits stay (below 2^-24 of that magnitude they round).
//
// Work.  The records of all requests and heads are one line of work; each CTA takes an equal share of it, found from the
// lengths on the device, so that ragged batches are balanced and a graph serves any lengths.  A CTA's warps take its
// records in turn, each through its own ring of cp.async copies, with a softmax of its own; they are joined in shared memory,
// and pieces of a request's head that several CTAs share by a second kernel, in a fixed order.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kv4.cuh"
#include "pieces.cuh"

namespace sa {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kStages = 4;
constexpr int kLeast = 4;           // records a CTA takes at least
constexpr float kSlack = 8.0f;      // a row's reference maximum is raised when one passes it by more (log2 units)
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
  Div G, by_row_tiles;
  int causal;
  float c_log2;
  // workspace: joined pieces, [CTA][2][rows of a tile]
  float* part_o;
  float2* part_ml;
  int4* head;                       // [CTA]: request, segment, pieces of the segment that starts here (0: none)
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
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
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit values, a row to four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// (x & mask) | bits
template <uint32_t kMask, uint32_t kBits>
__device__ __forceinline__ uint32_t insert(uint32_t x) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "n"(kMask), "n"(kBits));
  return y;
}
// K: eight codes as FP16 pairs (i, i + 4): 256 + c for i = 0 and 2, 16 + c for i = 1 and 3.
__device__ __forceinline__ void k_pairs(uint32_t w, uint32_t (&a)[4]) {
  const uint32_t x = w << 2, y = w >> 6;
  a[0] = insert<0x003c003cu, 0x5c005c00u>(x);
  a[1] = insert<0x03c003c0u, 0x4c004c00u>(x);
  a[2] = insert<0x003c003cu, 0x5c005c00u>(y);
  a[3] = insert<0x03c003c0u, 0x4c004c00u>(y);
}
// V: four codes of each of two tokens as BF16 pairs 16 + c.
__device__ __forceinline__ void v_pairs(uint32_t x, uint32_t (&a)[4]) {
  a[0] = insert<0x00780078u, 0x41804180u>(x << 3);
  a[1] = insert<0x00780078u, 0x41804180u>(x >> 1);
  a[2] = insert<0x00780078u, 0x41804180u>(x >> 5);
  a[3] = insert<0x00780078u, 0x41804180u>(x >> 9);
}
__device__ __forceinline__ void scales_of(uint32_t w, float& a, float& b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}

__device__ __forceinline__ int tokens_of(const AttnParams& p, int b) { return min(max(__ldg(p.kv_len + b), 0), p.capacity); }

// The line of work: request b's records, once for each of its segments.
struct Line {
  long long total, share;   // records, and those of a CTA
};
// Sums v over the CTA's threads up to and including this one; total: all of them.
__device__ __forceinline__ long long scan(long long v, long long* warp_sums, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) v += warp_sums[w];
    total += warp_sums[w];
  }
  return v;
}

template <int kCols>   // columns of eight queries
struct Tile {
  float o[4][2][kCols][4];   // [group][pair of channel rows][column]: O^T
  float sum[kCols][4];       // 24 sum p scale of group r (the lane's row) for the lane's two queries
  float m[kCols][2], l[kCols][2];
};

template <int kCols>
__global__ void __launch_bounds__(kThreads, kCols == 1 ? 3 : 2) kv4_attn_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kRows = 8 * kCols;
  constexpr int kRing = kStages * kKvRecord;
  constexpr int kJoin = (kRows * kDim + 2 * kRows) * 4;   // a warp's O, m and l
  __shared__ __align__(16) unsigned char ring[kWarps][kRing > kJoin ? kRing : kJoin];
  __shared__ long long warp_sums[kWarps];
  __shared__ long long s_before;
  __shared__ int s_b;
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, t = lane & 3;

  // the CTA's share of the line
  long long total = 0, before = 0;
  const int b0 = threadIdx.x;
  auto work_of = [&](int b) { return b < p.B ? (long long)((tokens_of(p, b) + kKvTile - 1) / kKvTile) * p.segments : 0ll; };
  long long first_scan = scan(work_of(b0), warp_sums, total);
  for (int c = kThreads; c < p.B; c += kThreads) {
    long long more;
    scan(work_of(c + threadIdx.x), warp_sums, more);
    total += more;
  }
  const long long share = max((long long)kLeast, (total + gridDim.x - 1) / gridDim.x);
  long long at = blockIdx.x * share;
  const long long stop = min(at + share, total);
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
  if (threadIdx.x == 0) p.head[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (at >= stop) return;
  // the request that `at` is in
  for (int c = 0; c < p.B; c += kThreads) {
    long long sum = 0;
    const long long mine = work_of(c + threadIdx.x);
    const long long incl = before + (c == 0 ? first_scan : scan(mine, warp_sums, sum));
    if (at >= incl - mine && at < incl) {
      s_b = c + threadIdx.x;
      s_before = incl - mine;
    }
    if (c == 0) scan(mine, warp_sums, sum);
    before += sum;
    __syncthreads();
    if (at < before) break;
  }
  __syncthreads();
  int b = s_b;
  before = s_before;

  while (at < stop) {
    const int len = tokens_of(p, b), tiles = (len + kKvTile - 1) / kKvTile;
    const long long whole = (long long)tiles * p.segments;
    if (at >= before + whole) {   // the next request
      before += whole;
      ++b;
      continue;
    }
    const int seg = (int)((at - before) / tiles);
    const long long seg_start = before + (long long)seg * tiles;
    const int lo = (int)(at - seg_start), hi = (int)min((long long)tiles, stop - seg_start);
    const int head = div_by(seg, p.by_row_tiles), row0 = (seg - head * p.row_tiles) * kRows;
    at = seg_start + hi;

    // queries: B operands of K's products, and the constants' part of them
    uint32_t qf[kCols][4][4];
    float off[kCols][4][2], factor[kCols][2];
    int limit[kCols][2], all = len;   // keys before `all` are seen by every query of the tile
#pragma unroll
    for (int n = 0; n < kCols; ++n) {
      const int row = row0 + 8 * n + r;
      const int s = div_by(row, p.G), g0 = row - s * (int)p.G.d;
      uint4 raw[4] = {};
      if (row < p.rows) {
        const uint4* const src = reinterpret_cast<const uint4*>(p.q + b * p.q_str[0] + s * p.q_str[1] +
                                                                (long long)(head * (int)p.G.d + g0) * p.q_str[2]);
#pragma unroll
        for (int g = 0; g < 4; ++g) raw[g] = __ldg(src + 4 * g + t);
      }
      float top = 0.0f;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint32_t w[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x, y;
          scales_of(w[i], x, y);
          top = fmaxf(top, fmaxf(fabsf(x), fabsf(y)));
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = min(max((int)(__float_as_uint(top) >> 23), 27), 253);
      const float down = __uint_as_float((uint32_t)(254 - e) << 23);
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
        off[n][g][0] = d[0];
        off[n][g][1] = d[1];
      }
      const float up = __uint_as_float((uint32_t)e << 23) * p.c_log2;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = 2 * t + c, at_row = row0 + 8 * n + col;
        factor[n][c] = __shfl_sync(0xffffffffu, up, col * 4);
        const int tok = div_by(at_row, p.G);
        limit[n][c] = p.causal ? min(len, len - p.S + tok + 1) : len;
      }
    }
    if (p.causal) all = max(0, min(len, len - p.S + div_by(row0, p.G) + 1));

    Tile<kCols> acc = {};
#pragma unroll
    for (int n = 0; n < kCols; ++n) acc.m[n][0] = acc.m[n][1] = -INFINITY;

    // the warp's records: lo + warp, and every kWarps-th from there
    unsigned char* const mine = ring[warp];
    uint32_t there = 0;                               // bit of a slot: its record has a page
    int to_load = lo + warp;
    int page = to_load < hi ? kv_page(p.pages, b, to_load) : -1;
    auto load = [&](int slot) {
      there &= ~(1u << slot);
      if (to_load < hi) {
        if (page >= 0) {
          there |= 1u << slot;
          const unsigned char* const from = kv_record(p.pages, page, head, to_load);
#pragma unroll
          for (int i = 0; i < 5; ++i)
            if (i < 4 || lane < 16) cp_async16(mine + slot * kKvRecord + (lane + 32 * i) * 16, from + (lane + 32 * i) * 16);
        }
        to_load += kWarps;
        if (to_load < hi) page = kv_page(p.pages, b, to_load);
      }
      cp_async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) load(i);

    int slot = 0;
    for (int tile = lo + warp; tile < hi; tile += kWarps) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      const bool held = (there >> slot) & 1;
      const unsigned char* const rec = mine + slot * kKvRecord;
      const int into = slot == 0 ? kStages - 1 : slot - 1;
      slot = slot + 1 == kStages ? 0 : slot + 1;
      if (!held) {   // no page: its keys are not there
        load(into);
        continue;
      }
      const uint4 k0 = *reinterpret_cast<const uint4*>(rec + lane * 16), k1 = *reinterpret_cast<const uint4*>(rec + 512 + lane * 16);
      const uint4 s0 = *reinterpret_cast<const uint4*>(rec + kKvScales + r * 16);
      const uint4 s1 = *reinterpret_cast<const uint4*>(rec + kKvScales + 128 + r * 16);
      load(into);   // (read by all lanes before the warp was last together)

      // scores
      float sc[kCols][4] = {};
      {
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
        float ks[2][4];
        scales_of(s0.x, ks[0][0], ks[0][1]);
        scales_of(s0.y, ks[0][2], ks[0][3]);
        scales_of(s1.x, ks[1][0], ks[1][1]);
        scales_of(s1.y, ks[1][2], ks[1][3]);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t a[4], c[4];
          k_pairs(w0[g], a);
          k_pairs(w1[g], c);
#pragma unroll
          for (int n = 0; n < kCols; ++n) {
            float d[4] = {off[n][g][0], off[n][g][1], off[n][g][0], off[n][g][1]};
            mma_f16(d, a[0], c[0], a[1], c[1], qf[n][g][0], qf[n][g][1]);
            mma_f16(d, a[2], c[2], a[3], c[3], qf[n][g][2], qf[n][g][3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[n][i] = fmaf(ks[i >> 1][g], d[i], sc[n][i]);
          }
        }
      }
      const bool edge = (tile + 1) * kKvTile > all;
      bool raise = false;
#pragma unroll
      for (int n = 0; n < kCols; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sc[n][i] *= factor[n][i & 1];
          if (edge && tile * kKvTile + r + 8 * (i >> 1) >= limit[n][i & 1]) sc[n][i] = -INFINITY;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) raise = raise || fmaxf(sc[n][c], sc[n][2 + c]) > acc.m[n][c] + kSlack;
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int n = 0; n < kCols; ++n) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float top = fmaxf(fmaxf(sc[n][c], sc[n][2 + c]), acc.m[n][c]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float shrink = top == -INFINITY ? 1.0f : ex2_approx(acc.m[n][c] - top);
            acc.m[n][c] = top;
            acc.l[n][c] *= shrink;
#pragma unroll
            for (int i = c; i < 4; i += 2) {
              acc.sum[n][i] *= shrink;
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                acc.o[g][0][n][i] *= shrink;
                acc.o[g][1][n][i] *= shrink;
              }
            }
          }
        }
      }
      const uint4 v0 = *reinterpret_cast<const uint4*>(rec + kKvV + lane * 16);
      const uint4 v1 = *reinterpret_cast<const uint4*>(rec + kKvV + 512 + lane * 16);
#pragma unroll
      for (int n = 0; n < kCols; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float m = acc.m[n][i & 1];
          sc[n][i] = ex2_approx(sc[n][i] - (m == -INFINITY ? 0.0f : m));
          acc.l[n][i & 1] += sc[n][i];
        }
      }
      // what a token without a key holds as scales may be anything
      float vs[2][4];
      scales_of(s0.z, vs[0][0], vs[0][1]);
      scales_of(s0.w, vs[0][2], vs[0][3]);
      scales_of(s1.z, vs[1][0], vs[1][1]);
      scales_of(s1.w, vs[1][2], vs[1][3]);
      if (edge) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (tile * kKvTile + r + 8 * h >= len)
#pragma unroll
            for (int g = 0; g < 4; ++g) vs[h][g] = 0.0f;
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint32_t a0 = g < 2 ? v0.x : v0.y, c0 = g < 2 ? v0.z : v0.w, a1 = g < 2 ? v1.x : v1.y, c1 = g < 2 ? v1.z : v1.w;
        uint32_t x[4], y[4];
        v_pairs(__byte_perm(a0, c0, g & 1 ? 0x7632 : 0x5410), x);
        v_pairs(__byte_perm(a1, c1, g & 1 ? 0x7632 : 0x5410), y);
        const uint32_t ones = r == g ? 0x41c041c0u : 0u;   // 24 in row g
#pragma unroll
        for (int n = 0; n < kCols; ++n) {
          const uint32_t p0 = transpose8(pack_bf16x2(sc[n][0] * vs[0][g], sc[n][1] * vs[0][g]));
          const uint32_t p1 = transpose8(pack_bf16x2(sc[n][2] * vs[1][g], sc[n][3] * vs[1][g]));
          mma_bf16(acc.o[g][0][n], x[0], x[1], y[0], y[1], p0, p1);
          mma_bf16(acc.o[g][1][n], x[2], x[3], y[2], y[3], p0, p1);
          mma_bf16(acc.sum[n], ones, 0u, ones, 0u, p0, p1);
        }
      }
    }
    cp_async_wait<0>();
    __syncwarp();

    // the warps' results, joined
    float* const mo = reinterpret_cast<float*>(mine);              // [kRows][kDim], then m and l
    float2* const ml = reinterpret_cast<float2*>(mo + kRows * kDim);
#pragma unroll
    for (int n = 0; n < kCols; ++n) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float l = acc.l[n][c];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        const int col = 8 * n + 2 * t + c;
        if (r == 0) ml[col] = make_float2(acc.m[n][c], l);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float sum = __shfl_sync(0xffffffffu, acc.sum[n][c], 4 * g + t);
#pragma unroll
          for (int u = 0; u < 2; ++u)
            *reinterpret_cast<float2*>(mo + col * kDim + 32 * g + 4 * r + 2 * u) =
                make_float2(acc.o[g][u][n][c] - sum, acc.o[g][u][n][2 + c] - sum);
        }
      }
    }
    __syncthreads();
    const bool complete = lo == 0 && hi == tiles;
    const int piece = 2 * blockIdx.x + (lo == 0);
    if (!complete && lo == 0 && threadIdx.x == 0) {
      const long long last = seg_start + tiles - 1;
      p.head[blockIdx.x] = make_int4(b, seg, (int)(last / share - blockIdx.x) + 1, 0);
    }
    // a warp takes a row: four channels a lane
    for (int row = warp; row < kRows && row0 + row < p.rows; row += kWarps) {
      float m = -INFINITY, l = 0.0f;
      float2 each[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        each[w] = reinterpret_cast<const float2*>(reinterpret_cast<const float*>(ring[w]) + kRows * kDim)[row];
        m = fmaxf(m, each[w].x);
      }
      float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = each[w].x == -INFINITY ? 0.0f : ex2_approx(each[w].x - m);
        const float4 v = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(ring[w]) + row * kDim)[lane];
        l = fmaf(f, each[w].y, l);
        sum = make_float4(fmaf(f, v.x, sum.x), fmaf(f, v.y, sum.y), fmaf(f, v.z, sum.z), fmaf(f, v.w, sum.w));
      }
      if (!complete) {
        reinterpret_cast<float4*>(p.part_o + ((long long)piece * kRows + row) * kDim)[lane] = sum;
        if (lane == 0) p.part_ml[(long long)piece * kRows + row] = make_float2(m, l);
        continue;
      }
      const int s = div_by(row0 + row, p.G), h = head * (int)p.G.d + row0 + row - s * (int)p.G.d;
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
      reinterpret_cast<uint2*>(p.o + b * p.o_str[0] + s * p.o_str[1] + h * p.o_str[2])[lane] =
          make_uint2(pack_bf16x2(sum.x * inv, sum.y * inv), pack_bf16x2(sum.z * inv, sum.w * inv));
      if (lane == 0)
        p.lse[((long long)b * p.Hq + h) * p.S + s] = l > 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
    __syncthreads();   // before the rings are filled again
  }
}

// Segments that several CTAs share: a row's pieces, the CTAs' one after another.
template <int kRows>
__global__ void __launch_bounds__(256) kv4_join_kernel(const __grid_constant__ AttnParams p) {
  __shared__ float4 sums[8][32];
  __shared__ float2 mls[8];
  griddep_wait();
  const int4 what = p.head[blockIdx.x];
  if (what.z == 0) return;
  const int b = what.x, head = div_by(what.y, p.by_row_tiles), row0 = (what.y - head * p.row_tiles) * kRows;
  const int row = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (row0 + row >= p.rows) return;
  // (the first CTA's piece is its second: it may have another segment's end before)
  auto place = [&](int i) { return (2ll * (blockIdx.x + i) + (i == 0)) * kRows + row; };
  float m = -INFINITY, l = 0.0f;
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  constexpr int kTogether = 4;
  for (int i0 = warp; i0 < what.z; i0 += 8 * kTogether) {
    float2 ml[kTogether];
    float4 v[kTogether];
#pragma unroll
    for (int u = 0; u < kTogether; ++u) {
      const int i = i0 + 8 * u;
      ml[u] = i < what.z ? p.part_ml[place(i)] : make_float2(-INFINITY, 0.0f);
      v[u] = i < what.z ? reinterpret_cast<const float4*>(p.part_o + place(i) * kDim)[lane] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll
    for (int u = 0; u < kTogether; ++u) {
      if (ml[u].x == -INFINITY) continue;
      const float top = fmaxf(m, ml[u].x), fm = m == -INFINITY ? 0.0f : ex2_approx(m - top), f = ex2_approx(ml[u].x - top);
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
  m = -INFINITY;
  l = 0.0f;
  sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int w = 0; w < 8; ++w) m = fmaxf(m, mls[w].x);
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const float f = mls[w].x == -INFINITY ? 0.0f : ex2_approx(mls[w].x - m);
    const float4 v = sums[w][lane];
    l = fmaf(f, mls[w].y, l);
    sum = make_float4(fmaf(f, v.x, sum.x), fmaf(f, v.y, sum.y), fmaf(f, v.z, sum.z), fmaf(f, v.w, sum.w));
  }
  const int s = div_by(row0 + row, p.G), h = head * (int)p.G.d + row0 + row - s * (int)p.G.d;
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  reinterpret_cast<uint2*>(p.o + b * p.o_str[0] + s * p.o_str[1] + h * p.o_str[2])[lane] =
      make_uint2(pack_bf16x2(sum.x * inv, sum.y * inv), pack_bf16x2(sum.z * inv, sum.w * inv));
  if (lane == 0)
    p.lse[((long long)b * p.Hq + h) * p.S + s] = l > 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// Columns of eight queries a CTA works on, and CTAs.
struct Grid {
  int cols, row_tiles, ctas;
};
Grid grid_of(int B, int S, int Hq, int Hkv, int max_pages, int page_size) {
  Grid g;
  const long long rows = (long long)S * (Hq / Hkv);
  g.cols = rows <= 8 ? 1 : 2;
  g.row_tiles = (int)((rows + 8 * g.cols - 1) / (8 * g.cols));
  // no more CTAs than the cache could give work to
  const double most = (double)max_pages * (page_size / kKvTile) * B * Hkv * g.row_tiles / kLeast + 1.0;
  const int fit = 152 * (g.cols == 1 ? 3 : 2);
  g.ctas = most < fit ? (int)most : fit;
  return g;
}

}  // namespace

size_t attn_kv4_workspace(int B, int S, int Hq, int Hkv, int max_pages, int page_size) {
  const Grid g = grid_of(B, S, Hq, Hkv, max_pages, page_size);
  return (size_t)g.ctas * (16 + 2 * 8 * g.cols * (kDim * 4 + 8));
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
  p.capacity = capacity < (1ll << 30) ? (int)capacity : 1 << 30;
  p.G = make_div(a.Hq / a.Hkv);
  p.by_row_tiles = make_div(g.row_tiles);
  p.causal = a.causal;
  p.c_log2 = a.c_log2;
  p.head = reinterpret_cast<int4*>(workspace);
  p.part_o = reinterpret_cast<float*>(p.head + g.ctas);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + (size_t)g.ctas * 2 * 8 * g.cols * kDim);
  cudaError_t e = g.cols == 1 ? launch_dependent(kv4_attn_kernel<1>, dim3((unsigned)g.ctas), kThreads, 0, stream, p)
                              : launch_dependent(kv4_attn_kernel<2>, dim3((unsigned)g.ctas), kThreads, 0, stream, p);
  if (e != cudaSuccess) return e;
  return g.cols == 1 ? launch_dependent(kv4_join_kernel<8>, dim3((unsigned)g.ctas, 8), 256, 0, stream, p)
                     : launch_dependent(kv4_join_kernel<16>, dim3((unsigned)g.ctas, 16), 256, 0, stream, p);
}

}  // namespace sa
