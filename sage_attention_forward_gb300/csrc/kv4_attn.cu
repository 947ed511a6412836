// Attention over a K/V cache in 4 bits, sm_103a: O = softmax(scale q K^T) V for one or a few queries of each request.
//
// Bound by memory: 144 bytes of cache a token and key head, read once for all queries that share the head.
//
// Products.  Keys (and V's channels) are the rows of the mma, the queries of a key head (tokens x heads that share it) its
// columns: with few queries no part of a product is empty, and each code is unpacked once for all of them.
//   S^T = sum_g scale_K[key, g] (codes_g q_g)        m16n8k32 in e4m3, one for each 32 channels, scaled in FP32
//   O^T[group g] = sum_j codes (p_j scale_V[j, g])   m16n8k16 in BF16; P is scaled for each group in FP32, then rounded once
// A 4-bit code in the low half of a byte is the e4m3 value code / 512, subnormal or not: K's codes become operands by a mask
// and a shift, eight of them at a time.  Q, scaled so that its row's largest magnitude is in [128, 256), is the sum of two
// e4m3 terms, 4 bits of it and the 4 bits below (kept 32 times as large); the terms are neighbouring columns, so that a lane has
// both parts of its scores.  What is below 2^-16 of the row's largest magnitude rounds.  The codes' bias of 8 is taken off by
// accumulators that start at -8 q summed over the channels, a product of the same operands.  V's codes are put into the
// mantissa of BF16 128 and 136 subtracted, exactly.
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
constexpr float kLow = 32.0f;       // Q's second term is kept this much larger
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
// d = a b + (c0, c1) for both of a lane's rows
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, float c0, float c1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %10, %11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
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
// V: four codes of each of two tokens, 4 bits each in halves of x, as BF16 pairs of code - 8.
__device__ __forceinline__ void v_pairs(uint32_t x, uint32_t (&a)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t y;
    asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xEA;" : "=r"(y) : "r"(x >> (4 * i)));   // (x & mask) | 128
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(a[i]) : "r"(y), "r"(0x3f803f80u), "r"(0xc308c308u));   // y - 136
  }
}
// Two values as e4m3 (a in the low byte), and back.
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
  unsigned short d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(b), "f"(a));
  return d;
}
__device__ __forceinline__ float2 of_e4m3_pair(uint32_t d) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)d));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ void scales_of(uint32_t w, float& a, float& b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}

__device__ __forceinline__ int tokens_of(const AttnParams& p, int b) { return min(max(__ldg(p.kv_len + b), 0), p.capacity); }

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

// kFours: queries of a CTA, four at a time (1, 2 or 4).
template <int kFours>
__global__ void __launch_bounds__(kThreads, kFours == 1 ? 4 : kFours == 2 ? 3 : 2) kv4_attn_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kRows = 4 * kFours;
  constexpr int kCols = (kFours + 1) / 2;                  // columns of eight in the product with V
  constexpr int kRing = kStages * kKvRecord;
  constexpr int kJoin = (kRows * kDim + 2 * kRows) * 4;    // a warp's O, m and l
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

    // queries: the column of this lane holds one of two terms of query r / 2 (of each four)
    uint32_t qf[kFours][4][2];
    float off[kFours][4][2], factor[kFours];
    int limit[kFours], all = len;   // keys before `all` are seen by every query of the tile
#pragma unroll
    for (int n = 0; n < kFours; ++n) {
      const int row = row0 + 4 * n + (r >> 1);
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
        float x[8];
        unpack<__nv_bfloat16>(raw[g], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = max((int)(__float_as_uint(top) >> 23), 27);
      const float to = __uint_as_float((uint32_t)(261 - e) << 23);   // 2^7 over the power of two in `top`
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float x[8];
        unpack<__nv_bfloat16>(raw[g], x);
        uint32_t term[4];   // of channels (0, 2), (4, 6), (1, 3), (5, 7)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = 4 * (i & 1) + (i >> 1);
          const float u = x[c] * to, v = x[c + 2] * to;
          term[i] = e4m3_pair(u, v);
          const float2 high = of_e4m3_pair(term[i]);
          if (r & 1) term[i] = e4m3_pair((u - high.x) * kLow, (v - high.y) * kLow);
        }
        qf[n][g][0] = term[0] | term[1] << 16;
        qf[n][g][1] = term[2] | term[3] << 16;
        float d[4];
        mma_e4m3(d, 0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u, qf[n][g][0], qf[n][g][1], 0.0f, 0.0f);   // -8 / 512
        off[n][g][0] = d[0];
        off[n][g][1] = d[1];
      }
      // (codes are 1 / 512 of themselves, q 2^7 over its power of two)
      const float up = __uint_as_float((uint32_t)e << 23) * (4.0f * p.c_log2);
      factor[n] = __shfl_sync(0xffffffffu, up, 8 * t);
      const int tok = div_by(row0 + 4 * n + t, p.G);
      limit[n] = p.causal ? min(len, len - p.S + tok + 1) : len;
    }
    if (p.causal) all = max(0, min(len, len - p.S + div_by(row0, p.G) + 1));

    // [group][pair of channel rows][column]; kFours = 1: columns 2 t and 2 t + 1 are query t with the scales of an even
    // and of an odd group, one of which counts; else queries t and t + 4 of eight
    float acc[4][2][kCols][4] = {};
    float m[kFours], l[kFours];
#pragma unroll
    for (int n = 0; n < kFours; ++n) {
      m[n] = -INFINITY;
      l[n] = 0.0f;
    }

    // the warp's records, one after another: [first, last)
    const int first = lo + (int)((long long)(hi - lo) * warp / kWarps);
    const int last = lo + (int)((long long)(hi - lo) * (warp + 1) / kWarps);
    unsigned char* const mine = ring[warp];
    uint32_t there = 0;                               // bit of a slot: its record has a page
    int to_load = first, left = 0, page = -1;         // left: records of the current page
    const unsigned char* from = nullptr;
    int next = first < last ? kv_page(p.pages, b, first) : -1;
    auto load = [&](int slot) {
      if (to_load < last) {
        if (left == 0) {
          page = next;
          left = (int)p.pages.tiles.d - (to_load - div_by(to_load, p.pages.tiles) * (int)p.pages.tiles.d);
          if (page >= 0) from = kv_record(p.pages, page, head, to_load) + lane * 16;
          if (to_load + left < last) next = kv_page(p.pages, b, to_load + left);
        }
        there &= ~(1u << slot);
        if (page >= 0) {
          there |= 1u << slot;
          unsigned char* const into = mine + slot * kKvRecord + lane * 16;
#pragma unroll
          for (int i = 0; i < 5; ++i)
            if (i < 4 || lane < 16) cp_async16(into + i * 512, from + i * 512);
          from += kKvRecord;
        }
        ++to_load;
        --left;
      }
      cp_async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) load(i);

    int slot = 0;
#pragma unroll 1
    for (int tile = first; tile < last; ++tile) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      const bool held = (there >> slot) & 1;
      const unsigned char* const rec = mine + slot * kKvRecord;
      load(slot == 0 ? kStages - 1 : slot - 1);   // (read by all lanes before the warp was last together)
      slot = slot + 1 == kStages ? 0 : slot + 1;
      if (!held) continue;   // no page: its keys are not there
      const uint4 k0 = *reinterpret_cast<const uint4*>(rec + lane * 16), k1 = *reinterpret_cast<const uint4*>(rec + 512 + lane * 16);
      const uint4 s0 = *reinterpret_cast<const uint4*>(rec + kKvScales + r * 16);
      const uint4 s1 = *reinterpret_cast<const uint4*>(rec + kKvScales + 128 + r * 16);
      const uint4 v0 = *reinterpret_cast<const uint4*>(rec + kKvV + lane * 16);
      const uint4 v1 = *reinterpret_cast<const uint4*>(rec + kKvV + 512 + lane * 16);

      // scores of keys r and r + 8 for query t of each four
      float sc[kFours][2] = {};
      {
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
        float ks[2][4];
        scales_of(s0.x, ks[0][0], ks[0][1]);
        scales_of(s0.y, ks[0][2], ks[0][3]);
        scales_of(s1.x, ks[1][0], ks[1][1]);
        scales_of(s1.y, ks[1][2], ks[1][3]);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint32_t a0 = w0[g] & 0x0f0f0f0fu, a1 = w1[g] & 0x0f0f0f0fu;
          const uint32_t a2 = (w0[g] >> 4) & 0x0f0f0f0fu, a3 = (w1[g] >> 4) & 0x0f0f0f0fu;
#pragma unroll
          for (int n = 0; n < kFours; ++n) {
            float d[4];
            mma_e4m3(d, a0, a1, a2, a3, qf[n][g][0], qf[n][g][1], off[n][g][0], off[n][g][1]);
            sc[n][0] = fmaf(ks[0][g], fmaf(d[1], 1.0f / kLow, d[0]), sc[n][0]);
            sc[n][1] = fmaf(ks[1][g], fmaf(d[3], 1.0f / kLow, d[2]), sc[n][1]);
          }
        }
      }
      const bool edge = (tile + 1) * kKvTile > all;
      bool raise = false;
#pragma unroll
      for (int n = 0; n < kFours; ++n) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          sc[n][h] *= factor[n];
          if (edge && tile * kKvTile + r + 8 * h >= limit[n]) sc[n][h] = -INFINITY;
        }
        raise = raise || fmaxf(sc[n][0], sc[n][1]) > m[n] + kSlack;
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int n = 0; n < kFours; ++n) {
          float top = fmaxf(fmaxf(sc[n][0], sc[n][1]), m[n]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const float shrink = top == -INFINITY ? 1.0f : ex2_approx(m[n] - top);
          m[n] = top;
          l[n] *= shrink;
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (kFours == 1 || (i & 1) == (n & 1)) acc[g][u][n / 2][i] *= shrink;
        }
      }
#pragma unroll
      for (int n = 0; n < kFours; ++n) {
        const float at_m = m[n] == -INFINITY ? 0.0f : m[n];
        sc[n][0] = ex2_approx(sc[n][0] - at_m);
        sc[n][1] = ex2_approx(sc[n][1] - at_m);
        l[n] += sc[n][0] + sc[n][1];
      }
      // what a token that is not there holds as scales may be anything
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
      uint32_t p0[kCols], p1[kCols];   // B operands: keys 0 to 7 and 8 to 15
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint32_t a0 = g < 2 ? v0.x : v0.y, c0 = g < 2 ? v0.z : v0.w, a1 = g < 2 ? v1.x : v1.y, c1 = g < 2 ? v1.z : v1.w;
        uint32_t x[4], y[4];
        v_pairs(__byte_perm(a0, c0, g & 1 ? 0x7632 : 0x5410), x);
        v_pairs(__byte_perm(a1, c1, g & 1 ? 0x7632 : 0x5410), y);
        if (kFours == 1) {
          if (g % 2 == 0) {
            p0[0] = transpose8(pack_bf16x2(sc[0][0] * vs[0][g], sc[0][0] * vs[0][g + 1]));
            p1[0] = transpose8(pack_bf16x2(sc[0][1] * vs[1][g], sc[0][1] * vs[1][g + 1]));
          }
        } else {
#pragma unroll
          for (int n = 0; n < kCols; ++n) {
            p0[n] = transpose8(pack_bf16x2(sc[2 * n][0] * vs[0][g], sc[2 * n + 1][0] * vs[0][g]));
            p1[n] = transpose8(pack_bf16x2(sc[2 * n][1] * vs[1][g], sc[2 * n + 1][1] * vs[1][g]));
          }
        }
#pragma unroll
        for (int n = 0; n < kCols; ++n) {
          mma_bf16(acc[g][0][n], x[0], x[1], y[0], y[1], p0[n], p1[n]);
          mma_bf16(acc[g][1][n], x[2], x[3], y[2], y[3], p0[n], p1[n]);
        }
      }
    }
    cp_async_wait<0>();
    __syncwarp();

    // the warps' results, joined
    float* const mo = reinterpret_cast<float*>(mine);              // [kRows][kDim], then m and l
    float2* const ml = reinterpret_cast<float2*>(mo + kRows * kDim);
#pragma unroll
    for (int n = 0; n < kFours; ++n) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[n] += __shfl_xor_sync(0xffffffffu, l[n], o);
      const int row = 4 * n + t;
      if (r == 0) ml[row] = make_float2(m[n], l[n]);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int c = kFours == 1 ? g & 1 : n & 1;
#pragma unroll
        for (int u = 0; u < 2; ++u)
          *reinterpret_cast<float2*>(mo + row * kDim + 32 * g + 4 * r + 2 * u) =
              make_float2(acc[g][u][n / 2][c], acc[g][u][n / 2][2 + c]);
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

// Queries a CTA works on, four at a time, tiles of them, and CTAs.
struct Grid {
  int fours, row_tiles, ctas;
};
Grid grid_of(int B, int S, int Hq, int Hkv, int max_pages, int page_size) {
  Grid g;
  const long long rows = (long long)S * (Hq / Hkv);
  g.fours = rows <= 4 ? 1 : rows <= 8 ? 2 : 4;
  g.row_tiles = (int)((rows + 4 * g.fours - 1) / (4 * g.fours));
  // no more CTAs than the cache could give work to
  const double most = (double)max_pages * (page_size / kKvTile) * B * Hkv * g.row_tiles / kLeast + 1.0;
  const int fit = 152 * (g.fours == 1 ? 4 : g.fours == 2 ? 3 : 2);
  g.ctas = most < fit ? (int)most : fit;
  return g;
}

template <int kFours>
cudaError_t launch_both(const AttnParams& p, int ctas, cudaStream_t stream) {
  const cudaError_t e = launch_dependent(kv4_attn_kernel<kFours>, dim3((unsigned)ctas), kThreads, 0, stream, p);
  if (e != cudaSuccess) return e;
  return launch_dependent(kv4_join_kernel<4 * kFours>, dim3((unsigned)ctas, 4 * kFours), 256, 0, stream, p);
}

}  // namespace

size_t attn_kv4_workspace(int B, int S, int Hq, int Hkv, int max_pages, int page_size) {
  const Grid g = grid_of(B, S, Hq, Hkv, max_pages, page_size);
  return (size_t)g.ctas * (16 + 2 * 4 * g.fours * (kDim * 4 + 8));
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
  p.part_ml = reinterpret_cast<float2*>(p.part_o + (size_t)g.ctas * 2 * 4 * g.fours * kDim);
  switch (g.fours) {
    case 1: return launch_both<1>(p, g.ctas, stream);
    case 2: return launch_both<2>(p, g.ctas, stream);
    default: return launch_both<4>(p, g.ctas, stream);
  }
}

}  // namespace sa
