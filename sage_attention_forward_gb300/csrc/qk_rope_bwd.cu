// Backward of the norm of Q and K with the rotation, sm_103a.
//
//   g = rope^T(dy),  xhat = x r,  r = 1 / sqrt(sum x^2 / N + eps), formed again from x
//   dx = r (g w - xhat sum(g w xhat) / N),   dw = sum over rows of g xhat
//
// Bound by memory: x and dy are read and dx written once.  Units and lanes as in the forward (qk_rope.cu), but CTAs walk
// over the units, first Q's, then K's, and a lane keeps the sums of dw of its own 16 channels in registers over all of
// its rows.  Each CTA writes its sums once to the workspace; a second kernel adds them up in one fixed order: no atomics,
// the same bits every time.  Those sums take half of a thread's 128 registers, and at the 16 warps an SM that are left it is
// instructions and their order that count: two channels an instruction, the lanes of a row known to the kernel, one row's
// work not mixed with the next one's (16896 x 48 heads of 128 BF16: 110.4 -> 102.6 us, 0.91 of the copy rate; rows through
// shared memory, four ahead, 114).
#include <cuda_runtime.h>

#include <algorithm>

#include "qk_rope.cuh"

namespace sa {
namespace {

// Rows of a slot whose loads are under way (two where registers reach for them), and CTAs an SM.
constexpr int rows_ahead(int map, int pairs, int lanes, bool wide) {
  return map < kAny ? (wide || map == kApart || lanes == 5 ? 1 : 2) : pairs == 8 ? 1 : 2;
}
constexpr int ctas_an_sm(int map, int pairs, bool wide) {
  return map < kAny ? (map == kApart && wide ? 1 : 2) : pairs == 4 ? 2 : 1;
}

__device__ __forceinline__ void prefetch_l2(const void* at) { asm volatile("prefetch.global.L2 [%0];" ::"l"(at)); }

template <class T, int kMap, int kPairs, int kLanes>
__global__ void __launch_bounds__(kRopeThreads, ctas_an_sm(kMap, kPairs, sizeof(T) == 4))
    rope_bwd_kernel(const __grid_constant__ RopeParams p) {
  using L = RopeLane<T, kMap, kPairs, kLanes>;
  constexpr int kAhead = rows_ahead(kMap, kPairs, kLanes, sizeof(T) == 4);
  // The row behind those comes as far as L2, which takes no registers (8002 x 40 heads of 64 FP32 45.9 -> 43.9 us, 33000 x 40 of
  // 80 BF16 133 -> 123, of 128 165 -> 162; by other maps it cost up to 5 %).
  constexpr bool kFetch = kLanes > 0 && (kMap == kHalf || kMap == kNext);
  // the weights by lanes, [kPairs / 2][lanes] of four (registers do not reach for them); then the tables,
  // [warps][p.shared bytes], or at the end the warps' sums, [warps][N]
  extern __shared__ float4 shared[];
  unsigned char* const tables = reinterpret_cast<unsigned char*>(shared + kPairs / 2 * 32);
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const L ln(p, lane);
  const int slot = lane / ln.lanes;
  const uint32_t mine = slot < ln.slots && ln.some() ? slot : 1u << 31;   // (no head of any token's)
  float2* const table = reinterpret_cast<float2*>(tables + warp * p.shared);
  float* const swap = reinterpret_cast<float*>(table + p.table);
  float* const sums = reinterpret_cast<float*>(tables);

  for (int which = 0; which < 2; ++which) {
    const RopeSide& sd = p.side[which];
    if (sd.heads == 0) continue;
    float da[kPairs] = {}, db[kPairs] = {};
    if (warp == 0 && slot == 0) {
      float w[2 * kPairs];
      ln.weights(sd.w, p, w);
#pragma unroll
      for (int k = 0; k < kPairs / 2; ++k)
        shared[k * ln.lanes + ln.l] = make_float4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    }
    __syncthreads();
    for (int unit = blockIdx.x * kRopeWarps + warp; unit < sd.units; unit += gridDim.x * kRopeWarps) {
      const int token = sd.parts == 1 ? unit : unit / sd.parts, first = (unit - token * sd.parts) * sd.per_unit;
      const int end = min(first + sd.per_unit, sd.heads);
      const int b = div_by(token, p.S), s = token - b * (int)p.S.d;
      RopeWalk<T> x, dy, dx;
      x.start(sd.x, sd.xs, b, s, first, end, slot);
      dy.start(sd.dy, sd.ds, b, s, first, end, slot);
      dx.start(sd.y, sd.ys, b, s, first, end, slot);
      typename L::Raw rx[kAhead], rd[kAhead];
      auto load = [&](int u, int at) {   // heads from `at` on
        if (at + mine < (uint32_t)end) {
          ln.load(x.row, rx[u]);
          ln.load(dy.row, rd[u]);
        } else {
          rx[u] = rd[u] = {};
        }
        x.next(ln.slots, sd.x_step);
        dy.next(ln.slots, sd.d_step);
        if (kFetch && at + ln.slots + mine < (uint32_t)end) {
          prefetch_l2(x.row + ln.ca);
          prefetch_l2(dy.row + ln.ca);
          if (kMap == kHalf) {
            prefetch_l2(x.row + ln.cb);
            prefetch_l2(dy.row + ln.cb);
          }
        }
      };
#pragma unroll
      for (int u = 0; u < kAhead; ++u) load(u, first + u * ln.slots);
      if (L::kExchange && lane == 0) swap[16 * 32] = 0.0f;
      rope_table<kMap>(p, ln.lanes, b, s, lane, table);
      for (int base = first; base < end; base += kAhead * ln.slots) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (base + u * ln.slots >= end) break;
          float a[kPairs], c[kPairs], ga[kPairs], gc[kPairs];
          const bool in = base + u * ln.slots + mine < (uint32_t)end;
          ln.values(rx[u], a, c);
          ln.values(rd[u], ga, gc);
          load(u, base + (u + kAhead) * ln.slots);
          __syncwarp();   // (the next row's work is not drawn before this one's: registers do not reach for both)
          const float r = rsqrtf(fmaf(rope_row_sum<kLanes>(rope_squares(a, c), ln.lanes, ln.l), p.inv_n, p.eps));
          rope_turn<kPairs>(p, ln, table, swap, lane, ga, gc);
          float dot0 = 0.0f, dot1 = 0.0f;
#pragma unroll
          for (int i = 0; i < kPairs; i += 2) {
            const float4 w = load_shared(shared + i / 2 * ln.lanes + ln.l);
            fmul2(a[i], a[i + 1], a[i], a[i + 1], r, r);
            fmul2(c[i], c[i + 1], c[i], c[i + 1], r, r);
            ffma2(da[i], da[i + 1], ga[i], ga[i + 1], a[i], a[i + 1], da[i], da[i + 1]);
            ffma2(db[i], db[i + 1], gc[i], gc[i + 1], c[i], c[i + 1], db[i], db[i + 1]);
            fmul2(ga[i], ga[i + 1], ga[i], ga[i + 1], w.x, w.y);
            fmul2(gc[i], gc[i + 1], gc[i], gc[i + 1], w.z, w.w);
            ffma2(dot0, dot1, ga[i], ga[i + 1], a[i], a[i + 1], dot0, dot1);
            ffma2(dot0, dot1, gc[i], gc[i + 1], c[i], c[i + 1], dot0, dot1);
          }
          const float dot = rope_row_sum<kLanes>(dot0 + dot1, ln.lanes, ln.l) * -p.inv_n;
          if (in) {
#pragma unroll
            for (int i = 0; i < kPairs; i += 2) {
              ffma2(a[i], a[i + 1], a[i], a[i + 1], dot, dot, ga[i], ga[i + 1]);
              ffma2(c[i], c[i + 1], c[i], c[i + 1], dot, dot, gc[i], gc[i + 1]);
              fmul2(a[i], a[i + 1], a[i], a[i + 1], r, r);
              fmul2(c[i], c[i + 1], c[i], c[i + 1], r, r);
            }
            ln.store(dx.row, a, c);
          }
          dx.next(ln.slots, sd.y_step);
        }
      }
    }
    if (sd.partial == nullptr) {
      __syncthreads();   // Q's weights are no longer read
      continue;
    }
    // the warp's slots, then the CTA's warps, in order
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const float a = da[i], c = db[i];
      for (int o = ln.lanes; o + ln.lanes <= 32; o += ln.lanes) {
        da[i] += __shfl_down_sync(0xffffffffu, a, o);
        db[i] += __shfl_down_sync(0xffffffffu, c, o);
      }
    }
    __syncthreads();   // the tables, or Q's sums, are no longer read
    if (slot == 0 && ln.some()) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const int ia = ln.first(i), ib = ln.second(i);
        if (ia < p.N) sums[warp * p.N + ia] = da[i];
        if (ib < p.N) sums[warp * p.N + ib] = db[i];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.N; c += kRopeThreads) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kRopeWarps; ++w) v += sums[w * p.N + c];
      sd.partial[(long long)blockIdx.x * p.N + c] = v;
    }
    __syncthreads();   // before the tables are written again
  }
}

// dw of 8 channels of Q (blockIdx.y = 0) or K: 64 threads a channel, each over its share of the CTAs in order.
__global__ void __launch_bounds__(512) rope_grad_kernel(const float* q_parts, const float* k_parts, int n_parts, int N, void* dqw,
                                                        void* dkw, int type) {
  __shared__ float sum[64][9];
  griddep_wait();
  const float* const parts = blockIdx.y ? k_parts : q_parts;
  void* const out = blockIdx.y ? dkw : dqw;
  if (parts == nullptr) return;
  const int c = blockIdx.x * 8 + (threadIdx.x & 7), g = threadIdx.x >> 3;
  float v = 0.0f;
  if (c < N) {
#pragma unroll 8
    for (int i = g; i < n_parts; i += 64) v += __ldcs(parts + (long long)i * N + c);
  }
  sum[g][threadIdx.x & 7] = v;
  __syncthreads();
  if (threadIdx.x >= 256) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;   // a warp joins a channel
  v = sum[lane][warp] + sum[lane + 32][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int mine = blockIdx.x * 8 + warp;
  if (lane != 0 || mine >= N) return;
  if (type == kF32) reinterpret_cast<float*>(out)[mine] = v;
  else if (type == kBF16) reinterpret_cast<__nv_bfloat16*>(out)[mine] = __float2bfloat16(v);
  else reinterpret_cast<__half*>(out)[mine] = __float2half(v);
}

template <class T>
cudaError_t launch_bwd(const RopeParams& p, int& ctas, bool vec, bool next, cudaStream_t stream) {
  return with_rope_map<true>(p, vec, next, [&](auto map, auto pairs, auto lanes) {
    const size_t tables = (size_t)kRopeWarps * p.shared, sums = (size_t)kRopeWarps * p.N * sizeof(float);
    constexpr int kMap = decltype(map)::value, kPairs = decltype(pairs)::value, kLanes = decltype(lanes)::value;
    ctas = std::min(ctas, 152 * ctas_an_sm(kMap, kPairs, sizeof(T) == 4));
    return launch_dependent(rope_bwd_kernel<T, kMap, kPairs, kLanes>, dim3((unsigned)ctas), kRopeThreads,
                            kPairs / 2 * 32 * sizeof(float4) + (tables > sums ? tables : sums), stream, p);
  });
}

}  // namespace

// What the workspace has room for, of any kernel: up to four CTAs an SM, of which the present ones take two at most (launch_bwd;
// the size is the interface's and stays).  K's sums begin where Q's would end at that number.  A CTA may have no unit.
int rope_bwd_ctas(int B, int S, int Hq, int Hk) {
  const long long warps = ((long long)B * S * (Hq > Hk ? Hq : Hk) + 3) / 4;
  const long long ctas = (warps + kRopeWarps - 1) / kRopeWarps;
  return ctas < 4 * 152 ? (int)ctas : 4 * 152;
}

cudaError_t launch_qk_norm_rope_bwd(const RopeArgs& a, float* workspace, cudaStream_t stream) {
  RopeParams p;
  rope_params(p, a);
  const bool vec = rope_shape(p, a, true);
  int ctas = rope_bwd_ctas(a.B, a.S, a.side[0].H, a.side[1].H);
  for (int i = 0; i < 2; ++i) {
    RopeSide& s = p.side[i];
    const int H = a.side[i].H;
    s.per_unit = (H + p.slots - 1) / p.slots * p.slots;
    while (s.per_unit > p.slots && (long long)p.tokens * ((H + s.per_unit - 1) / s.per_unit) < 152 * 32)
      s.per_unit = (s.per_unit / 2 + p.slots - 1) / p.slots * p.slots;
    s.parts = (H + s.per_unit - 1) / std::max(s.per_unit, 1);
    s.units = p.tokens * s.parts;
    if (H > 0 && a.side[i].dw != nullptr) s.partial = workspace + (size_t)i * ctas * a.N;
  }
  cudaError_t e = a.type == kF32    ? launch_bwd<float>(p, ctas, vec, a.interleaved, stream)
                  : a.type == kBF16 ? launch_bwd<__nv_bfloat16>(p, ctas, vec, a.interleaved, stream)
                                    : launch_bwd<__half>(p, ctas, vec, a.interleaved, stream);
  if (e != cudaSuccess || (p.side[0].partial == nullptr && p.side[1].partial == nullptr)) return e;
  return launch_dependent(rope_grad_kernel, dim3((unsigned)(a.N + 7) / 8, 2), 512, 0, stream,
                          static_cast<const float*>(p.side[0].partial), static_cast<const float*>(p.side[1].partial), ctas,
                          a.N, a.side[0].dw, a.side[1].dw, a.w_type);
}

}  // namespace sa
