// Rotary positions of Q and K, and their norm with the rotation in the same pass, sm_103a.
//
//   rotation:   y = rope(x)             (its backward: the same with the angles negated)
//   with norm:  y = rope(x r w),  r = 1 / sqrt(sum x^2 / N + eps)
//
// Bound by memory: x is read and y written once.  A unit is a warp's: some heads of one token, of Q or of K, the
// token's cosines formed once for all of them (qk_rope.cuh).  A lane holds both channels of its pairs, 16 channels in
// all, so the rotation takes no exchange; a head of 128 channels is 8 lanes', and a warp has four rows' worth of four
// heads each under way.
#include <cuda_runtime.h>

#include "qk_rope.cuh"

namespace sa {
namespace {

template <class T, int kMap, int kPairs, bool kNorm>
__global__ void __launch_bounds__(kRopeThreads) rope_fwd_kernel(const __grid_constant__ RopeParams p) {
  using L = RopeLane<T, kMap, kPairs>;
  constexpr int kAhead = sizeof(T) == 4 || (!L::kVec && kPairs == 8) ? 2 : 4;   // rows of a slot under way
  extern __shared__ __align__(16) float2 tables[];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int unit = blockIdx.x * kRopeWarps + warp;
  const int token = div_by(unit, p.by_parts), part = unit - token * (int)p.by_parts.d;
  if (token >= p.tokens) return;
  const int which = part >= p.side[0].parts;
  const RopeSide& sd = p.side[which];
  const int first = (which ? part - p.side[0].parts : part) * p.per_unit;
  const int end = min(first + p.per_unit, sd.heads);
  const int b = div_by(token, p.S), s = token - b * (int)p.S.d;
  const L ln(p, lane);
  const int slot = L::kVec ? lane / p.lanes : 0;
  const bool mine = slot < p.slots && ln.some();
  const T* const x = reinterpret_cast<const T*>(sd.x) + b * sd.xs[0] + s * sd.xs[1];
  T* const y = reinterpret_cast<T*>(sd.y) + b * sd.ys[0] + s * sd.ys[1];
  typename L::Raw raw[kAhead];
  auto load = [&](int u, int h) {
    if (mine && h < end) ln.load(x + h * sd.xs[2], p.pairs, raw[u]);
  };
  int h = first + slot;
#pragma unroll
  for (int u = 0; u < kAhead; ++u) load(u, h + u * p.slots);

  float2* const table = tables + warp * p.table;
  rope_table<L::kVec>(p, b, s, lane, table);
  float cs[kPairs], sn[kPairs], wa[kPairs], wb[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int at = L::kVec ? (i / 2 * p.lanes + ln.l) * 2 + i % 2 : ln.pair(i);
    const float2 t = ln.pair(i) < p.pairs ? table[at] : make_float2(1.0f, 0.0f);
    cs[i] = t.x;
    sn[i] = t.y;
  }
  if (kNorm) ln.weights(sd.w, p, wa, wb);

  for (int base = first; base < end; base += kAhead * p.slots) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u, h += p.slots) {
      if (base + u * p.slots >= end) break;
      float a[kPairs], c[kPairs];
      const bool in = mine && h < end;
      if (in) {
        ln.values(raw[u], a, c);
      } else {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) a[i] = c[i] = 0.0f;
      }
      load(u, h + kAhead * p.slots);
      if (kNorm) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) sum = fmaf(a[i], a[i], fmaf(c[i], c[i], sum));
        sum = rope_row_sum(sum, p.lanes);
        const float r = rsqrtf(fmaf(sum, p.inv_n, p.eps));
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          a[i] = a[i] * r * wa[i];
          c[i] = c[i] * r * wb[i];
        }
      }
      if (in) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          if (ln.pair(i) >= p.pairs) continue;   // (an infinity beside a channel that passes stays out of it)
          const float a0 = a[i];
          a[i] = a0 * cs[i] - c[i] * sn[i];
          c[i] = c[i] * cs[i] + a0 * sn[i];
        }
        ln.store(y + h * sd.ys[2], p.pairs, a, c);
      }
    }
  }
}

template <class T, bool kNorm>
cudaError_t launch_fwd(RopeParams& p, bool vec, bool next, cudaStream_t stream) {
  const long long units = (long long)p.tokens * p.by_parts.d;
  return with_rope_map(vec, next, p.N, [&](auto map, auto pairs) {
    return launch_dependent(rope_fwd_kernel<T, decltype(map)::value, decltype(pairs)::value, kNorm>, dim3((unsigned)((units + kRopeWarps - 1) / kRopeWarps)),
                            kRopeThreads, (size_t)kRopeWarps * p.table * sizeof(float2), stream, p);
  });
}
template <bool kNorm>
cudaError_t launch_typed(RopeParams& p, int type, bool vec, bool next, cudaStream_t stream) {
  if (type == kF32) return launch_fwd<float, kNorm>(p, vec, next, stream);
  if (type == kBF16) return launch_fwd<__nv_bfloat16, kNorm>(p, vec, next, stream);
  return launch_fwd<__half, kNorm>(p, vec, next, stream);
}

}  // namespace

cudaError_t launch_rope_fwd(const RopeArgs& a, bool norm, cudaStream_t stream) {
  RopeParams p;
  rope_params(p, a);
  const bool vec = rope_shape(p, a, norm);
  // All heads of a token in one unit, so that its cosines are formed once; fewer where that leaves warps idle.
  const int heads = a.side[0].H > a.side[1].H ? a.side[0].H : a.side[1].H;
  auto parts = [&](int H) { return (H + p.per_unit - 1) / p.per_unit; };
  p.per_unit = (heads + p.slots - 1) / p.slots * p.slots;
  while (p.per_unit > p.slots &&
         (long long)p.tokens * (parts(a.side[0].H) + parts(a.side[1].H)) < 152 * 32)
    p.per_unit = (p.per_unit / 2 + p.slots - 1) / p.slots * p.slots;
  for (int i = 0; i < 2; ++i) p.side[i].parts = parts(a.side[i].H);
  p.by_parts = make_div(p.side[0].parts + p.side[1].parts);
  return norm ? launch_typed<true>(p, a.type, vec, a.interleaved, stream)
              : launch_typed<false>(p, a.type, vec, a.interleaved, stream);
}

}  // namespace sa
