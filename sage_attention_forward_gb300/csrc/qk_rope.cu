// Rotary positions of Q and K, and their norm with the rotation in the same pass, sm_103a.
//
//   rotation:   y = rope(x)             (its backward: the same with the angles negated)
//   with norm:  y = rope(x r w),  r = 1 / sqrt(sum x^2 / N + eps)
//
// Bound by memory: x is read and y written once.  A unit is a warp's: heads of one token, Q's and then K's, the token's
// cosines formed once for all of them (qk_rope.cuh).  A lane holds both channels of its pairs, 16 channels in
// all, so the rotation takes no exchange (but of halves that are no whole pieces: their partners come through shared
// memory); a head of 128 channels is 8 lanes', and a warp works on four heads at a time.
#include <cuda_runtime.h>

#include "qk_rope.cuh"

namespace sa {
namespace {

// Rows of a slot whose loads are under way, and CTAs an SM: loads in flight are what the kernels wait for, and more warps with
// fewer rows each do better (76112 x 80 heads of 128 BF16: four rows, two CTAs 546 us; two, three 497; two, four 467; with the
// norm, 33000 x 40 heads in halves: two, three 106.5; two, four 102.9).
constexpr int rows_ahead(int map, bool wide) { return map < kAny && wide ? 1 : 2; }
constexpr int ctas_an_sm(int map, int pairs, bool wide) {
  return map >= kAny ? (pairs == 4 ? 3 : 1) : map == kApart ? (wide ? 2 : 3) : wide ? 3 : 4;
}

template <class T, int kMap, int kPairs, int kLanes, bool kNorm>
__global__ void __launch_bounds__(kRopeThreads, ctas_an_sm(kMap, kPairs, sizeof(T) == 4))
    rope_fwd_kernel(const __grid_constant__ RopeParams p) {
  using L = RopeLane<T, kMap, kPairs, kLanes>;
  constexpr int kAhead = rows_ahead(kMap, sizeof(T) == 4);
  // kNorm: the weights of Q and of K by lanes, [2][kPairs / 2][lanes] of four (held in registers they take the warps that hide
  // the loads); then the tables
  extern __shared__ __align__(16) float4 shared[];
  unsigned char* const tables = reinterpret_cast<unsigned char*>(shared + (kNorm ? kPairs * 32 : 0));
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if constexpr (kNorm) {
    const L ln(p, lane);
    if (warp < 2 && lane < ln.lanes) {
      float w[2 * kPairs];
      ln.weights(p.side[warp].w, p, w);
#pragma unroll
      for (int k = 0; k < kPairs / 2; ++k)
        shared[(warp * (kPairs / 2) * 32) + k * ln.lanes + ln.l] = make_float4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    }
    __syncthreads();
  }
  const int unit = blockIdx.x * kRopeWarps + warp;
  const int token = div_by(unit, p.by_parts), part = unit - token * (int)p.by_parts.d;
  if (token >= p.tokens) return;
  const int b = div_by(token, p.S), s = token - b * (int)p.S.d;
  const L ln(p, lane);
  const int slot = lane / ln.lanes;
  const bool mine = slot < ln.slots && ln.some();
  // the unit's share of Q's heads, then of K's, p.slots of them a turn
  const int turns_q = p.side[0].turns, turns = turns_q + p.side[1].turns;
  auto share = [&](RopeWalk<T>& w, int which, const void* base, const long long (&str)[3]) {
    const RopeSide& sd = p.side[which];
    w.start(base, str, b, s, part * sd.per_unit, min((part + 1) * sd.per_unit, sd.heads), slot);
  };
  RopeWalk<T> in, out;
  int to_load = 0;
  share(in, 0, p.side[0].x, p.side[0].xs);
  share(out, 0, p.side[0].y, p.side[0].ys);
  typename L::Raw raw[kAhead];
  auto load = [&](int u) {
    if (to_load == turns_q) share(in, 1, p.side[1].x, p.side[1].xs);
    if (mine && in.head < in.end && to_load < turns) ln.load(in.row, raw[u]);
    else raw[u] = {};
    in.next(ln.slots, p.side[to_load >= turns_q].x_step);
    ++to_load;
  };
#pragma unroll
  for (int u = 0; u < kAhead; ++u) load(u);

  float2* const table = reinterpret_cast<float2*>(tables + warp * p.shared);
  float* const swap = reinterpret_cast<float*>(table + p.table);
  if (L::kExchange && lane == 0) swap[16 * 32] = 0.0f;
  rope_table<kMap>(p, ln.lanes, b, s, lane, table);

  for (int base = 0; base < turns; base += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (base + u >= turns) break;
      if (base + u == turns_q) share(out, 1, p.side[1].y, p.side[1].ys);
      float a[kPairs], c[kPairs];
      const bool some = mine && out.head < out.end;
      ln.values(raw[u], a, c);
      load(u);
      if constexpr (kNorm) {
        const float sum = rope_row_sum<kLanes>(rope_squares(a, c), ln.lanes, ln.l), r = rsqrtf(fmaf(sum, p.inv_n, p.eps));
        const float4* const weights = shared + (base + u >= turns_q ? kPairs / 2 * 32 : 0) + ln.l;
#pragma unroll
        for (int k = 0; k < kPairs / 2; ++k) {
          float4 w = load_shared(weights + k * ln.lanes);
          fmul2(w.x, w.y, w.x, w.y, r, r);
          fmul2(w.z, w.w, w.z, w.w, r, r);
          fmul2(a[2 * k], a[2 * k + 1], a[2 * k], a[2 * k + 1], w.x, w.y);
          fmul2(c[2 * k], c[2 * k + 1], c[2 * k], c[2 * k + 1], w.z, w.w);
        }
      }
      if (L::kExchange || some) rope_turn<kPairs>(p, ln, table, swap, lane, a, c);
      if (some) ln.store(out.row, a, c);
      out.next(ln.slots, p.side[base + u >= turns_q].y_step);
    }
  }
}

template <class T, bool kNorm>
cudaError_t launch_fwd(RopeParams& p, bool vec, bool next, cudaStream_t stream) {
  const long long units = (long long)p.tokens * p.by_parts.d;
  return with_rope_map<kNorm>(p, vec, next, [&](auto map, auto pairs, auto lanes) {
    constexpr int kPairs = decltype(pairs)::value;
    return launch_dependent(rope_fwd_kernel<T, decltype(map)::value, kPairs, decltype(lanes)::value, kNorm>,
                            dim3((unsigned)((units + kRopeWarps - 1) / kRopeWarps)), kRopeThreads,
                            (kNorm ? kPairs * 32 * sizeof(float4) : 0) + kRopeWarps * p.shared, stream, p);
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
  // All heads of a token in one unit, so that its cosines are formed once; parts of them where that leaves warps idle.
  const int turns = (a.side[0].H + p.slots - 1) / p.slots + (a.side[1].H + p.slots - 1) / p.slots;
  int parts = 1;
  while (2 * parts <= turns && (long long)p.tokens * parts < 152 * 32) parts *= 2;
  for (int i = 0; i < 2; ++i) {
    RopeSide& s = p.side[i];
    s.per_unit = ((a.side[i].H + parts - 1) / parts + p.slots - 1) / p.slots * p.slots;
    s.turns = s.per_unit / p.slots;
  }
  p.by_parts = make_div(parts);
  return norm ? launch_typed<true>(p, a.type, vec, a.interleaved, stream)
              : launch_typed<false>(p, a.type, vec, a.interleaved, stream);
}

}  // namespace sa
