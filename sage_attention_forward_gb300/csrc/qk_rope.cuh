// What the rotation of Q and K, and their norm with the rotation, share in both directions.
//
//   angle(t, i) = position(t, axis(i)) w_i         y = m (a cos - b sin, b cos + a sin) of each pair (a, b) of channels
//
// Frequencies come as turns a position in units of 2^-64, so that the whole turns of an angle fall off in the
// product of two integers, for any position of 32 bits, without tables of cosines in memory and without 64-bit floating
// point (of which an SM has little).  What is left is off by less than 2^-30 turns (the table's entries by up to 3.5 units,
// the axis being in two bits, times 2^31; the product is cut at 2^-32), and then rounded to 24 bits: 2^-26 turns at most.  A
// warp forms the cosines of one token once, in shared memory, and takes them for all of the token's heads.
#pragma once

#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "pieces.cuh"
#include "ptx_train.cuh"

namespace sa {

constexpr int kRopeThreads = 256, kRopeWarps = kRopeThreads / 32;

struct RopeSide {
  const void *x, *dy;             // dy: backward of the norm (the rotation's own backward reads x)
  void* y;                        // y, or dx
  const void* w;
  float* partial;                 // backward: [CTAs][N] sums of dw, or nullptr
  long long xs[3], ds[3], ys[3];  // element strides (b, s, h)
  long long x_step, d_step, y_step;   // from a turn's heads to the next one's
  int heads, per_unit, turns;     // heads of a unit, in turns of p.slots
  int parts, units;               // backward: units of a token, and of all tokens
};
struct RopeParams {
  RopeSide side[2];               // Q and K
  const int* pos;                 // or nullptr: the place in the sequence
  const unsigned long long* freq;
  long long pos_str[3];           // element strides (b, s, axis)
  int tokens, N, pairs, axes;
  int table, shared;              // cosines and sines of a warp; its bytes of shared memory
  int lanes, slots, per, word;         // lanes a row, rows a warp takes at a time; by the channel:
                                  // pairs a lane, pairs of neighbours aligned to their size
  Div S, by_parts;                // by_parts: units that a token's heads are divided into
  float magnitude, eps, inv_n;
  int inverse, w_type, w_vec;     // w_vec: weights by 16 bytes
};

// Where a lane's channels are.  By 16-byte pieces, 16 channels a lane: kNext, pairs of neighbours; kHalf, halves that are whole
// pieces: both channels of eight pairs; kApart, other halves: 16 neighbours, whose partners come through shared memory.  By the
// channel: kAny, kAnyNext: pairs l, l + lanes, ... of a row's lanes l.
enum RopeMap : int { kHalf = 0, kNext = 1, kApart = 2, kAny = 3, kAnyNext = 4 };
constexpr int kSwap = 17 * 32;   // kApart: floats of a warp's exchange: [16][lane], then a zero

// kLanes: lanes a row where the kernel is made for that number (sums over them unrolled, offsets known), or 0.
template <class T, int kMap, int kPairs, int kLanes>
struct RopeLane {
  static constexpr bool kVec = kMap < kAny, kExchange = kMap == kApart;
  static constexpr int kPieces = kVec ? (int)sizeof(T) : 1;   // 16-byte pieces of a lane's 16 channels
  struct Raw {
    uint4 piece[kVec ? kPieces : 1];
    uint32_t a[kVec ? 1 : kPairs], b[kVec ? 1 : kPairs];   // bits of the channels; 16-bit neighbours both in a
  };
  static constexpr bool kShort = sizeof(T) == 2;
  __device__ __forceinline__ bool neighbours() const { return kMap == kAnyNext && word; }
  int l, ca, cb, last;   // kVec: first channels of the two runs of eight; last: N
  int lanes, slots;      // p.lanes, p.slots
  int word;              // else: pairs l, l + lanes, ...; pairs of neighbours as one access
  int at_a[kVec ? 1 : kPairs], at_b[kVec ? 1 : kPairs];   // else: the channels of each pair
  int from[kMap == kApart ? 16 : 1];                      // kApart: where the exchange has the channels' partners

  __device__ __forceinline__ RopeLane(const RopeParams& p, int lane) {
    lanes = kLanes > 0 ? kLanes : p.lanes;
    slots = kLanes > 0 ? 32 / kLanes : p.slots;
    l = lane % lanes;
    word = p.word;
    last = p.N;
    const bool turned = kMap == kHalf && 8 * l < p.pairs;
    ca = turned ? 8 * l : 16 * l;
    cb = turned ? p.pairs + 8 * l : 16 * l + 8;
    if constexpr (kMap == kApart) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int c = 16 * l + i, t = c < p.pairs ? c + p.pairs : c - p.pairs;
        from[i] = c < 2 * p.pairs ? (t & 15) * 32 + lane - l + (t >> 4) : 16 * 32;
      }
    }
    if constexpr (!kVec) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const bool half = kMap == kAny && pair(i) < p.pairs;
        at_a[i] = half ? pair(i) : 2 * pair(i);
        at_b[i] = half ? pair(i) + p.pairs : 2 * pair(i) + 1;
      }
    }
  }
  // kVec: the lane has channels of a row
  __device__ __forceinline__ bool some() const { return !kVec || 16 * l < last; }
  __device__ __forceinline__ int pair(int i) const { return kVec ? 8 * l + i : l + lanes * i; }
  __device__ __forceinline__ int first(int i) const {
    if constexpr (kVec) return kMap == kHalf ? ca + i : 16 * l + 2 * i;
    else return at_a[i];
  }
  __device__ __forceinline__ int second(int i) const {
    if constexpr (kVec) return kMap == kHalf ? cb + i : 16 * l + 2 * i + 1;
    else return at_b[i];
  }
  __device__ __forceinline__ void load(const T* row, Raw& r) const {
    if constexpr (kVec) {
      constexpr int half = kPieces / 2;
#pragma unroll
      for (int k = 0; k < half; ++k) {
        r.piece[k] = __ldcs(reinterpret_cast<const uint4*>(row + ca) + k);
        r.piece[half + k] = __ldcs(reinterpret_cast<const uint4*>(row + cb) + k);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const int a = first(i), b = second(i);
        if (neighbours()) {   // (N is even)
          r.a[i] = r.b[i] = 0u;
          if (a >= last) continue;
          if constexpr (kShort) {
            r.a[i] = *reinterpret_cast<const uint32_t*>(row + a);
          } else {
            const uint2 two = *reinterpret_cast<const uint2*>(row + a);
            r.a[i] = two.x;
            r.b[i] = two.y;
          }
        } else if constexpr (kShort) {
          r.a[i] = a < last ? reinterpret_cast<const unsigned short*>(row)[a] : 0u;
          r.b[i] = b < last ? reinterpret_cast<const unsigned short*>(row)[b] : 0u;
        } else {
          r.a[i] = a < last ? reinterpret_cast<const uint32_t*>(row)[a] : 0u;
          r.b[i] = b < last ? reinterpret_cast<const uint32_t*>(row)[b] : 0u;
        }
      }
    }
  }
  __device__ __forceinline__ void values(const Raw& r, float (&a)[kPairs], float (&b)[kPairs]) const {
    if constexpr (kVec) {
      float x[16];
#pragma unroll
      for (int k = 0; k < kPieces; ++k) unpack<T>(r.piece[k], x + k * Piece<T>::kN);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = kMap == kHalf ? x[i] : x[2 * i];
        b[i] = kMap == kHalf ? x[8 + i] : x[2 * i + 1];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        if constexpr (kShort) {
          float two[2], other[2];
          unpack_word(r.a[i], two, T());
          unpack_word(r.b[i], other, T());
          a[i] = two[0];
          b[i] = neighbours() ? two[1] : other[0];
        } else {
          a[i] = __uint_as_float(r.a[i]);
          b[i] = __uint_as_float(r.b[i]);
        }
      }
    }
  }
  __device__ __forceinline__ void store(T* row, const float (&a)[kPairs], const float (&b)[kPairs]) const {
    if constexpr (kVec) {
      float x[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[kMap == kHalf ? i : 2 * i] = a[i];
        x[kMap == kHalf ? 8 + i : 2 * i + 1] = b[i];
      }
      constexpr int half = kPieces / 2;
#pragma unroll
      for (int k = 0; k < half; ++k) {
        __stcs(reinterpret_cast<uint4*>(row + ca) + k, pack<T>(x + k * Piece<T>::kN));
        __stcs(reinterpret_cast<uint4*>(row + cb) + k, pack<T>(x + (half + k) * Piece<T>::kN));
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const int ia = first(i), ib = second(i);
        if (neighbours()) {
          const float two[2] = {a[i], b[i]};
          if (ia >= last) continue;
          if constexpr (kShort) *reinterpret_cast<uint32_t*>(row + ia) = pack_word(two, T());
          else *reinterpret_cast<float2*>(row + ia) = make_float2(a[i], b[i]);
        } else {
          if (ia < last) row[ia] = T(a[i]);
          if (ib < last) row[ib] = T(b[i]);
        }
      }
    }
  }
  // The weights of the lane's channels (1 without weights, or where there is no channel).
  // Those of pairs i and i + 1 (i even) in v[2 i], v[2 i + 1], then their second channels'.
  __device__ __forceinline__ void weights(const void* w, const RopeParams& p, float (&v)[2 * kPairs]) const {
    float a[kPairs], b[kPairs];
    weights(w, p, a, b);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      v[i / 2 * 4 + i % 2] = a[i];
      v[i / 2 * 4 + 2 + i % 2] = b[i];
    }
  }
  __device__ __forceinline__ void weights(const void* w, const RopeParams& p, float (&a)[kPairs],
                                          float (&b)[kPairs]) const {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) a[i] = b[i] = 1.0f;
    if (w == nullptr || !some()) return;
    if constexpr (kVec) {
      if (p.w_vec) {
        if (p.w_type == kF32) {
          RopeLane<float, kMap, 8, kLanes>(p, l).take(reinterpret_cast<const float*>(w), a, b);
        } else {
          take(reinterpret_cast<const T*>(w), a, b);
        }
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int ia = first(i), ib = second(i);
      if (p.w_type == kF32) {
        const float* f = reinterpret_cast<const float*>(w);
        if (ia < last) a[i] = f[ia];
        if (ib < last) b[i] = f[ib];
      } else {
        const T* f = reinterpret_cast<const T*>(w);
        if (ia < last) a[i] = (float)f[ia];
        if (ib < last) b[i] = (float)f[ib];
      }
    }
  }
  __device__ __forceinline__ void take(const T* row, float (&a)[kPairs], float (&b)[kPairs]) const {
    Raw r;
    load(row, r);
    values(r, a, b);
  }
};

// A lane's rows of a token, p.slots heads a turn: Q's from `first` on, then K's.
template <class T>
struct RopeWalk {
  T* row;
  int head, end;   // the lane's head of the next turn; heads end here
  __device__ __forceinline__ void start(const void* base, const long long (&str)[3], int b, int s, int first, int stop, int slot) {
    head = first + slot;
    end = stop;
    row = reinterpret_cast<T*>(const_cast<void*>(base)) + b * str[0] + s * str[1] + head * str[2];
  }
  __device__ __forceinline__ void next(int slots, long long step) {
    row += step;
    head += slots;
  }
};

// Cosine and sine (times the magnitude) of a token's pairs, to `table`; the sine negated for the backward.  By pieces: in the
// order in which lanes read them, [4][lanes] of two pairs (both cosines, both sines), or for kApart [8][lanes] of two channels, a
// first half's sine negated and (1, 0) where a channel passes; else pair by pair.
template <int kMap>
__device__ __forceinline__ void rope_table(const RopeParams& p, int lanes, int b, int s, int lane, float2* table) {
  constexpr bool kVec = kMap < kAny;
  __syncwarp();   // the last token's are no longer read
  for (int i = lane; i < p.pairs; i += 32) {
    const unsigned long long f = __ldg(p.freq + i);
    int at = s;
    if (p.pos != nullptr) {
      const int axis = min((int)(f & 3), p.axes - 1);
      at = __ldg(p.pos + b * p.pos_str[0] + s * p.pos_str[1] + axis * p.pos_str[2]);
    }
    const unsigned long long turns = (unsigned long long)(long long)at * (f & ~3ull);
    float sn, cs;   // of half turns in [-1, 1)
    sincospif((float)(int)(turns >> 32) * 0x1p-31f, &sn, &cs);
    cs *= p.magnitude;
    sn *= p.inverse ? -p.magnitude : p.magnitude;
    if (kMap == kApart) {
      const int c = i + p.pairs;
      table[((i % 16 / 2) * lanes + i / 16) * 2 + i % 2] = make_float2(cs, -sn);
      table[((c % 16 / 2) * lanes + c / 16) * 2 + c % 2] = make_float2(cs, sn);
    } else if (kVec) {
      float* const two = reinterpret_cast<float*>(table + ((i % 8 / 2) * lanes + i / 8) * 2);
      two[i % 2] = cs;
      two[2 + i % 2] = sn;
    } else {
      table[i] = make_float2(cs, sn);
    }
  }
  if (kMap == kApart)
    for (int c = 2 * p.pairs + lane; c < 16 * lanes; c += 32)
      table[((c % 16 / 2) * lanes + c / 16) * 2 + c % 2] = make_float2(1.0f, 0.0f);
  __syncwarp();
}

// (volatile: held in registers over the rows, weights and cosines would spill)
__device__ __forceinline__ float4 load_shared(const float4* at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(smem_u32(at)));
  return v;
}

__device__ __forceinline__ float2 load_shared(const float2* at) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(smem_u32(at)));
  return v;
}

// The sum of squares of a lane's channels.
template <int kPairs>
__device__ __forceinline__ float rope_squares(const float (&a)[kPairs], const float (&b)[kPairs]) {
  float x = 0.0f, y = 0.0f;
#pragma unroll
  for (int i = 0; i < kPairs; i += 2) {
    ffma2(x, y, a[i], a[i + 1], a[i], a[i + 1], x, y);
    ffma2(x, y, b[i], b[i + 1], b[i], b[i + 1], x, y);
  }
  return x + y;
}

// The rotation of a lane's channels (every lane of the warp takes part).
template <int kPairs, class L>
__device__ __forceinline__ void rope_turn(const RopeParams& p, const L& ln, const float2* table, float* swap, int lane,
                                          float (&a)[kPairs], float (&b)[kPairs]) {
  if constexpr (L::kExchange) {
    __syncwarp();   // the last row's are no longer read
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      swap[2 * i * 32 + lane] = a[i];
      swap[(2 * i + 1) * 32 + lane] = b[i];
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      const float4 t = load_shared(reinterpret_cast<const float4*>(table) + k * ln.lanes + ln.l);   // of two channels
      a[k] = a[k] * t.x + swap[ln.from[2 * k]] * t.y;
      b[k] = b[k] * t.z + swap[ln.from[2 * k + 1]] * t.w;
    }
  } else {
    // (pairs that pass: an infinity beside a channel that passes stays out of it)
    auto turn = [&](int i, float cs, float sn) {
      const float a0 = a[i];
      a[i] = a0 * cs - b[i] * sn;
      b[i] = b[i] * cs + a0 * sn;
    };
    if constexpr (L::kVec) {
      const int turned = p.pairs - ln.pair(0);   // of the lane's eight
      if (turned <= 0) return;
#pragma unroll
      for (int k = 0; k < kPairs / 2; ++k) {
        const float4 t = load_shared(reinterpret_cast<const float4*>(table) + k * ln.lanes + ln.l);
        float &a0 = a[2 * k], &a1 = a[2 * k + 1], &b0 = b[2 * k], &b1 = b[2 * k + 1];
        if (turned > 2 * k + 1) {
          float x0, x1;   // two products in one instruction; one of a sign that it does not have in two
          const float y0 = -b0 * t.z, y1 = -b1 * t.w;
          fmul2(x0, x1, a0, a1, t.z, t.w);
          ffma2(a0, a1, a0, a1, t.x, t.y, y0, y1);
          ffma2(b0, b1, b0, b1, t.x, t.y, x0, x1);
        } else if (turned == 2 * k + 1) {
          turn(2 * k, t.x, t.z);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        if (ln.pair(i) >= p.pairs) continue;
        const float2 t = load_shared(table + ln.pair(i));
        turn(i, t.x, t.y);
      }
    }
  }
}

// Sum over the lanes of a row, the same in all of them.
template <int kLanes>
__device__ __forceinline__ float rope_row_sum(float v, int lanes, int l) {
  const int n = kLanes > 0 ? kLanes : lanes;
  if ((n & (n - 1)) == 0) {
#pragma unroll
    for (int o = 1; o < n; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  float sum = v;   // in a row's first lane
#pragma unroll
  for (int o = 1; o < n; ++o) sum += __shfl_down_sync(0xffffffffu, v, o);
  return __shfl_sync(0xffffffffu, sum, (int)(threadIdx.x & 31) - l);
}

// Calls f with the map, the pairs a lane and, for a norm, the lanes a row where they are usual ones (8: 128 channels; by pieces
// 4 and 5, too: 64 and 80; else 0), as constants.
template <bool kNorm, class F>
cudaError_t with_rope_map(const RopeParams& p, bool vec, bool next, F&& f) {
  using std::integral_constant;
  constexpr integral_constant<int, 0> any{};
  constexpr integral_constant<int, 8> eight{};
  auto pieces = [&](auto map) {
    if constexpr (kNorm) {
      if (p.lanes == 8) return f(map, eight, eight);
      if (p.lanes == 4) return f(map, eight, integral_constant<int, 4>{});
      if (p.lanes == 5) return f(map, eight, integral_constant<int, 5>{});
    }
    return f(map, eight, any);
  };
  auto channels = [&](auto pairs, auto lanes) {
    return next ? f(integral_constant<int, kAnyNext>{}, pairs, lanes) : f(integral_constant<int, kAny>{}, pairs, lanes);
  };
  if (vec && next) return pieces(integral_constant<int, kNext>{});
  if (vec) return p.pairs % 8 == 0 ? pieces(integral_constant<int, kHalf>{}) : pieces(integral_constant<int, kApart>{});
  if (p.per == 8) return channels(eight, any);
  if constexpr (kNorm) {
    if (p.lanes == 8) return channels(integral_constant<int, 4>{}, eight);
  }
  return channels(integral_constant<int, 4>{}, any);
}

// Whether rows go by 16 bytes (kApart while its shared memory stays below 48 KB); lanes a row and rows a warp.
inline bool rope_shape(RopeParams& p, const RopeArgs& a, bool norm) {
  const int piece = a.type == kF32 ? 4 : 8;
  bool vec = a.N % 16 == 0 && (a.interleaved || a.R % 16 == 0 || a.N <= 256), word = a.N % 2 == 0;
  for (int i = 0; i < 2; ++i) {
    const RopeArgs::Side& s = a.side[i];
    if (s.H == 0) continue;
    const void* ptr[3] = {s.x, s.dy, s.y};
    const long long* str[3] = {s.x_str, s.dy_str, s.y_str};
    for (int k = 0; k < 3; ++k) {
      if (ptr[k] == nullptr) continue;
      vec = vec && (reinterpret_cast<uintptr_t>(ptr[k]) & 15u) == 0 && (a.B == 1 || str[k][0] % piece == 0) &&
            (a.S == 1 || str[k][1] % piece == 0) && (s.H == 1 || str[k][2] % piece == 0);
      word = word && reinterpret_cast<uintptr_t>(ptr[k]) % (a.type == kF32 ? 8 : 4) == 0 && (a.B == 1 || str[k][0] % 2 == 0) &&
             (a.S == 1 || str[k][1] % 2 == 0) && (s.H == 1 || str[k][2] % 2 == 0);
    }
  }
  p.word = word;
  const int pairs = (a.N + 1) / 2;
  auto lanes = [&](int n) {
    // a norm's sums go over a power of two of lanes, unless more rows a turn pay for the longer way: three in place of two do
    // (33000 x 40 heads of 80 BF16, backward: 157 -> 148 us), five in place of four do not (96 channels: 163 -> 169)
    int up = n;
    while (norm && (up & (up - 1)) != 0) ++up;
    return 2 * (32 / n) >= 3 * (32 / up) ? n : up;
  };
  // by the channel: four pairs a lane, or eight where that leaves fewer lanes idle (N = 130: a row takes 17 of 32, or 9)
  const int four = lanes((pairs + 3) / 4), eight = lanes((pairs + 7) / 8);
  p.per = !vec && four <= 32 && 5 * (32 / four) * 2 >= 4 * (32 / eight) ? 4 : 8;
  p.lanes = vec ? lanes(a.N / 16) : p.per == 4 ? four : eight;
  p.slots = 32 / p.lanes;
  const bool apart = vec && !a.interleaved && p.pairs % 8 != 0;
  p.table = apart ? 16 * p.lanes : vec ? 8 * p.lanes : p.pairs;
  p.shared = (p.table + (apart ? kSwap / 2 : 0)) * (int)sizeof(float2);
  for (RopeSide& s : p.side) {
    s.x_step = s.xs[2] * p.slots;
    s.d_step = s.ds[2] * p.slots;
    s.y_step = s.ys[2] * p.slots;
  }
  return vec;
}

inline void rope_params(RopeParams& p, const RopeArgs& a) {
  p.w_vec = 1;
  for (int i = 0; i < 2; ++i) {
    const RopeArgs::Side& s = a.side[i];
    p.w_vec = p.w_vec && (reinterpret_cast<uintptr_t>(s.w) & 15u) == 0;
    p.side[i].x = s.x;
    p.side[i].dy = s.dy;
    p.side[i].y = s.y;
    p.side[i].w = s.w;
    p.side[i].partial = nullptr;
    p.side[i].heads = s.H;
    for (int k = 0; k < 3; ++k) {
      p.side[i].xs[k] = s.x_str[k];
      p.side[i].ds[k] = s.dy_str[k];
      p.side[i].ys[k] = s.y_str[k];
      p.pos_str[k] = a.pos_str[k];
    }
  }
  p.pos = a.pos;
  p.freq = a.freq;
  p.tokens = a.B * a.S;
  p.N = a.N;
  p.pairs = a.R / 2;
  p.axes = a.axes;
  p.S = make_div(a.S);
  p.magnitude = a.magnitude;
  // With eps = 0 the r of zeros would be infinite, and rows that a turn does not have are zeros: dw would be NaN.  The smallest
  // eps changes no mean square from 2^-124 on.  (An r of 0 for those rows, chosen in the backward's loop, cost it 1 to 2 %.)
  p.eps = std::max(a.eps, 0x1p-149f);
  p.inv_n = 1.0f / (float)a.N;
  p.inverse = a.inverse;
  p.w_type = a.w_type;
}

}  // namespace sa
