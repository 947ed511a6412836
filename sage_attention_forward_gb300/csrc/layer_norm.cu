// Layer norm over the channels of rows, forward and backward, sm_103a.
//
//   mean = sum x / N,  rstd = 1 / sqrt(sum (x - mean)^2 / N + eps),  xhat = (x - mean) rstd
//   y    = xhat w + b
//   g    = dy w,  dx = rstd (g - sum g / N - xhat sum (g xhat) / N)
//   dw   = sum over rows of dy xhat,  db = sum over rows of dy
//
// Both directions are bound by memory: the forward reads x and writes y, the backward reads x and
// dy and writes dx, once each.  A row is held in registers, in 32 bits, between its statistics (two
// passes over the registers, so that no square of a large mean is subtracted) and its result.
// Rows of up to 512 channels (256 in the backward) take 4 to 32 lanes of a warp, 16 (8) channels a lane;
// longer ones a CTA, 16 channels a thread, through a ring of rows in shared memory where their alignment
// allows it (20000 x 9000 BF16 without it, 32 channels a thread: 237 us forward and 320 backward, so 129
// and 196).  CTAs walk over the rows: while a row is worked on the next one's loads are under way, and in
// the backward pass a thread keeps the sums of dw and db of its own channels in registers over all of its
// rows.  Each CTA writes its sums once to the workspace, and a second kernel adds them up, in one fixed
// order: no atomics, the same bits every time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "ptx_train.cuh"

namespace sa {
namespace {

struct Rows {
  long long str[3];   // element strides (b, s, h)
  int even;           // all rows are str[2] apart
};
struct LnParams {
  const void *x, *dy, *w, *b;
  void *y, *dx;
  float *mean, *rstd;             // outputs of the forward, inputs of the backward
  Rows xs, ys, dys, dxs;
  int rows, N;
  Div S, H;
  float eps;
  int w_type;                     // type of w and b
  float* partial;                 // backward: [2][CTAs][N] sums of dw and db, or nullptr
  int ring;                       // through shared memory: rows in the backward's ring
  int slot;                       // bytes of a row's place in it
};

// Where a row starts, in elements.  (The backward's ring takes the general form: with the other one it
// was slower up to 8192 channels, 400 us instead of 368 for 76112 x 5120.)
__device__ __forceinline__ long long row_in_ring(const LnParams& p, const Rows& r, int row) {
  const int bs = div_by(row, p.H), h = row - bs * (int)p.H.d, b = div_by(bs, p.S), s = bs - b * (int)p.S.d;
  return (long long)b * r.str[0] + (long long)s * r.str[1] + (long long)h * r.str[2];
}

__device__ __forceinline__ long long row_at(const LnParams& p, const Rows& r, int row) {
  return r.even ? (long long)row * r.str[2] : row_in_ring(p, r, row);
}

template <class T>
struct Piece {   // 16 bytes
  static constexpr int kN = 16 / sizeof(T);
  T v[kN];
};
// The piece of channels [c, c + kN) of a row; channels past N are 0.  kVec: rows, strides and weights
// allow 16-byte accesses, and N is a whole number of pieces.
template <bool kVec, class T>
__device__ __forceinline__ uint4 load_piece(const T* row, int c, const LnParams& p) {
  uint4 raw = make_uint4(0u, 0u, 0u, 0u);
  if (c >= p.N) return raw;
  if (kVec) return __ldcs(reinterpret_cast<const uint4*>(row + c));
  Piece<T> t = *reinterpret_cast<Piece<T>*>(&raw);
#pragma unroll
  for (int e = 0; e < Piece<T>::kN; ++e)
    if (c + e < p.N) t.v[e] = row[c + e];
  return *reinterpret_cast<uint4*>(&t);
}
__device__ __forceinline__ void unpack_word(uint32_t w, float* x, __nv_bfloat16) {
  x[0] = __uint_as_float(w << 16);
  x[1] = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void unpack_word(uint32_t w, float* x, __half) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  x[0] = f.x;
  x[1] = f.y;
}
__device__ __forceinline__ void unpack_word(uint32_t w, float* x, float) { x[0] = __uint_as_float(w); }
template <class T>
__device__ __forceinline__ void unpack(const uint4& raw, float* x) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack_word(w[i], x + i * (4 / sizeof(T)), T());
}
__device__ __forceinline__ uint32_t pack_word(const float* x, __nv_bfloat16) { return pack_bf16x2(x[0], x[1]); }
__device__ __forceinline__ uint32_t pack_word(const float* x, __half) {
  const __half2 h = __floats2half2_rn(x[0], x[1]);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_word(const float* x, float) { return __float_as_uint(x[0]); }
template <class T>
__device__ __forceinline__ uint4 pack(const float* x) {
  constexpr int k = 4 / sizeof(T);
  return make_uint4(pack_word(x, T()), pack_word(x + k, T()), pack_word(x + 2 * k, T()), pack_word(x + 3 * k, T()));
}
template <bool kVec, class T>
__device__ __forceinline__ void store_piece(T* row, int c, const float* x, const LnParams& p) {
  if (c >= p.N) return;
  const uint4 raw = pack<T>(x);
  if (kVec) {
    __stcs(reinterpret_cast<uint4*>(row + c), raw);
    return;
  }
  const Piece<T> t = *reinterpret_cast<const Piece<T>*>(&raw);
#pragma unroll
  for (int e = 0; e < Piece<T>::kN; ++e)
    if (c + e < p.N) row[c + e] = t.v[e];
}
// kN weights (or biases) from channel c on; `other` where there are none.
template <bool kVec, int kN>
__device__ __forceinline__ void load_weights(const void* w, int c, float other, const LnParams& p, float* out) {
#pragma unroll
  for (int e = 0; e < kN; ++e) out[e] = other;
  if (w == nullptr || c >= p.N) return;
  if (p.w_type == kF32) {
    const float* f = reinterpret_cast<const float*>(w) + c;
    if (kVec) {
#pragma unroll
      for (int e = 0; e < kN / 4; ++e) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(f) + e);
        out[4 * e] = v.x, out[4 * e + 1] = v.y, out[4 * e + 2] = v.z, out[4 * e + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (c + e < p.N) out[e] = __ldg(f + e);
    }
    return;
  }
  const unsigned short* s = reinterpret_cast<const unsigned short*>(w) + c;
  unsigned short raw[kN];
  if (kVec && kN == 8) {
    *reinterpret_cast<uint4*>(raw) = __ldg(reinterpret_cast<const uint4*>(s));
  } else {
#pragma unroll
    for (int e = 0; e < kN; ++e) raw[e] = kVec || c + e < p.N ? __ldg(s + e) : (unsigned short)0;
  }
#pragma unroll
  for (int e = 0; e < kN; ++e)
    out[e] = p.w_type == kBF16 ? __uint_as_float((uint32_t)raw[e] << 16) : __half2float(__ushort_as_half(raw[e]));
}

// How a row is spread: kLanes > 0 lanes of a warp, or (0) a CTA; kValues channels a thread, in pieces
// kLanes (or blockDim.x) apart.
template <int kLanes>
struct Spread {
  static constexpr bool kWarp = kLanes > 0;
  __device__ __forceinline__ static int lane() { return kWarp ? (int)(threadIdx.x & (kLanes - 1)) : (int)threadIdx.x; }
  __device__ __forceinline__ static int width() { return kWarp ? kLanes : (int)blockDim.x; }
  // rows that the grid works on at once, and this thread's first
  __device__ __forceinline__ static int step() { return kWarp ? (int)(gridDim.x * (blockDim.x / (kWarp ? kLanes : 1))) : (int)gridDim.x; }
  __device__ __forceinline__ static int first() {
    return kWarp ? (int)((blockIdx.x * blockDim.x + threadIdx.x) / (kWarp ? kLanes : 1)) : (int)blockIdx.x;
  }
};

// Sums over a row's threads, the same in all of them; every thread of the CTA (of the warp) calls it.  scratch: two
// floats per warp, another half of it in each call (turn), so that one barrier is enough.
template <int kLanes, int kSums>
__device__ __forceinline__ void row_sums(float (&v)[kSums], float (*scratch)[32][2], int& turn) {
  constexpr int kTop = kLanes > 0 ? kLanes / 2 : 16;
#pragma unroll
  for (int d = kTop; d >= 1; d >>= 1)
#pragma unroll
    for (int i = 0; i < kSums; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
  if (kLanes > 0) return;
  float(*s)[2] = scratch[turn & 1];
  ++turn;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < kSums; ++i) s[threadIdx.x >> 5][i] = v[i];
  __syncthreads();
  const int warps = (int)blockDim.x >> 5, lane = (int)threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < kSums; ++i) v[i] = lane < warps ? s[lane][i] : 0.0f;
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1)
#pragma unroll
    for (int i = 0; i < kSums; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
}

// kMax: the largest CTA (registers); kValues: channels a thread.
// kRows: rows whose loads are under way ahead of the one worked on.
template <class T, bool kVec, int kLanes, int kValues, int kRows, int kMax>
__global__ void __launch_bounds__(kMax) ln_fwd_kernel(const LnParams p) {
  using S = Spread<kLanes>;
  constexpr int kN = Piece<T>::kN, kPieces = kValues / kN;
  __shared__ float scratch[2][32][2];
  griddep_wait();
  const int lane = S::lane(), step = S::step();
  int row = S::first(), turn = 0;
  const float inv_n = 1.0f / (float)p.N;
  constexpr bool kHold = kValues <= 16;   // weights in registers, or again from L1 for each row
  float w[kHold ? kValues : 1], b[kHold ? kValues : 1];
  if (kHold) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      load_weights<kVec, kN>(p.w, (lane + k * S::width()) * kN, 1.0f, p, &w[kHold ? k * kN : 0]);
      load_weights<kVec, kN>(p.b, (lane + k * S::width()) * kN, 0.0f, p, &b[kHold ? k * kN : 0]);
    }
  }
  uint4 raw[kRows][kPieces];
  auto load = [&](uint4(&to)[kPieces], int r) {
    const T* x = reinterpret_cast<const T*>(p.x) + (r < p.rows ? row_at(p, p.xs, r) : 0);
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
      to[k] = r < p.rows ? load_piece<kVec, T>(x, (lane + k * S::width()) * kN, p) : make_uint4(0u, 0u, 0u, 0u);
  };
#pragma unroll
  for (int u = 0; u < kRows; ++u) load(raw[u], row + u * step);
  // (a warp's rows are consecutive: its lanes leave the loop together but for the last rows, whose
  // idle lanes work on zeros and store nothing)
  int base = S::kWarp ? row - (int)((threadIdx.x & 31) / (S::kWarp ? kLanes : 1)) : row;
  while (base < p.rows) {
#pragma unroll
  for (int u = 0; u < kRows; ++u, base += step, row += step) {
    if (base >= p.rows) break;
    float v[kValues];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) unpack<T>(raw[u][k], v + k * kN);
    load(raw[u], row + kRows * step);
    float sum[1], sum2[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kValues; i += 2) fadd2(sum2[0], sum2[1], sum2[0], sum2[1], v[i], v[i + 1]);   // (channels past N are 0)
    sum[0] = sum2[0] + sum2[1];
    row_sums<kLanes>(sum, scratch, turn);
    const float mean = sum[0] * inv_n;
    float sq[1], sq2[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int c = (lane + k * S::width()) * kN;
#pragma unroll
      for (int e = k * kN; e < (k + 1) * kN; e += 2) {
        fadd2(v[e], v[e + 1], v[e], v[e + 1], -mean, -mean);
        if (!kVec) {
          v[e] = c + e - k * kN < p.N ? v[e] : 0.0f;
          v[e + 1] = c + e + 1 - k * kN < p.N ? v[e + 1] : 0.0f;
        }
      }
      if (kVec && c >= p.N) continue;
#pragma unroll
      for (int e = k * kN; e < (k + 1) * kN; e += 2) ffma2(sq2[0], sq2[1], v[e], v[e + 1], v[e], v[e + 1], sq2[0], sq2[1]);
    }
    sq[0] = sq2[0] + sq2[1];
    row_sums<kLanes>(sq, scratch, turn);
    const float rstd = 1.0f / sqrtf(sq[0] * inv_n + p.eps);
    if (row < p.rows) {
      T* y = reinterpret_cast<T*>(p.y) + row_at(p, p.ys, row);
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int c = (lane + k * S::width()) * kN;
        float ww[kHold ? 1 : kN], bb[kHold ? 1 : kN], out[kN];
        if (!kHold) {
          load_weights<kVec, kN>(p.w, c, 1.0f, p, ww);
          load_weights<kVec, kN>(p.b, c, 0.0f, p, bb);
        }
        const float *pw = kHold ? &w[kHold ? k * kN : 0] : ww, *pb = kHold ? &b[kHold ? k * kN : 0] : bb;
#pragma unroll
        for (int e = 0; e < kN; e += 2) {
          fmul2(out[e], out[e + 1], v[k * kN + e], v[k * kN + e + 1], rstd, rstd);
          ffma2(out[e], out[e + 1], out[e], out[e + 1], pw[e], pw[e + 1], pb[e], pb[e + 1]);
        }
        store_piece<kVec, T>(y, c, out, p);
      }
      if (lane == 0) {
        p.mean[row] = mean;
        p.rstd[row] = rstd;
      }
    }
  }
  }
}

template <class T, bool kVec, int kLanes, int kValues, int kRows, int kMax>
__global__ void __launch_bounds__(kMax) ln_bwd_kernel(const LnParams p) {
  using S = Spread<kLanes>;
  constexpr int kN = Piece<T>::kN, kPieces = kValues / kN;
  // the next row's loads are under way while a row is worked on; not with 32 channels a thread, where
  // the registers do not reach
  constexpr bool kAhead = kValues <= 16, kWide = !kAhead;
  __shared__ float scratch[2][32][2];
  // a warp's rows: [warps][N], to add the warps up.  32 channels a thread: the thread's sums of dw and
  // db, [2][32][threads], for which there are no registers.
  extern __shared__ float sums[];
  griddep_wait();
  const int lane = S::lane(), step = S::step();
  int row = S::first(), turn = 0;
  const float inv_n = 1.0f / (float)p.N;
  constexpr bool kHold = !kWide;   // weights in registers, or again from L1 for each row
  float w[kHold ? kValues : 1];
  if (kHold) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
      load_weights<kVec, kN>(p.w, (lane + k * S::width()) * kN, 1.0f, p, &w[kHold ? k * kN : 0]);
  }
  float dw[kWide ? 1 : kValues] = {}, db[kWide ? 1 : kValues] = {};
  float* const wide = sums + threadIdx.x;
  if (kWide)
    for (int i = 0; i < 2 * kValues; ++i) wide[i * blockDim.x] = 0.0f;
  constexpr int kHeld = kAhead ? kPieces : 1;
  uint4 rx[kRows][kHeld], rd[kRows][kHeld];
  float mean[kRows], rstd[kRows];
  auto load = [&](int u, int r) {
    const bool in = r < p.rows;
    const T* x = reinterpret_cast<const T*>(p.x) + (in ? row_at(p, p.xs, r) : 0);
    const T* d = reinterpret_cast<const T*>(p.dy) + (in ? row_at(p, p.dys, r) : 0);
    if (kAhead) {
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        const int c = (lane + k * S::width()) * kN;
        rx[u][k] = in ? load_piece<kVec, T>(x, c, p) : make_uint4(0u, 0u, 0u, 0u);
        rd[u][k] = in ? load_piece<kVec, T>(d, c, p) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
    mean[u] = in ? __ldg(p.mean + r) : 0.0f;
    rstd[u] = in ? __ldg(p.rstd + r) : 0.0f;
  };
#pragma unroll
  for (int u = 0; u < kRows; ++u) load(u, row + u * step);
  int base = S::kWarp ? row - (int)((threadIdx.x & 31) / (S::kWarp ? kLanes : 1)) : row;
  while (base < p.rows) {
#pragma unroll
  for (int u = 0; u < kRows; ++u, base += step, row += step) {
    if (base >= p.rows) break;
    const float m = mean[u], rs = rstd[u];
    // 32 channels a thread are not held: each pass reads the row, the second time from the caches
    const T* const gx = reinterpret_cast<const T*>(p.x) + (kAhead ? 0 : row_at(p, p.xs, row));
    const T* const gd = reinterpret_cast<const T*>(p.dy) + (kAhead ? 0 : row_at(p, p.dys, row));
    // xhat and g of a piece's channels (where there is no channel dy is 0, and so is g)
    float xh[kAhead ? kValues : kN], g[kAhead ? kValues : kN], d[kN];
    auto piece = [&](int k, float* ph, float* pg) {
      float x[kN], ww[kHold ? 1 : kN];
      const int c = (lane + k * S::width()) * kN;
      unpack<T>(kAhead ? rx[u][kAhead ? k : 0] : load_piece<kVec, T>(gx, c, p), x);
      unpack<T>(kAhead ? rd[u][kAhead ? k : 0] : load_piece<kVec, T>(gd, c, p), d);
      if (!kHold) load_weights<kVec, kN>(p.w, c, 1.0f, p, ww);
      const float* pw = kHold ? &w[kHold ? k * kN : 0] : ww;
#pragma unroll
      for (int e = 0; e < kN; e += 2) {
        fadd2(ph[e], ph[e + 1], x[e], x[e + 1], -m, -m);
        fmul2(ph[e], ph[e + 1], ph[e], ph[e + 1], rs, rs);
        fmul2(pg[e], pg[e + 1], d[e], d[e + 1], pw[e], pw[e + 1]);
      }
    };
    float s[2], s0[2] = {0.0f, 0.0f}, s1[2] = {0.0f, 0.0f};   // sums of g and of g xhat
#pragma unroll(kAhead ? kPieces : 1)
    for (int k = 0; k < kPieces; ++k) {
      float *ph = xh + (kAhead ? k * kN : 0), *pg = g + (kAhead ? k * kN : 0);
      piece(k, ph, pg);
#pragma unroll
      for (int e = 0; e < kN; e += 2) {
        if (kWide) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            wide[(k * kN + e + i) * blockDim.x] += d[e + i] * ph[e + i];
            wide[(kValues + k * kN + e + i) * blockDim.x] += d[e + i];
          }
        } else {
          float *a = &dw[kWide ? 0 : k * kN + e], *b = &db[kWide ? 0 : k * kN + e];
          ffma2(a[0], a[1], d[e], d[e + 1], ph[e], ph[e + 1], a[0], a[1]);
          fadd2(b[0], b[1], b[0], b[1], d[e], d[e + 1]);
        }
        fadd2(s0[0], s0[1], s0[0], s0[1], pg[e], pg[e + 1]);
        ffma2(s1[0], s1[1], pg[e], pg[e + 1], ph[e], ph[e + 1], s1[0], s1[1]);
      }
    }
    load(u, row + kRows * step);
    s[0] = s0[0] + s0[1];
    s[1] = s1[0] + s1[1];
    row_sums<kLanes>(s, scratch, turn);
    const float m0 = -s[0] * inv_n, m1 = -s[1] * inv_n;
    if (row < p.rows) {
      T* dx = reinterpret_cast<T*>(p.dx) + row_at(p, p.dxs, row);
#pragma unroll(kAhead ? kPieces : 1)
      for (int k = 0; k < kPieces; ++k) {
        float *ph = xh + (kAhead ? k * kN : 0), *pg = g + (kAhead ? k * kN : 0), out[kN];
        if (!kAhead) piece(k, ph, pg);
#pragma unroll
        for (int e = 0; e < kN; e += 2) {
          ffma2(pg[e], pg[e + 1], ph[e], ph[e + 1], m1, m1, pg[e], pg[e + 1]);
          fadd2(pg[e], pg[e + 1], pg[e], pg[e + 1], m0, m0);
          fmul2(out[e], out[e + 1], pg[e], pg[e + 1], rs, rs);
        }
        store_piece<kVec, T>(dx, (lane + k * S::width()) * kN, out, p);
      }
    }
  }
  }
  if (p.partial == nullptr) return;
  // this CTA's sums: [2][CTAs][N]
  float* const out[2] = {p.partial + (long long)blockIdx.x * p.N,
                         p.partial + ((long long)gridDim.x + blockIdx.x) * p.N};
  if (!S::kWarp) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        const int c = (lane + k * S::width()) * kN + e;
        if (c < p.N) {
          out[0][c] = kWide ? wide[(k * kN + e) * blockDim.x] : dw[kWide ? 0 : k * kN + e];
          out[1][c] = kWide ? wide[(kValues + k * kN + e) * blockDim.x] : db[kWide ? 0 : k * kN + e];
        }
      }
    return;
  }
  const int warp = (int)threadIdx.x >> 5, warps = (int)blockDim.x >> 5;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* v = which == 0 ? dw : db;
#pragma unroll
    for (int i = 0; i < (kWide ? 1 : kValues); ++i)
#pragma unroll
      for (int d = S::kWarp ? kLanes : 32; d < 32; d <<= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
    __syncthreads();
    if ((threadIdx.x & 31) < (S::kWarp ? kLanes : 32)) {
#pragma unroll
      for (int k = 0; k < kPieces; ++k)
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const int c = (lane + k * S::width()) * kN + e;
          if (c < p.N) sums[warp * p.N + c] = v[kWide ? 0 : k * kN + e];
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.N; c += blockDim.x) {
      float a = 0.0f;
      for (int i = 0; i < warps; ++i) a += sums[i * p.N + c];
      out[which][c] = a;
    }
  }
}

// ------------------------------------------------------------------ rows of a CTA through shared memory
// Rows that a CTA takes, of up to 10240 channels (in the backward up to 16384, in FP32 up to 14080: two rows of x and dy
// have to fit), that allow 16-byte accesses: one thread copies whole rows ahead into a ring in shared memory (16 channels
// a thread are too few bytes under way otherwise: with the next row in registers the forward reached 3.3 and the
// backward 2.1 of 6.7 TB/s).
// The forward works on two rows at once (their sums share barriers and shuffles' latency) with the next
// two under way; the backward, which reads its rows twice, on one of three, or of two where three would
// leave room for fewer CTAs.
constexpr int kMaxRing = 4;
struct RowRing {
  uint64_t full[kMaxRing];
  uint32_t abort_flag;
};
__device__ uint32_t g_err_norm;
std::atomic<bool> g_launched{false};   // a kernel with a ring

__device__ __forceinline__ void ring_init(RowRing& r) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxRing; ++s) mbar_init(&r.full[s], 1);
    r.abort_flag = 0;
    fence_mbar_init();
  }
  griddep_wait();
  __syncthreads();
}
// The row in slot s has landed, for the (phase + 1)-th time.  Should the wait run out, that is recorded, and
// the rest of the kernel works on what is there: every thread keeps to its barriers.  The thread that loads loads
// nothing more then: a slot whose row has not landed is not asked for another one.
__device__ __forceinline__ bool ring_wait(RowRing& r, int s, int phase) {
  return mbar_wait<false>(&r.full[s], phase & 1, &r.abort_flag, &g_err_norm, kErrTimeoutTma);
}

// Rows that do not start and end on 16 bytes (an odd N) go through the same rings by whole 16-byte pieces of
// memory (kShift): piece j has the channels j * kN - shift and on.  The grid is a multiple of 8, so that all rows
// of a CTA have one shift, and a thread the same channels in each.  The first and the last piece of a row have
// channels of its neighbours, which are left out; those of the whole tensor's first and last row might
// reach over its ends, and are read by the channel.  (By the channel altogether 23778 x 1773 FP16 took 129 us
// forward and 252 backward, so 55 and 96.)
template <class T, bool kShift>
struct RowPieces {
  static constexpr int kN = Piece<T>::kN;
  int shift, count;   // channels before the row in its first piece; pieces of a row
  uint32_t in;        // which of the thread's channels there are
  __device__ __forceinline__ RowPieces(const LnParams& p, int tid, int threads) : shift(0), count(p.N / kN), in(0) {
    if (!kShift) return;
    shift = (int)((reinterpret_cast<uintptr_t>(p.x) / sizeof(T) + (uintptr_t)row_at(p, p.xs, blockIdx.x)) % kN);
    count = (shift + p.N + kN - 1) / kN;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int c = (tid + i / kN * threads) * kN - shift + i % kN;
      if (c >= 0 && c < p.N) in |= 1u << i;
    }
  }
  __device__ __forceinline__ bool head(const LnParams& p, int row) const { return kShift && shift > 0 && row == 0; }
  __device__ __forceinline__ bool tail(const LnParams& p, int row) const {
    return kShift && row == p.rows - 1 && (shift + p.N) % kN != 0;
  }
  // (one thread) bytes to come, and the row's pieces into its place
  __device__ __forceinline__ int bytes(const LnParams& p, int row) const {
    return (count - head(p, row) - tail(p, row)) * 16;
  }
  __device__ __forceinline__ void load(const LnParams& p, uint8_t* to, const T* at, int row, uint64_t* bar) const {
    bulk_load(to + (head(p, row) ? 16 : 0), at - shift + (head(p, row) ? kN : 0), bytes(p, row), bar);
  }
  // piece `j` of a row in shared memory; `at` is the row in global memory
  __device__ __forceinline__ uint4 read(const LnParams& p, const uint4* src, const T* at, int j, int row) const {
    if (j >= count) return make_uint4(0u, 0u, 0u, 0u);
    if (kShift && ((j == 0 && head(p, row)) || (j == count - 1 && tail(p, row)))) {
      Piece<T> t;
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        const int c = j * kN - shift + e;
        t.v[e] = at[min(max(c, 0), p.N - 1)];   // (channels that there are not are left out by the mask)
      }
      return *reinterpret_cast<uint4*>(&t);
    }
    return src[j];
  }
  // zeros for the channels that there are not
  __device__ __forceinline__ void mask(float* v, int i0) const {
    if (!kShift || ((in >> i0) & ((1u << kN) - 1)) == (1u << kN) - 1) return;
#pragma unroll
    for (int e = 0; e < kN; ++e) v[e] = (in >> (i0 + e)) & 1u ? v[e] : 0.0f;
  }
  __device__ __forceinline__ void weights(const LnParams& p, const void* w, int j, float other, float* out) const {
    if (!kShift) {
      load_weights<true, kN>(w, j * kN, other, p, out);
      return;
    }
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      const int c = j * kN - shift + e;
      out[e] = other;
      if (w == nullptr || c < 0 || c >= p.N) continue;
      if (p.w_type == kF32) out[e] = __ldg(reinterpret_cast<const float*>(w) + c);
      else if (p.w_type == kBF16) out[e] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(w)[c]);
      else out[e] = __half2float(reinterpret_cast<const __half*>(w)[c]);
    }
  }
  __device__ __forceinline__ void store(const LnParams& p, T* row, int j, const float* x) const {
    const int c = j * kN - shift;
    if (!kShift || (c >= 0 && c + kN <= p.N)) {
      store_piece<true, T>(row, c, x, p);
      return;
    }
    const uint4 raw = pack<T>(x);
    const Piece<T> t = *reinterpret_cast<const Piece<T>*>(&raw);
#pragma unroll
    for (int e = 0; e < kN; ++e)
      if (c + e >= 0 && c + e < p.N) row[c + e] = t.v[e];
  }
};

template <class T, bool kShift>
__global__ void __launch_bounds__(kShift ? 512 : 640) ln_fwd_ring_kernel(const LnParams p) {
  constexpr int kN = Piece<T>::kN, kValues = 16, kPieces = kValues / kN;
  extern __shared__ __align__(16) uint8_t rows_smem[];   // [2 turns][2 rows][N]
  __shared__ RowRing ring;
  __shared__ float scratch[2][32][2];
  const int tid = threadIdx.x, threads = blockDim.x;
  ring_init(ring);
  const RowPieces<T, kShift> pieces(p, tid, threads);
  float w[kValues], b[kValues];
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    pieces.weights(p, p.w, tid + k * threads, 1.0f, w + k * kN);
    pieces.weights(p, p.b, tid + k * threads, 0.0f, b + k * kN);
  }
  const float inv_n = 1.0f / (float)p.N;
  int issued = 0, turn = 0;
  // (thread 0) the rows of turn i: the CTA's rows 2 i and 2 i + 1
  auto issue = [&](int i) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const long long row = (long long)blockIdx.x + (2ll * i + r) * gridDim.x;
      if (row >= p.rows) return;
      const int slot = 2 * (i & 1) + r;
      mbar_arrive_expect_tx(&ring.full[slot], pieces.bytes(p, (int)row));
      if (withheld(issued++)) continue;
      pieces.load(p, rows_smem + slot * p.slot, reinterpret_cast<const T*>(p.x) + row_at(p, p.xs, (int)row), (int)row,
                  &ring.full[slot]);
    }
  };
  bool landed = true;   // all rows that were waited for
  if (tid == 0) {
    issue(0);
    issue(1);
  }
  for (int i = 0, row = blockIdx.x; row < p.rows; row += 2 * gridDim.x, ++i) {
    const bool two = row + (int)gridDim.x < p.rows;   // (the last turn may have one row)
    float v[2][kValues], sum[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int slot = 2 * (i & 1) + r;
      if (r == 0 || two) landed = ring_wait(ring, slot, i >> 1) && landed;
      const uint4* src = reinterpret_cast<const uint4*>(rows_smem + slot * p.slot);
      const int in_row = row + r * (int)gridDim.x;
      const T* x = reinterpret_cast<const T*>(p.x) + (kShift && (r == 0 || two) ? row_at(p, p.xs, in_row) : 0);
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int at = tid + k * threads;
        unpack<T>(r == 0 || two ? pieces.read(p, src, x, at, in_row) : make_uint4(0u, 0u, 0u, 0u), v[r] + k * kN);
        pieces.mask(v[r] + k * kN, k * kN);
      }
      float a[2] = {0.0f, 0.0f};
#pragma unroll
      for (int e = 0; e < kValues; e += 2) fadd2(a[0], a[1], a[0], a[1], v[r][e], v[r][e + 1]);
      sum[r] = a[0] + a[1];
    }
    row_sums<0>(sum, scratch, turn);
    if (tid == 0 && landed) issue(i + 2);   // (all threads have read this turn's rows: they met in row_sums)
    float sq[2], mean[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mean[r] = sum[r] * inv_n;
      float a[2] = {0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
#pragma unroll
        for (int e = k * kN; e < (k + 1) * kN; e += 2)
          fadd2(v[r][e], v[r][e + 1], v[r][e], v[r][e + 1], -mean[r], -mean[r]);
        if (!kShift && (tid + k * threads) * kN >= p.N) continue;
        pieces.mask(v[r] + k * kN, k * kN);
#pragma unroll
        for (int e = k * kN; e < (k + 1) * kN; e += 2)
          ffma2(a[0], a[1], v[r][e], v[r][e + 1], v[r][e], v[r][e + 1], a[0], a[1]);
      }
      sq[r] = a[0] + a[1];
    }
    row_sums<0>(sq, scratch, turn);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (r == 1 && !two) break;
      const int at = row + r * (int)gridDim.x;
      const float rstd = 1.0f / sqrtf(sq[r] * inv_n + p.eps);
      T* y = reinterpret_cast<T*>(p.y) + row_at(p, p.ys, at);
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        float out[kN];
#pragma unroll
        for (int e = 0; e < kN; e += 2) {
          const int a = k * kN + e;
          fmul2(out[e], out[e + 1], v[r][a], v[r][a + 1], rstd, rstd);
          ffma2(out[e], out[e + 1], out[e], out[e + 1], w[a], w[a + 1], b[a], b[a + 1]);
        }
        pieces.store(p, y, tid + k * threads, out);
      }
      if (tid == 0) {
        p.mean[at] = mean[r];
        p.rstd[at] = rstd;
      }
    }
  }
  if (tid == 0 && !landed)   // nothing may land in this CTA's shared memory after it has gone
    for (int n = issued > 4 ? issued - 4 : 0; n < issued; ++n)   // (the n-th row goes to slot n % 4)
      mbar_wait_teardown(&ring.full[n % 4], (n / 4) & 1);
}

// kMax = 640 (512 with kShift), or 1024 for the rows above 10240 channels, where the registers leave no
// room to hold the weights (12000 x 12288 FP32, with a row read again from the caches 781 us, so 343).
template <class T, int kMax, bool kShift>
__global__ void __launch_bounds__(kMax) ln_bwd_ring_kernel(const LnParams p) {
  constexpr int kValues = 16;
  constexpr bool kHold = kMax <= 640;
  constexpr int kN = Piece<T>::kN, kPieces = kValues / kN;
  extern __shared__ __align__(16) uint8_t rows_smem[];   // [ring][x and dy][N]
  __shared__ RowRing ring;
  __shared__ float scratch[2][32][2];
  const int tid = threadIdx.x, threads = blockDim.x, bytes = p.slot;
  ring_init(ring);
  const RowPieces<T, kShift> pieces(p, tid, threads);
  float w[kHold ? kValues : 1], dw[kValues] = {}, db[kValues] = {};
#pragma unroll
  for (int k = 0; k < (kHold ? kPieces : 0); ++k) pieces.weights(p, p.w, tid + k * threads, 1.0f, w + k * kN);
  const float inv_n = 1.0f / (float)p.N;
  auto place = [&](const Rows& r, int row) { return kHold ? row_in_ring(p, r, row) : row_at(p, r, row); };
  int issued = 0, turn = 0;
  auto issue = [&](long long row, int slot) {   // (thread 0)
    if (row >= p.rows) return;
    uint8_t* to = rows_smem + slot * 2 * bytes;
    uint64_t* bar = &ring.full[slot];
    mbar_arrive_expect_tx(bar, 2 * pieces.bytes(p, (int)row));
    if (withheld(issued++)) return;
    pieces.load(p, to, reinterpret_cast<const T*>(p.x) + place(p.xs, (int)row), (int)row, bar);
    pieces.load(p, to + bytes, reinterpret_cast<const T*>(p.dy) + place(p.dys, (int)row), (int)row, bar);
  };
  bool landed = true;   // all rows that were waited for
  if (tid == 0)
    for (int i = 0; i < p.ring; ++i) issue(blockIdx.x + (long long)i * gridDim.x, i);
  float next_mean = 0.0f, next_rstd = 0.0f;
  if ((int)blockIdx.x < p.rows) {
    next_mean = __ldg(p.mean + blockIdx.x);
    next_rstd = __ldg(p.rstd + blockIdx.x);
  }
  for (int row = blockIdx.x, i = 0, slot = 0, phase = 0; row < p.rows; row += gridDim.x, ++i) {
    const float m = next_mean, rs = next_rstd;
    if (row + (int)gridDim.x < p.rows) {
      next_mean = __ldg(p.mean + row + gridDim.x);
      next_rstd = __ldg(p.rstd + row + gridDim.x);
    }
    const uint4* sx = reinterpret_cast<const uint4*>(rows_smem + slot * 2 * bytes);
    const uint4* sd = reinterpret_cast<const uint4*>(rows_smem + slot * 2 * bytes + bytes);
    const T* const gx = reinterpret_cast<const T*>(p.x) + (kShift ? place(p.xs, row) : 0);
    const T* const gd = reinterpret_cast<const T*>(p.dy) + (kShift ? place(p.dys, row) : 0);
    landed = ring_wait(ring, slot, phase) && landed;
    float s[2], s0[2] = {0.0f, 0.0f}, s1[2] = {0.0f, 0.0f};   // sums of g and of g xhat
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int at = tid + k * threads;
      if (at >= pieces.count) continue;
      float x[kN], d[kN], lw[kHold ? 1 : kN];
      if (!kHold) pieces.weights(p, p.w, at, 1.0f, lw);
      const float* pw = kHold ? &w[kHold ? k * kN : 0] : lw;
      unpack<T>(pieces.read(p, sx, gx, at, row), x);
      unpack<T>(pieces.read(p, sd, gd, at, row), d);
      pieces.mask(x, k * kN);
      pieces.mask(d, k * kN);
#pragma unroll
      for (int e = 0; e < kN; e += 2) {
        const int a = k * kN + e;
        float xh[2], g[2];
        fadd2(xh[0], xh[1], x[e], x[e + 1], -m, -m);
        fmul2(xh[0], xh[1], xh[0], xh[1], rs, rs);
        fmul2(g[0], g[1], d[e], d[e + 1], pw[e], pw[e + 1]);
        ffma2(dw[a], dw[a + 1], d[e], d[e + 1], xh[0], xh[1], dw[a], dw[a + 1]);
        fadd2(db[a], db[a + 1], db[a], db[a + 1], d[e], d[e + 1]);
        fadd2(s0[0], s0[1], s0[0], s0[1], g[0], g[1]);
        ffma2(s1[0], s1[1], g[0], g[1], xh[0], xh[1], s1[0], s1[1]);
      }
    }
    s[0] = s0[0] + s0[1];
    s[1] = s1[0] + s1[1];
    row_sums<0>(s, scratch, turn);
    // (all threads have met: they are done with the row before this one, and its place is free)
    if (tid == 0 && i > 0 && landed) issue(row + (long long)(p.ring - 1) * gridDim.x, slot == 0 ? p.ring - 1 : slot - 1);
    const float m0 = -s[0] * inv_n, m1 = -s[1] * inv_n;
    T* dx = reinterpret_cast<T*>(p.dx) + place(p.dxs, row);
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int at = tid + k * threads;
      if (at >= pieces.count) continue;
      float x[kN], d[kN], out[kN], lw[kHold ? 1 : kN];
      if (!kHold) pieces.weights(p, p.w, at, 1.0f, lw);
      const float* pw = kHold ? &w[kHold ? k * kN : 0] : lw;
      unpack<T>(pieces.read(p, sx, gx, at, row), x);
      unpack<T>(pieces.read(p, sd, gd, at, row), d);
      pieces.mask(x, k * kN);
      pieces.mask(d, k * kN);
#pragma unroll
      for (int e = 0; e < kN; e += 2) {
        float xh[2], g[2];
        fadd2(xh[0], xh[1], x[e], x[e + 1], -m, -m);
        fmul2(xh[0], xh[1], xh[0], xh[1], rs, rs);
        fmul2(g[0], g[1], d[e], d[e + 1], pw[e], pw[e + 1]);
        ffma2(g[0], g[1], xh[0], xh[1], m1, m1, g[0], g[1]);
        fadd2(g[0], g[1], g[0], g[1], m0, m0);
        fmul2(out[e], out[e + 1], g[0], g[1], rs, rs);
      }
      pieces.store(p, dx, at, out);
    }
    if (++slot == p.ring) {
      slot = 0;
      ++phase;
    }
  }
  if (p.partial != nullptr) {   // this CTA's sums: [2][CTAs][N]
    float* const to_w = p.partial + (long long)blockIdx.x * p.N;
    float* const to_b = p.partial + ((long long)gridDim.x + blockIdx.x) * p.N;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int c = (tid + k * threads) * kN - pieces.shift;
      if (kShift) {
#pragma unroll
        for (int e = 0; e < kN; ++e)
          if ((pieces.in >> (k * kN + e)) & 1u) {
            to_w[c + e] = dw[k * kN + e];
            to_b[c + e] = db[k * kN + e];
          }
        continue;
      }
      if (c >= p.N) continue;
#pragma unroll
      for (int e = 0; e < kN; e += 4) {
        const int a = k * kN + e;
        *reinterpret_cast<float4*>(to_w + c + e) = make_float4(dw[a], dw[a + 1], dw[a + 2], dw[a + 3]);
        *reinterpret_cast<float4*>(to_b + c + e) = make_float4(db[a], db[a + 1], db[a + 2], db[a + 3]);
      }
    }
  }
  if (tid == 0 && !landed)
    for (int i = issued > p.ring ? issued - p.ring : 0; i < issued; ++i)
      mbar_wait_teardown(&ring.full[i % p.ring], (i / p.ring) & 1);
}

// dw and db from the CTAs' sums: a block takes 32 channels of one of them, its 32 warps every 32nd CTA.
__global__ void __launch_bounds__(1024) ln_grad_kernel(const float* partial, int n_parts, int N, void* dw, void* db,
                                                       int type) {
  __shared__ float s[32][33];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const float* part = partial + (long long)blockIdx.y * n_parts * N;
  float a = 0.0f;
  if (c < N)
    for (int i = warp; i < n_parts; i += 32) a += part[(long long)i * N + c];
  s[warp][lane] = a;
  __syncthreads();
  float v = s[lane][warp];   // channel `warp` of the block's
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int out = blockIdx.x * 32 + warp;
  if (lane != 0 || out >= N) return;
  void* to = blockIdx.y == 0 ? dw : db;
  if (type == kF32) reinterpret_cast<float*>(to)[out] = v;
  else if (type == kBF16) reinterpret_cast<__nv_bfloat16*>(to)[out] = __float2bfloat16_rn(v);
  else reinterpret_cast<__half*>(to)[out] = __float2half_rn(v);
}

// Rows of a warp under way ahead of the one worked on: as many as the registers hold.
template <class T, bool kVec, bool kBackward>
constexpr int kWarpRows = !kVec ? 1 : sizeof(T) == 2 ? 3 : kBackward ? 2 : 1;
struct Shape {
  int lanes, threads, ctas;
  bool wide;   // 32 channels a thread
};
// The sums' place in the workspace is sized by this too: it goes by the sizes alone.
Shape shape_of(int rows, int N, bool backward) {
  Shape s = {};
  constexpr int kSms = 152;
  // 16 channels a lane, in the backward 8 (where the sums take two more registers a channel)
  const int a_lane = backward ? 8 : 16;
  if (N <= 32 * a_lane) {
    s.lanes = N <= 4 * a_lane ? 4 : N <= 8 * a_lane ? 8 : N <= 16 * a_lane ? 16 : 32;
    s.threads = 256;
    const int per = s.threads / s.lanes;
    s.ctas = (rows + per - 1) / per;
  } else {
    s.wide = N > 8192;
    const int per = s.wide && !backward ? 32 : 16;   // (the backward's wide rows: see below)
    s.threads = ((N + per - 1) / per + 31) / 32 * 32;
    s.ctas = rows;
  }
  // CTAs that an SM holds by their registers (what the launch bounds allow a thread)
  const int regs = backward && s.wide ? 64 : s.wide ? 128 : 96;
  int per_sm = 65536 / (regs * s.threads);
  if (per_sm < 1) per_sm = 1;
  const int cap = kSms * per_sm;
  if (s.ctas > cap) s.ctas = cap;
  if (s.ctas < 1) s.ctas = 1;
  return s;
}

size_t bwd_smem(const Shape& s, int N) {
  if (s.lanes > 0) return (size_t)(s.threads / 32) * N * sizeof(float);   // at most 8 KB
  return s.wide ? (size_t)64 * s.threads * sizeof(float) : 0;             // at most 128 KB
}

template <class T, bool kVec, int kLanes, int kValues, bool kBackward>
cudaError_t launch_one(const LnParams& p, const Shape& s, cudaStream_t stream) {
  const dim3 grid((unsigned)s.ctas);
  if constexpr (kBackward) {
    auto* kernel = ln_bwd_kernel<T, kVec, kLanes, kValues, (kLanes > 0 ? kWarpRows<T, kVec, true> : 1), (kLanes > 0 ? 640 : 512)>;
    if constexpr (kValues == 32) {
      static ContextOnce attr_done;
      const cudaError_t e = attr_done.run([&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(64 * 512 * sizeof(float)));
      });
      if (e != cudaSuccess) return e;
    }
    return launch_dependent(kernel, grid, s.threads, bwd_smem(s, p.N), stream, p);
  } else {
    return launch_dependent(ln_fwd_kernel<T, kVec, kLanes, kValues, (kLanes > 0 ? kWarpRows<T, kVec, false> : 1), (kValues == 32 ? 512 : 640)>, grid, s.threads, 0,
                            stream, p);
  }
}
constexpr int kRingBytes = 220 * 1024;
// kShift: rows by pieces of memory (RowPieces); false where a CTA has not the threads for them, or the ring not the
// room for two rows.
template <class T, bool kShift, bool kBackward>
bool fits_ring(const LnParams& p, Shape& s, LnParams& q) {
  constexpr int kN = 16 / (int)sizeof(T);
  const int pieces = kShift ? (p.N + 2 * (kN - 1)) / kN : p.N / kN;   // at most
  if (!kShift && s.wide && p.N <= 16 * 640) {   // a CTA of up to 640 threads will do
    s.wide = false;
    s.threads = ((p.N + 15) / 16 + 31) / 32 * 32;
  }
  if (s.lanes > 0 || (s.wide && (kShift || !kBackward || 4 * 16 * pieces > kRingBytes))) return false;
  while (s.threads * 16 < pieces * kN) s.threads += 32;
  if (s.threads > (s.wide ? 1024 : kShift ? 512 : 640)) return false;
  q = p;
  q.slot = 16 * pieces;
  return true;
}
template <class T, bool kShift, bool kBackward>
cudaError_t launch_ring(LnParams& q, const Shape& s, cudaStream_t stream) {
  static ContextOnce attr_done[2];
  auto* kernel = !kBackward ? ln_fwd_ring_kernel<T, kShift> : ln_bwd_ring_kernel<T, kShift ? 512 : 640, kShift>;
  if constexpr (kBackward && !kShift)
    if (s.wide) kernel = ln_bwd_ring_kernel<T, 1024, false>;
  const cudaError_t e = attr_done[s.wide].run([&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  });
  if (e != cudaSuccess) return e;
  const size_t row = q.slot;
  const int per_sm = s.wide ? 1 : 65536 / (96 * s.threads);
  q.ring = 6 * row * per_sm <= (size_t)kRingBytes ? 3 : 2;
  g_launched.store(true, std::memory_order_relaxed);
  return launch_dependent(kernel, dim3((unsigned)s.ctas), s.threads, kBackward ? 2 * q.ring * row : 4 * row, stream, q);
}
// shift: all rows of a tensor are equally far apart, and all tensors start at one distance from 16 bytes.  s: its CTAs
// become those that are launched.
template <class T, bool kVec, bool kBackward>
cudaError_t launch_typed(const LnParams& p, Shape& s, bool shift, cudaStream_t stream) {
  LnParams q;
  Shape t = s;
  if (kVec && fits_ring<T, false, kBackward>(p, t, q)) return launch_ring<T, false, kBackward>(q, t, stream);
  // (FP32 backward: by the channel, 29604 x 6345 430 us and 529 so)
  if constexpr (!kVec && !(kBackward && sizeof(T) == 4)) {
    if (!kBackward && t.lanes == 32) {   // 16 channels a lane: a warp of its own for each row
      t.lanes = 0;
      t.threads = 32;
      t.ctas = p.rows;
    }
    if (shift && fits_ring<T, true, kBackward>(p, t, q)) {
      // 128 registers a thread.  (A grid that is no multiple of 8 has no second row for any CTA.)
      const int cap = 152 * (65536 / (128 * t.threads));
      if (t.ctas > cap) t.ctas = cap;
      s.ctas = t.ctas;
      return launch_ring<T, true, kBackward>(q, t, stream);
    }
  }
  switch (s.lanes) {
    case 4: return launch_one<T, kVec, 4, kBackward ? 8 : 16, kBackward>(p, s, stream);
    case 8: return launch_one<T, kVec, 8, kBackward ? 8 : 16, kBackward>(p, s, stream);
    case 16: return launch_one<T, kVec, 16, kBackward ? 8 : 16, kBackward>(p, s, stream);
    case 32: return launch_one<T, kVec, 32, kBackward ? 8 : 16, kBackward>(p, s, stream);
  }
  if (s.wide) {   // 32 channels a thread, in the backward too
    t = s;
    t.threads = ((p.N + 31) / 32 + 31) / 32 * 32;
    return launch_one<T, kVec, 0, 32, kBackward>(p, t, stream);
  }
  return launch_one<T, false, 0, 16, kBackward>(p, s, stream);
}
template <bool kBackward>
cudaError_t launch_any(const LnParams& p, Shape& s, int type, bool vec, bool shift, cudaStream_t stream) {
  if (type == kF32)
    return vec ? launch_typed<float, true, kBackward>(p, s, shift, stream)
               : launch_typed<float, false, kBackward>(p, s, shift, stream);
  if (type == kBF16)
    return vec ? launch_typed<__nv_bfloat16, true, kBackward>(p, s, shift, stream)
               : launch_typed<__nv_bfloat16, false, kBackward>(p, s, shift, stream);
  return vec ? launch_typed<__half, true, kBackward>(p, s, shift, stream)
             : launch_typed<__half, false, kBackward>(p, s, shift, stream);
}

LnParams params_of(const LayerNormArgs& a) {
  LnParams p = {};
  p.x = a.x;
  p.w = a.w;
  p.b = a.b;
  p.mean = a.mean;
  p.rstd = a.rstd;
  p.rows = a.B * a.S * a.H;
  p.S = make_div(a.S);
  p.H = make_div(a.H);
  p.N = a.N;
  p.eps = a.eps;
  p.w_type = a.w_type;
  return p;
}
bool whole(const void* ptr, const long long* str, const LayerNormArgs& a) {
  const int n = a.type == kF32 ? 4 : 8;
  return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0 && (a.B == 1 || str[0] % n == 0) && (a.S == 1 || str[1] % n == 0) &&
         (a.H == 1 || str[2] % n == 0);
}
// Whether two tensors' rows start at the same distance from 16 bytes, and a's rows do not overlap.
bool same_shift(const void* a, const Rows& ra, const void* b, const Rows& rb, const LayerNormArgs& args) {
  const int n = args.type == kF32 ? 4 : 8;
  return ra.even && rb.even && ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) & 15u) == 0 &&
         (ra.str[2] - rb.str[2]) % n == 0 && ra.str[2] >= args.N;
}
void set_rows(Rows& r, const long long* str, const LayerNormArgs& a) {
  for (int i = 0; i < 3; ++i) r.str[i] = str[i];
  // (the stride of a dimension of one says nothing)
  if (a.H == 1) r.str[2] = a.S > 1 ? r.str[1] : r.str[0];
  r.even = (a.H == 1 || a.S == 1 || r.str[1] == a.H * r.str[2]) &&
           (a.B == 1 || (a.H == 1 && a.S == 1) || r.str[0] == (long long)a.S * a.H * r.str[2]);
}

}  // namespace

size_t layer_norm_bwd_workspace(int rows, int N) { return (size_t)2 * shape_of(rows, N, true).ctas * N * sizeof(float); }

cudaError_t launch_layer_norm_fwd(const LayerNormArgs& a, void* y, const long long y_str[3], cudaStream_t stream) {
  LnParams p = params_of(a);
  p.y = y;
  set_rows(p.xs, a.x_str, a);
  set_rows(p.ys, y_str, a);
  const bool w16 = ((reinterpret_cast<uintptr_t>(a.w) | reinterpret_cast<uintptr_t>(a.b)) & 15u) == 0;
  const bool vec = a.N % (a.type == kF32 ? 4 : 8) == 0 && whole(a.x, a.x_str, a) && whole(y, y_str, a) && w16;
  const bool shift = same_shift(a.x, p.xs, y, p.ys, a);
  Shape s = shape_of(p.rows, p.N, false);
  return launch_any<false>(p, s, a.type, vec, shift, stream);
}

cudaError_t launch_layer_norm_bwd(const LayerNormArgs& a, const void* dy, const long long dy_str[3], void* dx,
                                  const long long dx_str[3], void* dw, void* db, float* workspace,
                                  cudaStream_t stream) {
  LnParams p = params_of(a);
  p.dy = dy;
  p.dx = dx;
  set_rows(p.xs, a.x_str, a);
  set_rows(p.dys, dy_str, a);
  set_rows(p.dxs, dx_str, a);
  const bool w16 = (reinterpret_cast<uintptr_t>(a.w) & 15u) == 0;
  const bool vec = a.N % (a.type == kF32 ? 4 : 8) == 0 && whole(a.x, a.x_str, a) && whole(dy, dy_str, a) &&
                   whole(dx, dx_str, a) && w16;
  p.partial = dw != nullptr ? workspace : nullptr;
  Shape s = shape_of(p.rows, p.N, true);
  const bool shift = same_shift(a.x, p.xs, dy, p.dys, a) && same_shift(dy, p.dys, dx, p.dxs, a);
  cudaError_t e = launch_any<true>(p, s, a.type, vec, shift, stream);
  if (e != cudaSuccess || dw == nullptr) return e;
  return launch_dependent(ln_grad_kernel, dim3((unsigned)(p.N + 31) / 32, 2), 1024, 0, stream,
                          static_cast<const float*>(workspace), s.ctas, p.N, dw, db, a.w_type);
}

static const bool err_reader_added =
    add_err_reader([](uint32_t* out) { return read_and_clear_err(g_err_norm, g_launched, out); });

}  // namespace sa
