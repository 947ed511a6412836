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
// Rows of up to 512 channels take 4 to 32 lanes of a warp, 16 channels a lane; longer ones a CTA,
// 16 channels a thread (32 above 8192).  CTAs walk over the rows: while a row is worked on the
// next one's loads are under way, and in the backward pass a thread keeps the sums of dw and db
// of its own channels in registers over all of its rows.  Each CTA writes its sums once to the
// workspace, and a second kernel adds them up, in one fixed order: no atomics, the same bits every time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "ptx.cuh"

namespace sa {
namespace {

struct Rows {
  long long str[3];   // element strides (b, s, h)
};
struct LnParams {
  const void *x, *dy, *w, *b;
  void *y, *dx;
  float *mean, *rstd;             // outputs of the forward, inputs of the backward
  Rows xs, ys, dys, dxs;
  int rows, S, H, N;
  float eps;
  int w_type;                     // type of w and b
  float* partial;                 // backward: [2][CTAs][N] sums of dw and db, or nullptr
};

__device__ __forceinline__ long long row_at(const LnParams& p, const Rows& r, int row) {
  const int h = row % p.H, bs = row / p.H;
  return (long long)(bs / p.S) * r.str[0] + (long long)(bs % p.S) * r.str[1] + (long long)h * r.str[2];
}

template <class T>
struct Piece {   // 16 bytes
  static constexpr int kN = 16 / sizeof(T);
  T v[kN];
};
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float(float x) { return x; }
template <>
__device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }

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
template <bool kVec, class T>
__device__ __forceinline__ void store_piece(T* row, int c, const float* x, const LnParams& p) {
  if (c >= p.N) return;
  Piece<T> t;
#pragma unroll
  for (int e = 0; e < Piece<T>::kN; ++e) t.v[e] = from_float<T>(x[e]);
  if (kVec) {
    __stcs(reinterpret_cast<uint4*>(row + c), *reinterpret_cast<uint4*>(&t));
    return;
  }
#pragma unroll
  for (int e = 0; e < Piece<T>::kN; ++e)
    if (c + e < p.N) row[c + e] = t.v[e];
}
template <class T>
__device__ __forceinline__ void unpack(const uint4& raw, float* x) {
  const Piece<T> t = *reinterpret_cast<const Piece<T>*>(&raw);
#pragma unroll
  for (int e = 0; e < Piece<T>::kN; ++e) x[e] = to_float(t.v[e]);
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
template <class T, bool kVec, int kLanes, int kValues, int kMax>
__global__ void __launch_bounds__(kMax) ln_fwd_kernel(const LnParams p) {
  using S = Spread<kLanes>;
  constexpr int kN = Piece<T>::kN, kPieces = kValues / kN;
  __shared__ float scratch[2][32][2];
  griddep_wait();
  const int lane = S::lane(), step = S::step();
  int row = S::first(), turn = 0;
  const float inv_n = 1.0f / (float)p.N;
  uint4 raw[kPieces];
  auto load = [&](int r) {
    const T* x = reinterpret_cast<const T*>(p.x) + (r < p.rows ? row_at(p, p.xs, r) : 0);
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
      raw[k] = r < p.rows ? load_piece<kVec, T>(x, (lane + k * S::width()) * kN, p) : make_uint4(0u, 0u, 0u, 0u);
  };
  load(row);
  // (a warp's rows are consecutive: its lanes leave the loop together but for the last rows, whose
  // idle lanes work on zeros and store nothing)
  for (int base = S::kWarp ? row - (int)((threadIdx.x & 31) / (S::kWarp ? kLanes : 1)) : row; base < p.rows;
       base += step, row += step) {
    float v[kValues];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) unpack<T>(raw[k], v + k * kN);
    load(row + step);
    float sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < kValues; ++i) sum[0] += v[i];   // (channels past N are 0)
    row_sums<kLanes>(sum, scratch, turn);
    const float mean = sum[0] * inv_n;
    float sq[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        const bool in = (lane + k * S::width()) * kN + e < p.N;
        v[k * kN + e] = in ? v[k * kN + e] - mean : 0.0f;
        sq[0] = fmaf(v[k * kN + e], v[k * kN + e], sq[0]);
      }
    row_sums<kLanes>(sq, scratch, turn);
    const float rstd = 1.0f / sqrtf(sq[0] * inv_n + p.eps);
    if (row < p.rows) {
      T* y = reinterpret_cast<T*>(p.y) + row_at(p, p.ys, row);
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int c = (lane + k * S::width()) * kN;
        float ww[kN], bb[kN], out[kN];
        load_weights<kVec, kN>(p.w, c, 1.0f, p, ww);   // (from L1: registers for them would halve the rows in flight)
        load_weights<kVec, kN>(p.b, c, 0.0f, p, bb);
#pragma unroll
        for (int e = 0; e < kN; ++e) out[e] = fmaf(v[k * kN + e] * rstd, ww[e], bb[e]);
        store_piece<kVec, T>(y, c, out, p);
      }
      if (lane == 0) {
        p.mean[row] = mean;
        p.rstd[row] = rstd;
      }
    }
  }
}

template <class T, bool kVec, int kLanes, int kValues, int kMax>
__global__ void __launch_bounds__(kMax) ln_bwd_kernel(const LnParams p) {
  using S = Spread<kLanes>;
  constexpr int kN = Piece<T>::kN, kPieces = kValues / kN;
  // the next row's loads are under way while a row is worked on; not with 32 channels a thread,
  // where the registers do not reach
  constexpr bool kAhead = kValues <= 16, kWide = !kAhead;
  __shared__ float scratch[2][32][2];
  // a warp's rows: [warps][N], to add the warps up.  32 channels a thread: the thread's sums of dw and
  // db, [2][32][threads], for which there are no registers.
  extern __shared__ float sums[];
  griddep_wait();
  const int lane = S::lane(), step = S::step();
  int row = S::first(), turn = 0;
  const float inv_n = 1.0f / (float)p.N;
  float dw[kWide ? 1 : kValues] = {}, db[kWide ? 1 : kValues] = {};
  float* const wide = sums + threadIdx.x;
  if (kWide)
    for (int i = 0; i < 2 * kValues; ++i) wide[i * blockDim.x] = 0.0f;
  uint4 rx[kPieces], rd[kPieces];
  float mean, rstd;
  auto load = [&](int r) {
    const bool in = r < p.rows;
    const T* x = reinterpret_cast<const T*>(p.x) + (in ? row_at(p, p.xs, r) : 0);
    const T* d = reinterpret_cast<const T*>(p.dy) + (in ? row_at(p, p.dys, r) : 0);
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int c = (lane + k * S::width()) * kN;
      rx[k] = in ? load_piece<kVec, T>(x, c, p) : make_uint4(0u, 0u, 0u, 0u);
      rd[k] = in ? load_piece<kVec, T>(d, c, p) : make_uint4(0u, 0u, 0u, 0u);
    }
    mean = in ? __ldg(p.mean + r) : 0.0f;
    rstd = in ? __ldg(p.rstd + r) : 0.0f;
  };
  load(row);
  for (int base = S::kWarp ? row - (int)((threadIdx.x & 31) / (S::kWarp ? kLanes : 1)) : row; base < p.rows;
       base += step, row += step) {
    uint4 cx[kPieces], cd[kPieces];
    const float m = mean, rs = rstd;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      cx[k] = rx[k];
      cd[k] = rd[k];
    }
    if (kAhead) load(row + step);
    float s[2] = {0.0f, 0.0f};   // of g and of g xhat
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int c = (lane + k * S::width()) * kN;
      float x[kN], d[kN], ww[kN];
      unpack<T>(cx[k], x);
      unpack<T>(cd[k], d);
      load_weights<kVec, kN>(p.w, c, 1.0f, p, ww);
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        const float xh = (x[e] - m) * rs;      // (where there is no channel dy is 0)
        const float g = d[e] * ww[e];
        if (kWide) {
          wide[(k * kN + e) * blockDim.x] += d[e] * xh;
          wide[(kValues + k * kN + e) * blockDim.x] += d[e];
        } else {
          float &a = dw[kWide ? 0 : k * kN + e], &b = db[kWide ? 0 : k * kN + e];
          a = fmaf(d[e], xh, a);
          b += d[e];
        }
        s[0] += g;
        s[1] = fmaf(g, xh, s[1]);
      }
    }
    row_sums<kLanes>(s, scratch, turn);
    const float s0 = s[0] * inv_n, s1 = s[1] * inv_n;
    if (row < p.rows) {
      T* dx = reinterpret_cast<T*>(p.dx) + row_at(p, p.dxs, row);
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int c = (lane + k * S::width()) * kN;
        float x[kN], d[kN], ww[kN], out[kN];
        unpack<T>(cx[k], x);
        unpack<T>(cd[k], d);
        load_weights<kVec, kN>(p.w, c, 1.0f, p, ww);
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const float xh = (x[e] - m) * rs;
          const float g = d[e] * ww[e];
          out[e] = rs * (g - s0 - xh * s1);
        }
        store_piece<kVec, T>(dx, c, out, p);
      }
    }
    if (!kAhead) load(row + step);
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

constexpr int kBwdMax = 512;   // threads that the backward's registers are sized for
struct Shape {
  int lanes, threads, ctas;
  bool wide;   // 32 channels a thread
};
// The sums' place in the workspace is sized by this too: it goes by the sizes alone.
Shape shape_of(int rows, int N, bool backward) {
  Shape s = {};
  constexpr int kSms = 152;
  if (N <= 512) {
    s.lanes = N <= 64 ? 4 : N <= 128 ? 8 : N <= 256 ? 16 : 32;
    s.threads = 256;
    const int per = s.threads / s.lanes;
    s.ctas = (rows + per - 1) / per;
  } else {
    s.wide = N > 8192;
    const int per = s.wide ? 32 : 16;
    s.threads = ((N + per - 1) / per + 31) / 32 * 32;
    s.ctas = rows;
  }
  const int per_sm = 2048 / s.threads;   // (what the registers leave is fewer)
  const int cap = kSms * (backward ? (s.lanes ? 4 : per_sm < 2 ? 1 : per_sm < 8 ? per_sm / 2 : 4) : per_sm);
  if (s.ctas > cap) s.ctas = cap;
  if (s.ctas < 1) s.ctas = 1;
  return s;
}

size_t bwd_smem(const Shape& s, int N) {
  if (s.lanes > 0) return (size_t)(s.threads / 32) * N * sizeof(float);   // at most 16 KB
  return s.wide ? (size_t)64 * s.threads * sizeof(float) : 0;             // at most 128 KB
}

template <class T, bool kVec, int kLanes, int kValues, bool kBackward>
cudaError_t launch_one(const LnParams& p, const Shape& s, cudaStream_t stream) {
  const dim3 grid((unsigned)s.ctas);
  if constexpr (kBackward) {
    auto* kernel = ln_bwd_kernel<T, kVec, kLanes, kValues, kBwdMax>;
    if constexpr (kValues == 32) {
      static ContextOnce attr_done;
      const cudaError_t e = attr_done.run([&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(64 * 512 * sizeof(float)));
      });
      if (e != cudaSuccess) return e;
    }
    return launch_dependent(kernel, grid, s.threads, bwd_smem(s, p.N), stream, p);
  } else {
    return launch_dependent(ln_fwd_kernel<T, kVec, kLanes, kValues, kValues == 32 ? 512 : 1024>, grid, s.threads, 0,
                            stream, p);
  }
}
template <class T, bool kVec, bool kBackward>
cudaError_t launch_typed(const LnParams& p, const Shape& s, cudaStream_t stream) {
  switch (s.lanes) {
    case 4: return launch_one<T, kVec, 4, 16, kBackward>(p, s, stream);
    case 8: return launch_one<T, kVec, 8, 16, kBackward>(p, s, stream);
    case 16: return launch_one<T, kVec, 16, 16, kBackward>(p, s, stream);
    case 32: return launch_one<T, kVec, 32, 16, kBackward>(p, s, stream);
  }
  return s.wide ? launch_one<T, kVec, 0, 32, kBackward>(p, s, stream)
                : launch_one<T, kVec, 0, 16, kBackward>(p, s, stream);
}
template <bool kBackward>
cudaError_t launch_any(const LnParams& p, const Shape& s, int type, bool vec, cudaStream_t stream) {
  if (type == kF32) return vec ? launch_typed<float, true, kBackward>(p, s, stream) : launch_typed<float, false, kBackward>(p, s, stream);
  if (type == kBF16)
    return vec ? launch_typed<__nv_bfloat16, true, kBackward>(p, s, stream)
               : launch_typed<__nv_bfloat16, false, kBackward>(p, s, stream);
  return vec ? launch_typed<__half, true, kBackward>(p, s, stream) : launch_typed<__half, false, kBackward>(p, s, stream);
}

LnParams params_of(const LayerNormArgs& a) {
  LnParams p = {};
  p.x = a.x;
  p.w = a.w;
  p.b = a.b;
  p.mean = a.mean;
  p.rstd = a.rstd;
  p.rows = a.B * a.S * a.H;
  p.S = a.S;
  p.H = a.H;
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
void set_rows(Rows& r, const long long* str) {
  for (int i = 0; i < 3; ++i) r.str[i] = str[i];
}

}  // namespace

size_t layer_norm_bwd_workspace(int rows, int N) { return (size_t)2 * shape_of(rows, N, true).ctas * N * sizeof(float); }

cudaError_t launch_layer_norm_fwd(const LayerNormArgs& a, void* y, const long long y_str[3], cudaStream_t stream) {
  LnParams p = params_of(a);
  p.y = y;
  set_rows(p.xs, a.x_str);
  set_rows(p.ys, y_str);
  const bool w16 = ((reinterpret_cast<uintptr_t>(a.w) | reinterpret_cast<uintptr_t>(a.b)) & 15u) == 0;
  const bool vec = a.N % (a.type == kF32 ? 4 : 8) == 0 && whole(a.x, a.x_str, a) && whole(y, y_str, a) && w16;
  return launch_any<false>(p, shape_of(p.rows, p.N, false), a.type, vec, stream);
}

cudaError_t launch_layer_norm_bwd(const LayerNormArgs& a, const void* dy, const long long dy_str[3], void* dx,
                                  const long long dx_str[3], void* dw, void* db, float* workspace,
                                  cudaStream_t stream) {
  LnParams p = params_of(a);
  p.dy = dy;
  p.dx = dx;
  set_rows(p.xs, a.x_str);
  set_rows(p.dys, dy_str);
  set_rows(p.dxs, dx_str);
  const bool w16 = (reinterpret_cast<uintptr_t>(a.w) & 15u) == 0;
  const bool vec = a.N % (a.type == kF32 ? 4 : 8) == 0 && whole(a.x, a.x_str, a) && whole(dy, dy_str, a) &&
                   whole(dx, dx_str, a) && w16;
  p.partial = dw != nullptr ? workspace : nullptr;
  const Shape s = shape_of(p.rows, p.N, true);
  cudaError_t e = launch_any<true>(p, s, a.type, vec, stream);
  if (e != cudaSuccess || dw == nullptr) return e;
  return launch_dependent(ln_grad_kernel, dim3((unsigned)(p.N + 31) / 32, 2), 1024, 0, stream,
                          static_cast<const float*>(workspace), s.ctas, p.N, dw, db, a.w_type);
}

}  // namespace sa
