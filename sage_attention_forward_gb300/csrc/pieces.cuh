// 16-byte pieces of rows of BF16, FP16 or FP32 values and the 32-bit values that they stand for.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace sa {

template <class T>
struct Piece {   // 16 bytes
  static constexpr int kN = 16 / sizeof(T);
  T v[kN];
};
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

}  // namespace sa
