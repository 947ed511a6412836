// Writing to and reading from the K/V cache in 4 bits, sm_103a.
//
//   scale = -x_ext / 8 for each 32 channels of a token and head, x_ext the value of largest magnitude (exact in BF16)
//   code  = clamp(rint(x / scale), -8, 7), ties to even: x_ext itself has code -8
//
// Both are bound by memory (656 bytes a token and head in each direction).  A warp takes one record: half of it works on a
// token's K, half on its V, eight channels a lane, four lanes a group.  Several tokens' loads are under way together; the
// record is put together in shared memory and leaves (or arrives) in 16-byte pieces where it is whole, otherwise by the
// bytes of its tokens, so that two calls may fill one record.
#include <cuda_runtime.h>

#include "kv4.cuh"
#include "pieces.cuh"

namespace sa {
namespace {

constexpr int kWarps = 8;
constexpr int kAhead = 4;   // tokens whose loads are under way

struct CacheParams {
  KvPages pages;
  const void *k_in, *v_in;
  void *k_out, *v_out;
  long long k_str[3], v_str[3];   // element strides (b, s, h)
  const int *start, *count;       // [B]; count may be nullptr: S
  int B, S;
  Div heads, tiles;               // records that S tokens can touch
};

// What a warp works on: tokens [lo, hi) of tile `tile` of request b are the call's tokens from `first` on.
struct Work {
  int b, head, tile, lo, hi;
  long long first;   // the call's token at place 0 of the tile (may be negative)
  int n;             // the request's tokens in this call
  bool any;
};
__device__ __forceinline__ Work work_of(const CacheParams& p, int unit) {
  Work w;
  const int bh = div_by(unit, p.tiles), k = unit - bh * (int)p.tiles.d;
  w.b = div_by(bh, p.heads);
  w.head = bh - w.b * (int)p.heads.d;
  w.any = false;
  if (w.b >= p.B) return w;
  const int start = __ldg(p.start + w.b);
  w.n = p.count != nullptr ? min(max(__ldg(p.count + w.b), 0), p.S) : p.S;
  const long long tile = (long long)(start >> 4) + k;   // (start >> 4 rounds down)
  w.first = tile * kKvTile - start;
  w.lo = (int)max(0ll, -w.first);
  w.hi = (int)min((long long)kKvTile, (long long)p.S - w.first);
  w.any = w.lo < w.hi;
  w.tile = tile < 0 || tile > 0x7fffffff ? -1 : (int)tile;
  return w;
}

// Eight codes of one lane, bits 4 i.
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], float inv) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // x / scale is a quotient of two 8-bit significands: half an integer, or at least 2^-10 from one.  x inv is off by less than
    // 2^-18, so that in steps of 2^-11 (6144 added) halves are exact again and no other quotient becomes one; then the sum with
    // 1.5 2^23 + 8 rounds to even, and the integer stands in its low bits.
    const float q = fminf(fmaf(x[i], inv, 6144.0f), 6144.0f + 7.0f);
    const uint32_t c = __float_as_uint(q + (12582912.0f + 8.0f - 6144.0f));
    out = c * (1u << (4 * i)) + out;
  }
  constexpr uint32_t kMagic = 0x4b400000u;   // bits of 1.5 2^23, in `out` once for every code
  return out - kMagic * 0x11111111u;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// The value of largest magnitude of a group (four lanes' eight BF16 values each), the positive one of two.
__device__ __forceinline__ float extreme(const uint4& raw) {
  const uint32_t top = max2(max2(raw.x, raw.y), max2(raw.z, raw.w));
  const uint32_t low = min2(min2(raw.x, raw.y), min2(raw.z, raw.w)) ^ 0x80008000u;
  uint32_t both = max2(__byte_perm(top, low, 0x5410), __byte_perm(top, low, 0x7632));   // largest, and the smallest negated
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) both = max2(both, __shfl_xor_sync(0xffffffffu, both, o));
  const float hi = __uint_as_float(both << 16), lo = __uint_as_float(both & 0xffff0000u);
  return hi >= lo ? hi : -lo;
}

__global__ void __launch_bounds__(kWarps * 32) kv4_write_kernel(const __grid_constant__ CacheParams p) {
  __shared__ __align__(16) unsigned char tiles[kWarps][kKvRecord];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Work w = work_of(p, blockIdx.x * kWarps + warp);
  if (!w.any || w.tile < 0) return;
  const int hi = (int)min((long long)w.hi, w.n - w.first);
  const int page = kv_page(p.pages, w.b, w.tile);
  if (page < 0 || w.lo >= hi) return;
  unsigned char* const tile = tiles[warp];
  const bool is_v = lane >= 16;
  const int g = (lane & 15) >> 2, t = lane & 3;   // channels 32 g + 8 t
  const __nv_bfloat16* const in =
      reinterpret_cast<const __nv_bfloat16*>(is_v ? p.v_in : p.k_in) + 32 * g + 8 * t +
      (is_v ? w.b * p.v_str[0] + w.head * p.v_str[2] : w.b * p.k_str[0] + w.head * p.k_str[2]);
  const long long step = is_v ? p.v_str[1] : p.k_str[1];
  for (int j0 = w.lo; j0 < hi; j0 += kAhead) {
    uint4 raw[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (j0 + u < hi) raw[u] = __ldcs(reinterpret_cast<const uint4*>(in + (w.first + j0 + u) * step));
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = j0 + u;
      if (j >= hi) break;
      const float ext = extreme(raw[u]);
      const bool none = fabsf(ext) < 0x1p-100f;
      const float scale = none ? 0.0f : ext * -0.125f;
      float x[8];
      unpack<__nv_bfloat16>(raw[u], x);
      const uint32_t c = codes_of(x, none ? 0.0f : __fdividef(1.0f, scale));
      if (is_v) {
        // channels 8 t .. 8 t + 3 are r = 2 t's, the next four r = 2 t + 1's
        unsigned char* const at = tile + kKvV + (j >> 3) * 512 + (8 * t + (j & 7) / 2) * 16 + (j & 1) * 8 + g * 2;
        *reinterpret_cast<unsigned short*>(at) = (unsigned short)c;
        *reinterpret_cast<unsigned short*>(at + 64) = (unsigned short)(c >> 16);
      } else {
        *reinterpret_cast<uint32_t*>(tile + j * 64 + t * 16 + g * 4) = c;
      }
      if (t == 0)
        *reinterpret_cast<__nv_bfloat16*>(tile + kKvScales + j * 16 + (is_v ? 8 : 0) + 2 * g) = __float2bfloat16(scale);
    }
  }
  __syncwarp();
  unsigned char* const out = kv_record(p.pages, page, w.head, w.tile);
  if (w.lo == 0 && hi == kKvTile) {
    for (int i = lane; i < kKvRecord / 16; i += 32)
      reinterpret_cast<uint4*>(out)[i] = reinterpret_cast<const uint4*>(tile)[i];
    return;
  }
  for (int j = w.lo; j < hi; ++j) {
    if (lane < 4) {
      const int at = j * 64 + lane * 16;
      *reinterpret_cast<uint4*>(out + at) = *reinterpret_cast<const uint4*>(tile + at);
    } else if (lane < 12) {
      const int at = kKvV + (j >> 3) * 512 + (4 * (lane - 4) + (j & 7) / 2) * 16 + (j & 1) * 8;
      *reinterpret_cast<uint2*>(out + at) = *reinterpret_cast<const uint2*>(tile + at);
    } else if (lane == 12) {
      const int at = kKvScales + j * 16;
      *reinterpret_cast<uint4*>(out + at) = *reinterpret_cast<const uint4*>(tile + at);
    }
  }
}

__global__ void __launch_bounds__(kWarps * 32) kv4_read_kernel(const __grid_constant__ CacheParams p) {
  __shared__ __align__(16) unsigned char tiles[kWarps][kKvRecord];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Work w = work_of(p, blockIdx.x * kWarps + warp);
  if (!w.any) return;
  const int page = w.tile >= 0 ? kv_page(p.pages, w.b, w.tile) : -1;
  const int held = page < 0 ? w.lo : (int)max((long long)w.lo, min((long long)w.hi, w.n - w.first));   // tokens [lo, held)
  unsigned char* const tile = tiles[warp];
  if (held > w.lo) {
    const uint4* const from = reinterpret_cast<const uint4*>(kv_record(p.pages, page, w.head, w.tile));
#pragma unroll
    for (int i = 0; i < 5; ++i)
      if (i < 4 || lane < 16) reinterpret_cast<uint4*>(tile)[lane + 32 * i] = __ldcs(from + lane + 32 * i);
  }
  __syncwarp();
  const bool is_v = lane >= 16;
  const int g = (lane & 15) >> 2, t = lane & 3;
  __nv_bfloat16* const out =
      reinterpret_cast<__nv_bfloat16*>(is_v ? p.v_out : p.k_out) + 32 * g + 8 * t +
      (is_v ? w.b * p.v_str[0] + w.head * p.v_str[2] : w.b * p.k_str[0] + w.head * p.k_str[2]);
  const long long step = is_v ? p.v_str[1] : p.k_str[1];
#pragma unroll 4
  for (int j = w.lo; j < w.hi; ++j) {
    uint4 row = make_uint4(0u, 0u, 0u, 0u);
    if (j < held) {
      uint32_t c;
      if (is_v) {
        const unsigned char* const at = tile + kKvV + (j >> 3) * 512 + (8 * t + (j & 7) / 2) * 16 + (j & 1) * 8 + g * 2;
        c = *reinterpret_cast<const unsigned short*>(at) | (uint32_t)*reinterpret_cast<const unsigned short*>(at + 64) << 16;
      } else {
        c = *reinterpret_cast<const uint32_t*>(tile + j * 64 + t * 16 + g * 4);
      }
      const uint32_t scale = *reinterpret_cast<const unsigned short*>(tile + kKvScales + j * 16 + (is_v ? 8 : 0) + 2 * g) * 0x10001u;
      uint32_t pair[4];   // channels (i, i + 4): 128 + c, less 136, times the scale: rounded once
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t y;
        asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xEA;" : "=r"(y) : "r"(c >> (4 * i)), "r"(0x43004300u));
        asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(y) : "r"(0xc308c308u));
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(pair[i]) : "r"(y), "r"(scale));
      }
      row = make_uint4(__byte_perm(pair[0], pair[1], 0x5410), __byte_perm(pair[2], pair[3], 0x5410),
                       __byte_perm(pair[0], pair[1], 0x7632), __byte_perm(pair[2], pair[3], 0x7632));
    }
    __stcs(reinterpret_cast<uint4*>(out + (w.first + j) * step), row);
  }
}

CacheParams params_of(const Kv4Args& a) {
  CacheParams p;
  p.pages = kv4_pages(a);
  p.k_in = a.k;
  p.v_in = a.v;
  p.k_out = a.k_out;
  p.v_out = a.v_out;
  for (int i = 0; i < 3; ++i) {
    p.k_str[i] = a.k_str[i];
    p.v_str[i] = a.v_str[i];
  }
  p.start = a.start;
  p.count = a.count;
  p.B = a.B;
  p.S = a.S;
  p.heads = make_div(a.Hkv);
  p.tiles = make_div(kv4_tiles(a.S));
  return p;
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4Args& a, cudaStream_t stream) {
  const long long units = (long long)a.B * a.Hkv * kv4_tiles(a.S);
  return launch_dependent(kv4_write_kernel, dim3((unsigned)((units + kWarps - 1) / kWarps)), kWarps * 32, 0, stream,
                          params_of(a));
}
cudaError_t launch_kv4_read(const Kv4Args& a, cudaStream_t stream) {
  const long long units = (long long)a.B * a.Hkv * kv4_tiles(a.S);
  return launch_dependent(kv4_read_kernel, dim3((unsigned)((units + kWarps - 1) / kWarps)), kWarps * 32, 0, stream,
                          params_of(a));
}

}  // namespace sa
