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
constexpr int kAhead = 8;   // tokens whose loads are under way

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
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], float scale, float inv) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // The quotient by the reciprocal, its remainder taken off once (Markstein, "Computation of elementary functions on the
    // IBM RISC System/6000 processor", 1990): where x / scale is half an integer, this is exact.
    float q = x[i] * inv;
    q = fmaf(fmaf(-q, scale, x[i]), inv, q);
    q = fminf(fmaxf(q, -8.0f), 7.0f);
    const uint32_t c = __float_as_uint(q + (12582912.0f + 8.0f));   // 1.5 2^23: rounds to even, the integer in the low bits
    out |= (c & 15u) << (4 * i);
  }
  return out;
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
      float x[8];
      unpack<__nv_bfloat16>(raw[u], x);
      float top = x[0], low = x[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        top = fmaxf(top, x[i]);
        low = fminf(low, x[i]);
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
      }
      const float ext = top >= -low ? top : low;
      const bool none = fabsf(ext) < 0x1p-100f;
      const float scale = none ? 0.0f : ext * -0.125f;
      const uint32_t c = none ? 0x88888888u : codes_of(x, scale, __fdividef(1.0f, scale));
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
      const float scale =
          __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(tile + kKvScales + j * 16 + (is_v ? 8 : 0) + 2 * g));
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = (float)((int)((c >> (4 * i)) & 15u) - 8) * scale;
      row = pack<__nv_bfloat16>(x);
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
