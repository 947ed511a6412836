// What the C entry points share: error messages, checks of arguments, tensor maps (api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/sageattn.h"

#define TRY(x)                          \
  do {                                  \
    attn_status _s = (x);               \
    if (_s != ATTN_OK) return _s;       \
  } while (0)

namespace sa {
namespace api {

constexpr double kLog2e = 1.4426950408889634;

attn_status fail(attn_status s, const char* fmt, ...);
attn_status fail_cuda(cudaError_t e, const char* what);
attn_status check_device();
attn_status get_encoder();
attn_status tmap_bhsd_bf16(CUtensorMap* m, const void* ptr, int B, int S, int H, const long long str[3],
                           int rows = 128);
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
attn_status check_grid(int B, int H, long long S_pad);
attn_status check_strides(const char* name, const void* ptr, const int64_t* in, int B, int S, int H, long long out[3]);

}  // namespace api
}  // namespace sa
