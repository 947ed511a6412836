"""The warp of the training kernels that clears rows past a batch entry's last key reads every tile of its ring, so
the ring's slots have to wait for it too: were it a turn of the ring late, the parity that it waits for would
name a later tile, and the tile that it has to clear would be waited for until the kernel gives up.  That is a
matter of the schedule, so it is shown on the host: attn_tiles.cuh compiled with a model of the barriers, and
the clearing warp run last (CPU)."""
import os
import shutil
import subprocess

import pytest

from sage_attention_forward_gb300 import build as lib_build

HERE = os.path.dirname(os.path.abspath(__file__))

# attn_tiles.cuh's own instructions header, for the host: what clear_warp uses is in clear_model.cpp, the rest is
# declared, so that the header compiles.
PTX = r'''
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>
using std::max;
using std::min;
#undef __noinline__
#define __noinline__
namespace sa {
enum : uint32_t { kErrTimeoutTma = 1, kErrTimeoutMma = 2, kErrTimeoutSync = 4 };
constexpr uint32_t kErrSmemBase = 8;
constexpr int kFmtBF16 = 1;
constexpr uint32_t idesc_f32acc(int, int, bool, bool, int, int) { return 0; }
uint32_t smem_u32(const void*);
void mbar_arrive(uint64_t*);
bool mbar_wait_model(uint64_t*, uint32_t);
inline void mbar_init(uint64_t* bar, uint32_t n) { *bar = ((uint64_t)n << 48) | ((uint64_t)n << 32); }
inline void mbar_arrive_expect_tx(uint64_t*, uint32_t) {}   // (clc_try_cancel's answer completes the phase)
template <bool> bool mbar_try_wait(uint64_t* bar, uint32_t parity) { return mbar_wait_model(bar, parity); }
template <bool> bool mbar_wait(uint64_t* bar, uint32_t parity, volatile uint32_t*, uint32_t*, uint32_t) {
  return mbar_wait_model(bar, parity);
}
template <bool> bool mbar_wait_warp(uint64_t* bar, uint32_t parity, volatile uint32_t*, uint32_t*, uint32_t) {
  return mbar_wait_model(bar, parity);
}
inline bool mbar_wait_teardown(uint64_t* bar, uint32_t parity) { return mbar_wait_model(bar, parity); }
void clc_try_cancel(uint4*, uint64_t*);
bool clc_answer(const uint4*, uint32_t&, uint32_t&, uint32_t&);
inline void fence_proxy_async_smem() {}
void tma_load_4d(void*, const void*, uint64_t*, int, int, int, int);
void mma_f16_ss(uint32_t, uint64_t, uint64_t, uint32_t, uint32_t);
void mma_f16_ts(uint32_t, uint32_t, uint64_t, uint32_t, uint32_t);
void tmem_ld32(uint32_t, uint32_t (&)[32]);
void tmem_ld_wait();
void tmem_reg_fence(uint32_t (&)[32]);
uint32_t pack_bf16x2(float, float);
int div_by(int, const struct Div&);
}  // namespace sa
static struct { int x; } threadIdx, blockIdx;
inline void __syncwarp() {}
inline int __shfl_sync(unsigned, int x, int) { return x; }
inline bool __all_sync(unsigned, bool x) { return x; }
template <class T> T __shfl_xor_sync(unsigned, T x, int) { return x; }
template <class T> T __ldg(const T* p) { return *p; }
inline float __uint_as_float(uint32_t) { return 0; }
inline void atomicOr(uint32_t*, uint32_t) {}
'''


@pytest.mark.parametrize("ring,first", [(2, 0), (3, 1)])   # the forward's V, last tile; dQ's K, first tile
def test_a_late_clearing_warp(ring, first, tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    for name in ("attn_tiles.cuh", "kernels.h"):
        shutil.copy(os.path.join(lib_build.CSRC, name), tmp_path)
    (tmp_path / "ptx_train.cuh").write_text(PTX)
    cuda = os.path.join(os.path.dirname(os.path.dirname(lib_build.nvcc())), "include")
    exe = tmp_path / "model"
    cmd = ["g++", "-std=c++17", "-O1", "-w", "-fpermissive", f"-DSA_RING={ring}", f"-DSA_FIRST={first}", "-I", str(tmp_path),
           "-I", cuda, "-include", "cuda_runtime.h", os.path.join(HERE, "clear_model.cpp"), "-o", str(exe),
           "-Wl,--gc-sections", "-ffunction-sections"]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
