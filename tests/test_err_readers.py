"""Each translation unit with bounded waits registers the reader of its error word when the library is loaded.  One too
many would go unread, and a timeout with it: the status call says so (CPU: a library with that many is linked).  A unit none
of whose kernels has been launched costs the status call no copy, nor the loading of the unit."""
import ctypes
import os
import subprocess

from sage_attention_forward_gb300 import build as lib_build

MORE = r'''
#include "kernels.h"
static cudaError_t none(uint32_t* out) { *out = 0; return cudaSuccess; }
static const bool added[] = {%s};
extern "C" __attribute__((visibility("default"))) int refused() { int n = 0; for (bool b : added) n += !b; return n; }
'''


def status_with(more, tmp_path):
    src, so = tmp_path / f"more{more}.cpp", tmp_path / f"lib{more}.so"
    src.write_text(MORE % ", ".join(["sa::add_err_reader(none)"] * more))
    lib_build.build()
    objs = [os.path.join(lib_build.OUT_DIR, os.path.splitext(s)[0] + ".o")
            for s in lib_build.SOURCES + lib_build.HOST_SOURCES]
    cmd = [lib_build.nvcc()] + lib_build._flags() + ["-I", lib_build.CSRC, "-shared", str(src), *objs, "-o", str(so),
                                                     "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    lib = ctypes.CDLL(str(so))
    lib.attn_last_error.restype = ctypes.c_char_p
    lib.attn_get_device_status.argtypes = [ctypes.c_void_p]
    return lib.refused(), lib.attn_get_device_status(None), lib.attn_last_error().decode()


def test_every_error_word_is_read(tmp_path):
    assert status_with(1, tmp_path)[0] == 0
    refused, status, message = status_with(9, tmp_path)
    assert refused > 0 and status == 3 and "error words" in message


COPIES = r'''
#include <cuda_runtime.h>
#define OUT __attribute__((visibility("default")))
static int copies = 0;
extern "C" {
OUT int copies_made() { return copies; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemcpyFromSymbol(void* to, const void*, size_t n, size_t, enum cudaMemcpyKind) {
  ++copies;
  for (size_t i = 0; i < n; ++i) static_cast<char*>(to)[i] = 0;
  return cudaSuccess;
}
cudaError_t cudaMemcpyToSymbol(const void*, const void*, size_t, size_t, enum cudaMemcpyKind) {
  ++copies;
  return cudaSuccess;
}
}
'''


def test_units_that_were_not_used_cost_no_copy(tmp_path):
    """The library linked with the three runtime calls of the status call replaced by ones that count."""
    src, so = tmp_path / "copies.cpp", tmp_path / "libcopies.so"
    src.write_text(COPIES)
    lib_build.build()
    objs = [os.path.join(lib_build.OUT_DIR, os.path.splitext(s)[0] + ".o")
            for s in lib_build.SOURCES + lib_build.HOST_SOURCES]
    cmd = [lib_build.nvcc()] + lib_build._flags() + ["-shared", str(src), *objs, "-o", str(so), "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    lib = ctypes.CDLL(str(so))
    lib.attn_get_device_status.argtypes = [ctypes.c_void_p]
    assert lib.attn_get_device_status(None) == 0
    assert lib.copies_made() == 2   # the forward's word, read and cleared
