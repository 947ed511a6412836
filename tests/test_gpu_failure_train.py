"""The failure path of the training kernels on the GPU: with one load of each CTA announced and not made, the wait for
it gives up after its 2 s, the kernel returns, the host reads the timeout, and the context stays usable.

The kernels are those of a check build (SAGEATTN_CHECK_WITHHOLD, the number of the load that is left out), linked with the
library's other objects and run in a child process (the binding loads one library per process).  No fault, trap or
hang is involved: every wait is bounded.  In layer norm's rings the loads after the missing one are the point: the
thread that loads must ask for no further row in a slot whose row has not landed."""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest

from sage_attention_forward_gb300 import build as lib_build

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WITHHOLD = 3

CHILD = r'''
import sys
sys.path.insert(0, sys.argv[2])
import torch
import sage_attention_forward_gb300 as sa
sa._LIB_PATH = sys.argv[1]
withheld = int(sys.argv[3])
g = torch.Generator(device="cuda").manual_seed(1)
r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)


def gave_up(what):
    try:
        sa.attn_get_device_status()
    except sa.AttnError as e:
        assert "gave up on a bounded wait" in str(e), e
        print(what, "gave up")
    else:
        raise SystemExit(what + ": no timeout reported")
    sa.attn_get_device_status()   # (the read cleared it)


def usable():
    q = r(1, 300, 2, 128)
    o = sa.attn_fwd_bf16(q, q, q).double()
    p = torch.einsum("bihd,bjhd->bhij", q.double(), q.double()).mul(128 ** -0.5).softmax(-1)
    assert float((o - torch.einsum("bhij,bjhd->bihd", p, q.double())).norm() / o.norm()) < 0.01
    sa.attn_get_device_status()


# more key and query tiles an item than come before the missing one, and no more items than SMs (a CTA that gives up
# takes over no other's)
for kv_len in (None, torch.tensor([1000], dtype=torch.int32, device="cuda")):
    q, k, v, d = r(1, 768, 16, 128), r(1, 1024, 16, 128), r(1, 1024, 16, 128), r(1, 768, 16, 128)
    o, lse = sa.attn_fwd_bf16_lse(q, k, v, kv_len=kv_len)
    gave_up("attention forward")
    usable()
    sa.attn_bwd_bf16(d, q, k, v, o.zero_(), lse.fill_(9.0), kv_len=kv_len)
    gave_up("attention backward")
    usable()
# rows of a CTA through the ring (304 CTAs), by 16-byte accesses and by pieces of memory
for N in (5120, 4099):
    x, dy, w = r(304 * 12, N), r(304 * 12, N), r(N)
    y, mean, rstd = sa.layer_norm_fwd(x, w, w)
    gave_up("layer norm forward")
    usable()
    n = withheld * 152   # rows that came before the missing ones, whatever the CTAs
    X = x[:n].double()
    m = X.mean(-1, keepdim=True)
    s = (X - m).square().mean(-1, keepdim=True).add(1e-6).rsqrt()
    want = (X - m) * s * w.double() + w.double()
    assert float((y[:n].double() - want).norm() / want.norm()) < 2.0 ** -8
    mean, rstd = x.float().mean(-1), x.float().var(-1, unbiased=False).add(1e-6).rsqrt()
    sa.layer_norm_bwd(dy, x, w, mean, rstd)
    gave_up("layer norm backward")
    usable()
print("all gave up")
'''


def test_missing_loads_are_reported(cuda_dev):
    lib_build.build()
    out = os.path.join(lib_build.OUT_DIR, "check")          # in-tree, next to the library
    os.makedirs(out, exist_ok=True)
    names = ["attn_lse", "attn_bwd", "layer_norm"]

    def compile_one(name):
        cmd = [lib_build.nvcc()] + lib_build._flags([f"-DSAGEATTN_CHECK_WITHHOLD={WITHHOLD}"]) + [
            "-c", os.path.join(lib_build.CSRC, name + ".cu"), "-o", os.path.join(out, name + "_withhold.o")]
        return subprocess.run(cmd, capture_output=True, text=True, timeout=900)

    with ThreadPoolExecutor(3) as pool:
        for r in pool.map(compile_one, names):
            assert r.returncode == 0, r.stderr[-2000:]
    so = os.path.join(out, "libsageattn_withhold.so")
    objs = [os.path.join(out, n + "_withhold.o") for n in names]
    objs += [os.path.join(lib_build.OUT_DIR, f) for f in ("api.o", "api_train.o", "attn_fwd.o", "sage_prepare.o")]
    r = subprocess.run([lib_build.nvcc()] + lib_build.ARCH + ["-shared", "-o", so] + objs + ["-lcudart"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([sys.executable, "-c", CHILD, so, ROOT, str(WITHHOLD)], capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0 and "all gave up" in r.stdout, (r.stdout[-1000:], r.stderr[-3000:])
