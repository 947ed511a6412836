"""Refusals of the 4-bit cache's calls, sizes, and the reference's own record layout (CPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import kv4_ref as ref
import sage_attention_forward_gb300 as sa

I64x3 = ctypes.c_int64 * 3
FAKE, FAR = 0x100000, 0x10000000   # aligned non-null addresses; validation never dereferences them


def call(name, cache=FAKE, pages=8, size=64, table=FAKE, table_str=4, most=4, start=FAKE, count=None, k=FAR, v=2 * FAR, B=2,
         S=3, Hq=8, H=2, D=128, ks=(4096, 1024, 128), kv_len=FAKE, q=FAR, o=2 * FAR, lse=3 * FAR, scale=0.1, causal=1, ws=FAKE,
         ws_bytes=1 << 30):
    L, st = sa.lib(), I64x3(*ks)
    if name == "kv4_write":
        return L.kv4_write(k, v, cache, pages, size, table, table_str, most, start, count, B, S, H, D, st, st, None)
    if name == "kv4_read":
        return L.kv4_read(cache, pages, size, table, table_str, most, start, count, k, v, B, S, H, D, st, st, None)
    return L.attn_fwd_kv4(q, cache, pages, size, table, table_str, most, kv_len, o, lse, B, S, Hq, H, D, st, st, scale, causal,
                          ws, ws_bytes, None)


ALL = ("kv4_write", "kv4_read", "attn_fwd_kv4")
ATTN = ALL[2:]


@pytest.mark.parametrize("names,kw,status", [
    (ALL, dict(D=64), 3), (ALL, dict(B=-1), 1), (ALL, dict(S=-1), 1), (ALL, dict(H=-1, Hq=-1), 1), (ALL, dict(pages=-1), 1),
    (ALL, dict(most=-1), 1), (ALL, dict(size=0), 1), (ALL, dict(size=24), 1), (ALL, dict(size=-16), 1),
    (ALL, dict(size=1 << 20, most=1 << 11), 1), (ALL, dict(B=1 << 20, H=1 << 12, Hq=1 << 12), 1), (ALL, dict(B=1 << 10, S=1 << 30), 1),
    (ALL, dict(cache=None), 1), (ALL, dict(cache=FAKE + 8), 2), (ALL, dict(table=None), 1), (ALL, dict(table=FAKE + 2), 2),
    (ALL, dict(table_str=-1), 1),
    (ALL[:2], dict(k=None), 1), (ALL[:2], dict(v=FAR + 2), 2), (ALL[:2], dict(ks=(4096, 1020, 128)), 2),
    (ALL[:2], dict(ks=(4096, -1024, 128)), 1), (ALL[:2], dict(start=None), 1), (ALL[:2], dict(start=FAKE + 1), 2),
    (ALL[:2], dict(count=FAKE + 2), 2), (ALL[1:2], dict(v=FAR), 1),
    (ATTN, dict(Hq=7), 1), (ATTN, dict(Hq=0), 1), (ATTN, dict(causal=2), 1), (ATTN, dict(scale=-1.0), 1),
    (ATTN, dict(scale=math.inf), 1), (ATTN, dict(scale=math.nan), 1), (ATTN, dict(q=None), 1), (ATTN, dict(o=FAR + 8), 2),
    (ATTN, dict(o=FAR), 1), (ATTN, dict(kv_len=None), 1), (ATTN, dict(kv_len=FAKE + 2), 2), (ATTN, dict(lse=None), 1),
    (ATTN, dict(lse=FAR + 2), 2), (ATTN, dict(ws=None), 1), (ATTN, dict(ws=FAKE + 8), 2), (ATTN, dict(ws_bytes=64), 1),
    (ALL, dict(B=0), 0), (ALL, dict(S=0), 0), (ALL, dict(H=0, Hq=0, cache=None, table=None, k=None, v=None), 0),
    (ALL[:1], dict(pages=0, cache=None), 0), (ALL[:1], dict(most=0, table=None), 0),
])
def test_refusals(names, kw, status):
    for name in names:
        assert call(name, **kw) == status, (name, sa.lib().attn_last_error())
        if status:
            assert sa.lib().attn_last_error().decode() != ""


def test_accepted_up_to_the_device():
    if torch.cuda.is_available():
        pytest.skip("would run")
    for name in ALL:
        for kw in (dict(), dict(table_str=0), dict(B=1, table_str=-1), dict(size=48)):
            assert call(name, **kw) in (3, 4), (name, kw)


def test_sizes():
    L = sa.lib()
    assert L.kv4_cache_size(3, 8, 64) == 3 * 8 * 4 * 2304 == sa.kv4_cache(3, 8, 64, device="cpu").numel()
    assert L.kv4_cache_size(0, 8, 64) == 0 and L.kv4_cache_size(3, 8, 24) == 0
    size = L.attn_fwd_kv4_workspace_size
    assert size(0, 1, 8, 8, 4, 16) == 0 and size(1, 1, 7, 2, 4, 16) == 0 and size(1, 1, 8, 8, 4, 24) == 0
    # pieces of at most all CTAs of a wave; few for a small cache
    assert 0 < size(1, 1, 1, 1, 1, 16) < 200000 and size(64, 1, 32, 8, 1 << 12, 64) < 16 << 20
    with pytest.raises(ValueError):
        sa.kv4_cache(3, 8, 40, device="cpu")


def test_the_binding_refuses_what_is_not_on_the_gpu():
    cache, table = sa.kv4_cache(2, 1, 16, device="cpu"), torch.zeros((1, 2), dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)
    x = torch.zeros((1, 1, 1, 128), dtype=torch.bfloat16)
    for f in (lambda: sa.kv4_write(x, x, cache, table, n), lambda: sa.kv4_read(cache, table, n, 1),
              lambda: sa.attn_fwd_kv4(x, cache, table, n)):
        with pytest.raises(ValueError, match="CUDA"):
            f()


def test_reference_codes():
    """Exactly representable values come back; ties go to even; the extreme value's code is -8, the other end is cut at 7."""
    x = torch.zeros(128, dtype=torch.bfloat16)
    x[:32] = torch.arange(-16, 16).to(torch.bfloat16) / 2
    want = [min(7, int(round(c / 2))) for c in range(-16, 16)]
    for sign in (1, -1):
        code, scale = ref.quantise(sign * x)
        assert scale[0] == sign and code[:32].tolist() == want and want[0] == -8 and want[31] == 7
    x[:32] = 1.0
    x[5] = -1.0
    code, scale = ref.quantise(x)
    assert scale[0] == -0.125 and code[0] == -8 and code[5] == 7


def test_reference_records_have_no_overlap():
    """Each of the 4096 codes and 128 scales of a record has bits of its own."""
    seen = np.zeros(2304, dtype=np.int64)
    for which in range(2):
        for j in range(16):
            r = np.zeros(2304, dtype=np.uint8)
            ref.put(r, j, which, np.full(128, 7), torch.full((4,), -float("nan")))
            bits = np.unpackbits(r).reshape(2304, 8)
            seen[:2048] += bits[:2048].sum(1, dtype=np.int64)
            r2 = np.zeros(2304, dtype=np.uint8)
            ref.put(r2, j, which, np.full(128, -8), torch.full((4,), 1.0))
            seen[2048:] += (r2[2048:] != 0)
    assert (seen[:2048] == 8).all() and (seen[2048:] <= 1).all() and seen[2048:].sum() == 2 * 16 * 4 * 2
