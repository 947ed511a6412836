"""Refusals of the rotation's calls and the table of frequencies (CPU)."""
import ctypes
import math

import pytest
import torch

import sage_attention_forward_gb300 as sa

I64x3 = ctypes.c_int64 * 3
FAKE = 0x100000   # an aligned non-null address; validation never dereferences it
FAR = 0x10000000


def call(name="rope_fwd", q=FAKE, k=2 * FAKE, qo=FAR, ko=2 * FAR, B=1, S=4, Hq=2, Hk=2, N=128, qs=(1024, 256, 128),
         qos=None, pos=FAKE, ps=(4, 1, 0), axes=1, freq=FAKE, R=128, inter=0, m=1.0, dtype=0, qw=FAKE, kw=FAKE, eps=1e-6,
         w_dtype=0, dqo=3 * FAKE, dko=4 * FAKE, dqw=FAKE, dkw=FAKE, ws=FAKE, ws_bytes=1 << 20):
    L = sa.lib()
    st, ost = I64x3(*qs), I64x3(*(qos or qs))
    p = I64x3(*ps)
    if name in ("rope_fwd", "rope_bwd"):
        return getattr(L, name)(q, k, qo, ko, B, S, Hq, Hk, N, st, st, ost, ost, pos, p, axes, freq, R, inter, m, dtype, None)
    if name == "qk_norm_rope_fwd":
        return L.qk_norm_rope_fwd(q, k, qw, kw, qo, ko, B, S, Hq, Hk, N, st, st, ost, ost, eps, pos, p, axes, freq, R, inter,
                                  m, dtype, w_dtype, None)
    return L.qk_norm_rope_bwd(dqo, dko, q, k, qw, kw, qo, ko, dqw, dkw, B, S, Hq, Hk, N, st, st, st, st, ost, ost, eps, pos, p,
                              axes, freq, R, inter, m, dtype, w_dtype, ws, ws_bytes, None)


ALL = ("rope_fwd", "rope_bwd", "qk_norm_rope_fwd", "qk_norm_rope_bwd")
NORM = ALL[2:]


@pytest.mark.parametrize("names,kw,status", [
    (ALL, dict(dtype=3), 1), (ALL, dict(dtype=-1), 1),
    (ALL, dict(B=-1), 1), (ALL, dict(Hk=-1), 1), (ALL, dict(N=0), 1), (ALL, dict(N=513), 1),
    (ALL, dict(R=130), 1), (ALL, dict(R=63), 1), (ALL, dict(R=-2), 1), (ALL, dict(inter=2), 1),
    (ALL, dict(m=math.inf), 1), (ALL, dict(m=math.nan), 1),
    (ALL, dict(B=1 << 15, S=1 << 15), 1), (ALL, dict(B=1 << 30, S=1 << 30), 1), (ALL, dict(Hq=2 ** 31 - 1, Hk=2 ** 31 - 1), 1),
    (ALL, dict(freq=None), 1), (ALL, dict(freq=FAKE + 4), 2), (ALL, dict(pos=FAKE + 2), 2),
    (ALL, dict(axes=0), 1), (ALL, dict(axes=5), 1), (ALL, dict(ps=(0, -1, 0)), 1),
    (ALL, dict(q=None), 1), (ALL, dict(k=None), 1), (ALL, dict(qo=None), 1), (ALL, dict(q=FAKE + 1), 2),
    (ALL, dict(q=FAKE + 2, dtype=2, w_dtype=2), 2), (ALL, dict(qs=(1024, -256, 128)), 1), (ALL, dict(qos=(1024, 0, 128)), 1),
    (ALL, dict(qos=(1 << 38, 256, 128), B=2), 1),
    (ALL, dict(qo=FAKE + 256), 1),          # an output inside its input, a row on
    (ALL, dict(qo=2 * FAKE), 1),            # Q's output in K's place
    (ALL, dict(ko=FAR), 1),                 # both outputs in one place
    (NORM, dict(eps=-1.0), 1), (NORM, dict(eps=math.nan), 1), (NORM, dict(w_dtype=1), 1), (NORM, dict(qw=FAKE + 1), 2),
    (NORM[1:], dict(dqo=None), 1), (NORM[1:], dict(dqw=FAKE + 1), 2), (NORM[1:], dict(ws=None), 1),
    (NORM[1:], dict(ws=FAKE + 8), 2), (NORM[1:], dict(ws_bytes=16), 1), (NORM[1:], dict(ko=3 * FAKE), 1),
    (ALL[:3], dict(S=0), 0), (ALL[:3], dict(B=0, q=None, k=None, qo=None, ko=None), 0), (ALL[:3], dict(Hq=0, Hk=0), 0),
    (NORM[1:], dict(S=0, dqw=None, dkw=None), 0),
])
def test_refusals(names, kw, status):
    for name in names:
        assert call(name, **kw) == status, (name, sa.lib().attn_last_error())
        if status:
            assert sa.lib().attn_last_error().decode() != ""


def test_accepted_up_to_the_device():
    """What only the missing GPU stops: outputs in place, no K, no positions, no rotation."""
    for name in ALL:
        for kw in (dict(), dict(qo=FAKE, ko=2 * FAKE), dict(Hk=0, k=None, ko=None), dict(pos=None, axes=9), dict(R=0, freq=None),
                   dict(qs=(1024, 0, 128), qos=(1024, 256, 128))):
            if torch.cuda.is_available():
                pytest.skip("would run")
            assert call(name, **kw) in (3, 4), (name, kw, sa.lib().attn_last_error())
    assert call("qk_norm_rope_bwd", dqw=None, dkw=None, ws=None, ws_bytes=0) in (3, 4)


def test_workspace_sizes():
    size = sa.lib().qk_norm_rope_bwd_workspace_size
    assert size(0, 4, 2, 2, 128) == 0 and size(1, 4, 2, 2, 513) == 0 and size(1 << 20, 1 << 20, 1, 1, 8) == 0
    assert 0 < size(1, 1, 1, 0, 1) <= 8 and size(1, 1 << 20, 32, 32, 128) == 2 * 608 * 128 * 4


def test_frequencies():
    def radians(freq):
        return [((f % 2 ** 64) & ~3) / 2.0 ** 64 * 2 * math.pi for f in freq.tolist()]

    freq, m = sa.rope_frequencies(64, theta=5e5, device="cpu")
    assert m == 1.0 and freq.dtype == torch.int64
    for i, w in enumerate(radians(freq)):
        assert abs(w - 5e5 ** (-i / 32)) < 2e-16 + 2 * math.pi * 4 / 2 ** 64
    freq, _ = sa.rope_frequencies(128, axes=(16, 56, 56), device="cpu")
    assert [f & 3 for f in freq.tolist()] == [0] * 8 + [1] * 28 + [2] * 28
    assert radians(freq)[8] == pytest.approx(1.0) and radians(freq)[9] == pytest.approx(10000 ** (-1 / 28))
    lin = radians(sa.rope_frequencies(64, scaling={"kind": "linear", "factor": 4}, device="cpu")[0])
    assert lin[3] == pytest.approx(10000 ** (-3 / 32) / 4)
    ntk = radians(sa.rope_frequencies(64, scaling={"kind": "ntk", "factor": 4}, device="cpu")[0])
    assert ntk[0] == pytest.approx(1.0) and ntk[31] == pytest.approx(10000 ** (-31 / 32) / 4)
    bands = radians(sa.rope_frequencies(64, scaling={"kind": "bands", "factor": 8, "length": 8192}, device="cpu")[0])
    assert bands[0] == pytest.approx(1.0) and bands[31] == pytest.approx(10000 ** (-31 / 32) / 8)
    yarn, m = sa.rope_frequencies(64, scaling={"kind": "yarn", "factor": 16, "length": 4096}, device="cpu")
    assert m == pytest.approx(0.1 * math.log(16) + 1) and radians(yarn)[0] == pytest.approx(1.0)
    assert radians(yarn)[31] == pytest.approx(10000 ** (-31 / 32) / 16)
    for bad in (dict(rope_dim=3), dict(rope_dim=8, axes=(4, 2)), dict(rope_dim=8, axes=(5, 3)),
                dict(rope_dim=10, axes=(2,) * 5), dict(rope_dim=8, theta=0.0), dict(rope_dim=8, scaling={"kind": "other"}),
                dict(rope_dim=8, scaling={"kind": "yarn", "factor": 2}),
                dict(rope_dim=8, scaling={"kind": "linear", "factor": 2, "length": 8}),
                dict(rope_dim=8, scaling={"kind": "bands", "factor": 2, "length": 8, "low": 4, "high": 1})):
        with pytest.raises(ValueError):
            sa.rope_frequencies(device="cpu", **bad)


def test_the_binding_refuses_what_is_not_on_the_gpu():
    x, freq = torch.zeros((1, 2, 2, 8)), torch.zeros(4, dtype=torch.int64)
    for bad in (x, x[0], x.to(torch.float64)):
        with pytest.raises(ValueError):
            sa.rope_fwd(bad, None, freq)
