"""rope_fwd, rope_bwd, qk_norm_rope_fwd and qk_norm_rope_bwd on the GPU against their definitions in 64 bits."""
import math

import pytest
import torch

import rope_ref as ref
import sage_attention_forward_gb300 as sa

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def rows(seed, *shape, dtype, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * gain).to(dtype)


# B, S, Hq, Hk, N, R, interleaved, axes, scaling
CASES = [
    (1, 1, 1, 1, 2, 2, False, None, None),                 # the smallest head
    (2, 3, 1, 1, 1, 0, True, None, None),                  # one channel, nothing rotated
    (2, 5, 4, 2, 128, 128, False, None, None),
    (1, 7, 3, 3, 128, 128, True, (44, 42, 42), None),
    (3, 1, 32, 8, 128, 128, False, None, {"kind": "bands", "factor": 8, "length": 8192}),
    (2, 9, 5, 1, 80, 32, False, None, {"kind": "linear", "factor": 4}),   # five lanes a row
    (1, 33, 2, 2, 96, 96, True, None, {"kind": "yarn", "factor": 16, "length": 4096}),
    (1, 4, 3, 2, 64, 40, False, None, None),               # halves that are no whole pieces
    (1, 4, 3, 2, 64, 40, True, None, None),
    (2, 3, 2, 1, 77, 30, False, (10, 10, 10), None),       # rows off 16 bytes
    (2, 3, 2, 1, 77, 76, True, None, None),
    (1, 2, 2, 2, 256, 64, False, None, {"kind": "ntk", "factor": 2}),
    (1, 2, 3, 1, 250, 250, False, None, None),
    (1, 2, 3, 1, 251, 200, True, None, None),
    (1, 3, 2, 2, 512, 512, False, None, None),
    (1, 3, 2, 2, 509, 508, False, None, None),
    (1, 3, 2, 2, 511, 2, True, None, None),
    (1, 2, 70, 3, 16, 16, False, None, None),              # a lane a row, more heads than a pass
    (1, 400, 2, 0, 32, 32, False, None, None),             # no K
    (1, 19, 23, 11, 48, 48, False, None, None),            # three lanes a row, ten rows a turn
    (1, 11, 7, 4, 144, 144, False, None, None),            # nine lanes a row
    (2, 5, 4, 4, 160, 64, True, None, None),
    (1, 13, 9, 2, 80, 80, True, None, None),               # five lanes, six rows a turn
    (2, 31, 13, 3, 58, 58, True, None, None),              # by the channel, eight lanes a row
    (1, 7, 6, 5, 61, 40, False, None, None),
    (2, 3, 7, 2, 80, 34, False, None, None),               # halves that are no whole pieces, five lanes a row
    (1, 2, 3, 1, 512, 266, False, None, None),             # ... and all lanes one row's
    (1, 3, 5, 2, 128, 2, False, None, None),
    (2, 600, 4, 1, 32, 18, False, (6, 6, 6), None),        # ... sixteen rows a warp, many tokens
]


def make(case, seed, dtype, far=0):
    B, S, Hq, Hk, N, R, inter, axes, scaling = case
    freq, m = sa.rope_frequencies(R, axes=axes, scaling=scaling, device="cpu")
    g = torch.Generator().manual_seed(seed)
    n = len(axes or (0,))
    pos = torch.randint(-5, 1000, (B, S, n), generator=g, dtype=torch.int32)
    if far:
        pos = torch.randint(far - 1000, far, (B, S, n), generator=g, dtype=torch.int64).to(torch.int32)
    q, k = rows(seed + 1, B, S, Hq, N, dtype=dtype), rows(seed + 2, B, S, Hk, N, dtype=dtype)
    return freq, m, pos, q, k


def given(pos):
    return pos[..., 0] if pos.shape[-1] == 1 else pos


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_rotation_and_its_gradient(case, dtype, cuda_dev):
    t, inter = TYPES[dtype], case[6]
    freq, m, pos, q, k = make(case, 10, t)
    cos, sin = ref.cos_sin(freq, pos, case[0], case[1], m)
    for call, sign in ((sa.rope_fwd, 1), (sa.rope_bwd, -1)):
        got = call(q.to(cuda_dev), k.to(cuda_dev), freq.to(cuda_dev), given(pos).to(cuda_dev), interleaved=inter,
                   magnitude=m)
        for name, x, y in zip("qk", (q, k), got):
            want, bound = ref.rope(x.double(), cos, sign * sin, inter, m)
            ref.near(y, want, bound, name)


@pytest.mark.parametrize("w_type", ["same", "fp32", "none"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_norm_and_its_gradient(case, dtype, w_type, cuda_dev):
    t, inter, N = TYPES[dtype], case[6], case[4]
    freq, m, pos, q, k = make(case, 20, t)
    wt = t if w_type == "same" else torch.float32
    qw, kw = ((1 + rows(30 + i, N, dtype=torch.float32, gain=0.3)).to(wt) for i in range(2))
    dq, dk = rows(40, *q.shape, dtype=t, gain=0.1), rows(41, *k.shape, dtype=t, gain=0.1)
    cos, sin = ref.cos_sin(freq, pos, case[0], case[1], m)
    dev = lambda x: x.to(cuda_dev)  # noqa: E731
    weights = (None, None) if w_type == "none" else (dev(qw), dev(kw))
    how = {"eps": 1e-5, "interleaved": inter, "magnitude": m}
    y = sa.qk_norm_rope_fwd(dev(q), dev(k), *weights, dev(freq), dev(given(pos)), **how)
    got = sa.qk_norm_rope_bwd(dev(dq), dev(dk), dev(q), dev(k), *weights, dev(freq), dev(given(pos)), **how)
    for i, (name, x, d, w) in enumerate((("q", q, dq, qw), ("k", k, dk, kw))):
        w = torch.ones(N, dtype=torch.float64) if w_type == "none" else w.double()
        ref.near(y[i], *ref.norm_rope(x.double(), w, 1e-5, cos, sin, inter, m), name)
        dx, dx_bound, dw, dw_bound = ref.norm_rope_bwd(d.double(), x.double(), w, 1e-5, cos, sin, inter, m)
        ref.near(got[i], dx, dx_bound, "d" + name)
        if w_type == "none":
            assert got[2 + i] is None
        else:
            ref.near(got[2 + i], dw, dw_bound, f"d{name}_weight")


@pytest.mark.parametrize("far", [2 ** 20, 2 ** 31 - 1, -(2 ** 31) + 1000])
def test_far_positions(far, cuda_dev):
    case = (2, 4, 2, 1, 128, 128, False, None, None)
    freq, m, pos, q, k = make(case, 50, torch.float32, far)
    cos, sin = ref.cos_sin(freq, pos, 2, 4, m)
    got = sa.rope_fwd(q.to(cuda_dev), k.to(cuda_dev), freq.to(cuda_dev), given(pos).to(cuda_dev))
    for name, x, y in zip("qk", (q, k), got):
        ref.near(y, *ref.rope(x.double(), cos, sin, False, m), name)


def test_position_forms(cuda_dev):
    case = (2, 6, 2, 2, 64, 64, True, (32, 16, 16), None)
    freq, m, pos, q, k = make(case, 60, torch.bfloat16)
    q, k, f = q.to(cuda_dev), k.to(cuda_dev), freq.to(cuda_dev)
    # one batch entry's positions for all; a table whose rows and axes are far apart
    one = pos[:1].to(cuda_dev)
    wide = torch.zeros((4, 2, 12), dtype=torch.int32, device=cuda_dev).permute(1, 2, 0)[:, ::2, 1:]
    wide.copy_(one.expand(2, 6, 3))
    for p in (one, one.expand(2, 6, 3), wide):
        got = sa.rope_fwd(q, k, f, p, interleaved=True)
        cos, sin = ref.cos_sin(freq, p.cpu(), 2, 6, m)
        ref.near(got[0], *ref.rope(q.double().cpu(), cos, sin, True, m), "q")
    plain = sa.rope_frequencies(64, device=cuda_dev)[0]
    a = sa.rope_fwd(q, k, plain)                                         # places in the sequence
    for p in (torch.arange(6, dtype=torch.int32, device=cuda_dev), torch.arange(6, dtype=torch.int32, device=cuda_dev)[None]):
        b = sa.rope_fwd(q, k, plain, p)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_axis_past_the_last_is_the_last(cuda_dev):
    freq = sa.rope_frequencies(32, device="cpu")[0]
    x = rows(70, 1, 5, 2, 32, dtype=torch.float32).to(cuda_dev)
    p = torch.randint(0, 99, (1, 5, 2), dtype=torch.int32, device=cuda_dev)
    a = sa.rope_fwd(x, None, (freq | 3).to(cuda_dev), p)[0]
    b = sa.rope_fwd(x, None, (freq | 1).to(cuda_dev), p)[0]
    assert torch.equal(a, b)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N,R", [(128, 128), (128, 64), (77, 30)])
def test_strides_and_in_place(N, R, interleaved, cuda_dev):
    """Slices of a fused projection, heads before tokens, rows off 16 bytes, expanded inputs, outputs that are the inputs:
    the same bits as contiguous tensors'."""
    B, S, H = 2, 5, 3
    freq = sa.rope_frequencies(R, device=cuda_dev)[0]
    qkv = rows(80, B, S, 3, H, N, dtype=torch.bfloat16).to(cuda_dev)
    q, k = qkv[:, :, 0], qkv[:, :, 1]
    w = (1 + rows(81, N, dtype=torch.float32)).to(cuda_dev)
    how = {"interleaved": interleaved}
    want = sa.rope_fwd(q.contiguous(), k.contiguous(), freq, **how)
    norm = sa.qk_norm_rope_fwd(q.contiguous(), k.contiguous(), w, w, freq, **how)
    back = sa.qk_norm_rope_bwd(k.contiguous(), q.contiguous(), q.contiguous(), k.contiguous(), w, w, freq, **how)
    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))  # noqa: E731
    near = lambda a, b: all(torch.allclose(x.float(), y.float(), rtol=2 ** -7, atol=1e-5) for x, y in zip(a, b))  # noqa: E731
    assert same(sa.rope_fwd(q, k, freq, **how), want)
    heads = [t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for t in (q, k)]
    assert same(sa.rope_fwd(*heads, freq, **how), want)
    off = torch.empty(B * S * H * (N + 3) + 1, dtype=torch.bfloat16, device=cuda_dev)[1:].view(B, S, H, N + 3)[..., :N]
    off.copy_(q)
    out = torch.empty_like(qkv)
    # (other lanes hold a row there: the rotation rounds alike, the norm's sum is of another order)
    assert same(sa.rope_fwd(off, k, freq, q_out=out[:, :, 2], **how), want)
    assert near(sa.qk_norm_rope_fwd(off, k, w, w, freq, **how), norm)
    assert near(sa.qk_norm_rope_bwd(k, off, off, k, w, w, freq, **how), back)
    row = q[:, :, :1].expand(B, S, H, N)
    assert same(sa.rope_fwd(row, k, freq, **how)[:1], sa.rope_fwd(row.contiguous(), k, freq, **how)[:1])
    dy = torch.ones((), dtype=torch.bfloat16, device=cuda_dev).expand(B, S, H, N)
    if N == 1 or dy.stride(3) == 1:
        assert same(sa.rope_bwd(dy, None, freq, **how)[:1], sa.rope_bwd(dy.contiguous(), None, freq, **how)[:1])
    with pytest.raises(ValueError, match="unit channel stride"):
        sa.rope_bwd(dy, None, freq, **how)
    # in place, K first written where Q is still read in other rows
    again = qkv.clone()
    sa.rope_fwd(again[:, :, 0], again[:, :, 1], freq, q_out=again[:, :, 0], k_out=again[:, :, 1], **how)
    assert same((again[:, :, 0], again[:, :, 1]), want) and torch.equal(again[:, :, 2], qkv[:, :, 2])
    again = qkv.clone()
    sa.qk_norm_rope_fwd(again[:, :, 0], again[:, :, 1], w, w, freq, q_out=again[:, :, 0], k_out=again[:, :, 1], **how)
    assert same((again[:, :, 0], again[:, :, 1]), norm)
    for first in (True, False):   # dx in place of dy, and of x
        dq, dk, x, y = k.contiguous(), q.contiguous(), q.contiguous(), k.contiguous()
        got = sa.qk_norm_rope_bwd(dq, dk, x, y, w, w, freq, dq=dq if first else x, dk=dk if first else y, **how)
        assert same(got, back)


def test_gradient_matches_differences(cuda_dev):
    """dL/dx and dL/dw of L = sum(y c) against central differences, in FP32."""
    freq, m = sa.rope_frequencies(8, scaling={"kind": "yarn", "factor": 4, "length": 64}, device=cuda_dev)
    x, w = rows(90, 1, 3, 2, 10, dtype=torch.float32).to(cuda_dev), (1 + rows(91, 10, dtype=torch.float32)).to(cuda_dev)
    c = rows(92, 1, 3, 2, 10, dtype=torch.float32).to(cuda_dev)
    how = {"eps": 1e-3, "magnitude": m}
    loss = lambda x, w: float((sa.qk_norm_rope_fwd(x, None, w, None, freq, **how)[0].double() * c.double()).sum())  # noqa: E731
    dx, _, dw, _ = sa.qk_norm_rope_bwd(c, None, x, None, w, None, freq, **how)
    h = 2.0 ** -6   # error: h^2 / 6 times a third derivative of order 10, and 2^-24 of values of order 10 over 2 h
    for t, grad in ((x, dx), (w, dw)):
        for i in range(0, t.numel(), 3):
            up, down = t.clone(), t.clone()
            up.view(-1)[i] += h
            down.view(-1)[i] -= h
            args = ((up, w), (down, w)) if t is x else ((x, up), (x, down))
            num = (loss(*args[0]) - loss(*args[1])) / (2 * h)
            assert abs(num - float(grad.view(-1)[i])) < 5e-3, (i, num)


@pytest.mark.parametrize("dtype", TYPES)
def test_same_bits_on_any_stream_and_in_graphs(dtype, cuda_dev):
    t = TYPES[dtype]
    freq = sa.rope_frequencies(128, device=cuda_dev)[0]
    q, k = rows(100, 1, 700, 4, 128, dtype=t).to(cuda_dev), rows(101, 1, 700, 2, 128, dtype=t).to(cuda_dev)
    w = torch.ones(128, device=cuda_dev)
    want = sa.qk_norm_rope_bwd(q, k, q, k, w, w, freq)
    fwd = sa.qk_norm_rope_fwd(q, k, w, w, freq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = sa.qk_norm_rope_bwd(q, k, q, k, w, w, freq, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graphs = []
    for _ in range(2):   # two graphs, each with its own workspace
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = sa.qk_norm_rope_bwd(q, k, q, k, w, w, freq)
            out += sa.qk_norm_rope_fwd(q, k, w, w, freq) + sa.rope_fwd(q, k, freq)
        graphs.append((graph, out))
    for graph, out in graphs + graphs[::-1]:
        for o in out:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want + fwd, out))


def test_two_calls_at_once(cuda_dev):
    """On two streams, each with its own workspace: the bits of one call alone."""
    freq = sa.rope_frequencies(64, device=cuda_dev)[0]
    w = (1 + rows(105, 64, dtype=torch.float32, gain=0.2)).to(cuda_dev)
    tensors = [[rows(106 + 4 * j + i, 2, 900, 6, 64, dtype=torch.bfloat16).to(cuda_dev) for i in range(4)] for j in range(2)]
    want = [sa.qk_norm_rope_bwd(*t, w, w, freq) for t in tensors]
    streams = [torch.cuda.Stream() for _ in tensors]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [sa.qk_norm_rope_bwd(*t, w, w, freq, stream=s) for t, s in zip(tensors, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for a, b in zip(got, want) for x, y in zip(a, b))


def test_infinities_and_nan_stay_in_their_pair(cuda_dev):
    """The rotation of a pair says nothing about the channels beside it."""
    for inter, R in ((False, 32), (True, 32), (False, 36)):
        freq = sa.rope_frequencies(R, device=cuda_dev)[0]
        x = rows(110, 1, 2, 1, 64, dtype=torch.float32)
        x[0, 0, 0, 2], x[0, 1, 0, 40] = math.inf, math.nan
        y = sa.rope_fwd(x.to(cuda_dev), None, freq, interleaved=inter)[0].cpu()
        clean = torch.ones(64, dtype=torch.bool)
        clean[[2, 3] if inter else [2, 2 + R // 2]] = False
        assert torch.isfinite(y[0, 0, 0][clean]).all() and not torch.isfinite(y[0, 0, 0, 2])
        clean = torch.ones(64, dtype=torch.bool)
        clean[40] = False
        assert torch.isfinite(y[0, 1, 0][clean]).all() and torch.isnan(y[0, 1, 0, 40])


def test_no_rows(cuda_dev):
    freq = sa.rope_frequencies(64, device=cuda_dev)[0]
    w = torch.ones(64, device=cuda_dev, dtype=torch.bfloat16)
    x = torch.empty((2, 0, 4, 64), dtype=torch.bfloat16, device=cuda_dev)
    assert sa.rope_fwd(x, x, freq)[0].shape == x.shape
    dq, dk, dqw, dkw = sa.qk_norm_rope_bwd(x, x, x, x, w, w, freq)
    assert dq.shape == x.shape and not dqw.any() and not dkw.any()
    some = torch.randn((1, 3, 4, 64), device=cuda_dev).bfloat16()
    none = some[:, :, :0]
    _, _, dqw, dkw = sa.qk_norm_rope_bwd(some, none, some, none, w, w, freq)
    assert dqw.any() and not dkw.any()


def test_large_strides(cuda_dev):
    """Rows past 2^31 elements."""
    freq = sa.rope_frequencies(128, device=cuda_dev)[0]
    far = torch.empty(2 ** 31 + 4096, dtype=torch.bfloat16, device=cuda_dev)
    q = torch.as_strided(far, (2, 2, 2, 128), (2 ** 31, 256, 128, 1))
    q.copy_(rows(120, 2, 2, 2, 128, dtype=torch.bfloat16))
    want = sa.rope_fwd(q.contiguous(), None, freq)[0]
    w = torch.ones(128, device=cuda_dev)
    norm = sa.qk_norm_rope_fwd(q.contiguous(), None, w, None, freq)[0]
    assert torch.equal(sa.rope_fwd(q, None, freq)[0], want)
    assert torch.equal(sa.qk_norm_rope_fwd(q, None, w, None, freq, q_out=q)[0], norm)
