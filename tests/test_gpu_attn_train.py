"""attn_fwd_bf16_lse and attn_bwd_bf16 against 64 bits, elementwise within the bounds that
train_ref.py derives: lengths from one row, ragged tiles, shared key heads, causal masks,
per-entry key counts (zero among them), NaN in the padding, strided views, other streams, graphs."""
import math

import pytest
import torch

import sage_attention_forward_gb300 as sa
from train_ref import Reference, worst

pytestmark = pytest.mark.gpu


def make(dev, B, Sq, Sk, Hq, Hkv, seed=0, gain=1.0):
    g = torch.Generator(device=dev).manual_seed(1000 + seed)
    r = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    q, k, v, d = r(B, Sq, Hq, 128) * gain, r(B, Sk, Hkv, 128), r(B, Sk, Hkv, 128), r(B, Sq, Hq, 128) * 0.1
    return tuple(t.to(torch.bfloat16) for t in (q, k, v, d))


def check(q, k, v, d, scale=None, causal=False, kv_len=None, grads=True, ref_args=None, cosine=True):
    o, lse = sa.attn_fwd_bf16_lse(q, k, v, softmax_scale=scale, causal=causal, kv_len=kv_len)
    got = sa.attn_bwd_bf16(d, q, k, v, o, lse, softmax_scale=scale, causal=causal, kv_len=kv_len) if grads else ()
    torch.cuda.synchronize()
    sa.attn_get_device_status()
    ref = Reference(*(ref_args or (q, k, v)), scale, causal, kv_len)
    empty = torch.isinf(ref.lse)
    assert torch.equal(torch.isneginf(lse), empty)
    far = {"o": worst(o, ref.out(), ref.o_tol.permute(0, 2, 1, 3)),
           "lse": worst(torch.where(empty, torch.zeros_like(lse), lse), torch.where(empty, 0.0, ref.lse), ref.lse_tol)}
    if grads:
        ref.backward(d)
        for name, t in zip(("dq", "dk", "dv"), got):
            far[name] = worst(t, getattr(ref, name), getattr(ref, name + "_tol"))
            want = getattr(ref, name)
            cos = float((t.double() * want).sum() / (t.double().norm() * want.norm() + 1e-300))
            assert not cosine or float(want.norm()) < 1e-12 or cos > 0.9999, (name, cos)
    print(far)
    assert max(far.values()) <= 1.0, far
    return o, lse, got


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,Sq,Sk,Hq,Hkv", [
    (1, 1, 1, 1, 1), (1, 1, 129, 2, 1), (1, 130, 1, 1, 1), (2, 2, 3, 2, 2), (1, 128, 128, 1, 1), (1, 129, 127, 2, 2),
    (2, 200, 300, 6, 2), (1, 513, 257, 4, 1), (1, 257, 700, 3, 3), (1, 1000, 1000, 2, 2), (3, 384, 640, 8, 1)])
def test_shapes(cuda_dev, B, Sq, Sk, Hq, Hkv, causal):
    check(*make(cuda_dev, B, Sq, Sk, Hq, Hkv, seed=Sq + Sk), causal=causal)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Sq,Sk,lens", [(300, 300, [300, 1, 0, 129]), (70, 520, [128, 127, 129, 520]),
                                        (260, 40, [0, 40, 2, 1]), (1, 300, [1, 0, 300, 200]), (130, 256, [-5, 900, 256, 3])])
def test_key_counts_and_garbage_padding(cuda_dev, Sq, Sk, lens, causal):
    """Counts from zero to all (and outside [0, Sk], clamped); the padding holds NaN and infinities."""
    q, k, v, d = make(cuda_dev, len(lens), Sq, Sk, 4, 2, seed=7)
    n = torch.tensor(lens, dtype=torch.int32, device=cuda_dev)
    kk, vv = k.clone(), v.clone()
    for b, x in enumerate(lens):
        x = min(max(x, 0), Sk)
        kk[b, x:] = math.nan
        vv[b, x:] = math.inf
        kk[b, x + 1:] = -math.inf
        vv[b, x + 2:] = math.nan
    check(q, kk, vv, d, causal=causal, kv_len=n)


def test_zero_and_other_scales(cuda_dev):
    q, k, v, d = make(cuda_dev, 1, 200, 333, 2, 1, seed=3)
    for scale in (0.0, 0.02, 0.5):
        check(q, k, v, d, scale=scale)


def test_large_scores(cuda_dev):
    """Rows whose softmax is one key, next to ordinary ones: the reference maximum moves far."""
    q, k, v, d = make(cuda_dev, 1, 300, 500, 2, 2, seed=4)
    q = (q.float() * torch.pow(2.0, torch.tensor([0, 2, 4, 6], device=cuda_dev).repeat_interleave(75)).view(1, 300, 1, 1))
    check(q.to(torch.bfloat16), k, v, d, causal=False)


def test_strided_views(cuda_dev):
    """Q, K and V as slices of one projection, O and the gradients into slices of wider buffers."""
    B, S, H = 2, 190, 3
    g = torch.Generator(device=cuda_dev).manual_seed(5)
    qkv = torch.randn((B, S, 3, H, 128), generator=g, device=cuda_dev).to(torch.bfloat16)
    q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    d = torch.randn((B, H, S, 128), generator=g, device=cuda_dev).to(torch.bfloat16).permute(0, 2, 1, 3)
    o, lse, (dq, dk, dv) = check(q, k, v, d)
    wide = torch.full((B, S, 3, H, 136), 7.0, dtype=torch.bfloat16, device=cuda_dev)
    o2 = torch.empty((B, H, S, 128), dtype=torch.bfloat16, device=cuda_dev).permute(0, 2, 1, 3)
    sa.attn_fwd_bf16_lse(q, k, v, out=o2)
    views = [wide[:, :, i, :, :128] for i in range(3)]
    sa.attn_bwd_bf16(d, q, k, v, o2, lse, dq=views[0], dk=views[1], dv=views[2])
    assert torch.equal(o2, o) and all(torch.equal(a, b) for a, b in zip(views, (dq, dk, dv)))
    assert bool((wide[..., 128:] == 7).all())


def test_same_forward_as_attn_fwd_bf16(cuda_dev):
    """Without masks the forward is the BF16 forward."""
    q, k, v, _ = make(cuda_dev, 1, 700, 700, 2, 2, seed=6)
    o, _ = sa.attn_fwd_bf16_lse(q, k, v)
    assert torch.equal(o, sa.attn_fwd_bf16(q, k, v))


def test_only_the_gradients_rows_are_written(cuda_dev):
    """Buffers that hold more rows than the call has: the rest stays."""
    q, k, v, d = make(cuda_dev, 1, 100, 90, 2, 2, seed=8)
    o, lse = sa.attn_fwd_bf16_lse(q, k, v)
    want = sa.attn_bwd_bf16(d, q, k, v, o, lse)
    big = [torch.full((1, 256, 2, 128), 3.0, dtype=torch.bfloat16, device=cuda_dev) for _ in range(3)]
    n = [100, 90, 90]
    sa.attn_bwd_bf16(d, q, k, v, o, lse, dq=big[0][:, :100], dk=big[1][:, :90], dv=big[2][:, :90])
    for t, w, x in zip(big, want, n):
        assert torch.equal(t[:, :x], w) and bool((t[:, x:] == 3).all())


def test_repeats_on_another_stream_and_in_a_graph(cuda_dev):
    q, k, v, d = make(cuda_dev, 2, 400, 333, 4, 2, seed=9)
    n = torch.tensor([333, 200], dtype=torch.int32, device=cuda_dev)

    def step(stream=None):
        o, lse = sa.attn_fwd_bf16_lse(q, k, v, causal=True, kv_len=n, stream=stream)
        return (o, lse) + sa.attn_bwd_bf16(d, q, k, v, o, lse, causal=True, kv_len=n, stream=stream)

    first = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    other = step(stream=s)                 # every buffer of these calls belongs to s
    by_handle = step(stream=s.cuda_stream)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    assert all(torch.equal(a, b) for a, b in zip(first, by_handle))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = step()
    # the captured call reads the counts when it is replayed
    n.copy_(torch.tensor([100, 0], dtype=torch.int32))
    q.mul_(0.5)
    graph.replay()
    again = step()
    torch.cuda.synchronize()
    sa.attn_get_device_status()
    assert all(torch.equal(a, b) for a, b in zip(caught, again))
    assert not torch.equal(caught[0], first[0])


def test_two_graphs_at_once(cuda_dev):
    """Two captured steps on two streams keep their workspaces apart."""
    cases = [make(cuda_dev, 1, 500 + 20 * i, 600, 4, 4, seed=20 + i) for i in range(2)]

    def step(c):
        q, k, v, d = c
        o, lse = sa.attn_fwd_bf16_lse(q, k, v)
        return sa.attn_bwd_bf16(d, q, k, v, o, lse)

    want = [step(c) for c in cases]
    graphs, outs = [], []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(c))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(a, b) for a, b in zip(w, o))


def test_gradient_matches_differences_of_the_forward(cuda_dev):
    """<dQ, x> against a central difference of the 64-bit forward along x."""
    q, k, v, d = make(cuda_dev, 1, 150, 200, 2, 1, seed=11)
    o, lse = sa.attn_fwd_bf16_lse(q, k, v, causal=True)
    grads = sa.attn_bwd_bf16(d, q, k, v, o, lse, causal=True)
    ref = Reference(q, k, v, causal=True)
    ref.backward(d)
    args = [t.double() for t in (q, k, v)]
    f = lambda a: float((Reference(*a, causal=True).out() * d.double()).sum())  # noqa: E731
    h = 1e-5
    for at, (grad, tol) in enumerate(zip(grads, (ref.dq_tol, ref.dk_tol, ref.dv_tol))):
        x = torch.randn(grad.shape, generator=torch.Generator().manual_seed(at), dtype=torch.float64).to(cuda_dev)
        up, down = list(args), list(args)
        up[at], down[at] = args[at] + h * x, args[at] - h * x
        far = abs((f(up) - f(down)) / (2 * h) - float((grad.double() * x).sum()))
        assert far <= float((tol * x.abs()).sum()) + 1e-6


def test_long_axis(cuda_dev):
    """Few keys under many queries, and few queries over many keys."""
    check(*make(cuda_dev, 1, 6000, 130, 2, 1, seed=12))
    check(*make(cuda_dev, 1, 3, 6000, 2, 1, seed=13), causal=True)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,Sq,Sk,Hq,Hkv,lens", [
    (3, 300, 300, 64, 64, [300, 1, 0]), (2, 520, 200, 96, 32, [200, 130]), (5, 100, 700, 80, 40, [0, 700, 0, 129, 640]),
    (1, 700, 1100, 100, 100, None)])
def test_more_items_than_sms(cuda_dev, B, Sq, Sk, Hq, Hkv, lens, causal):
    """Each CTA takes several items: long ones, short ones and empty ones after one another."""
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=cuda_dev)
    check(*make(cuda_dev, B, Sq, Sk, Hq, Hkv, seed=30 + B), causal=causal, kv_len=n)


def test_empty_problem(cuda_dev):
    z = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=cuda_dev)  # noqa: E731
    o, lse = sa.attn_fwd_bf16_lse(z(0, 30, 2, 128), z(0, 40, 2, 128), z(0, 40, 2, 128))
    assert o.shape == (0, 30, 2, 128) and lse.shape == (0, 2, 30)
    dq, dk, dv = sa.attn_bwd_bf16(o, z(0, 30, 2, 128), z(0, 40, 2, 128), z(0, 40, 2, 128), o, lse)
    assert dq.shape == o.shape and dk.shape == dv.shape == (0, 40, 2, 128)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,Sq,Sk,Hq,Hkv,lens", [
    (1, 2000, 130, 4, 2, None), (1, 1500, 128, 3, 3, [77]), (2, 1111, 257, 4, 1, [257, 0]), (1, 700, 1, 8, 1, None),
    (1, 130, 400, 40, 1, [300]), (1, 3000, 300, 2, 1, [1])])
def test_divided_sums(cuda_dev, B, Sq, Sk, Hq, Hkv, lens, causal):
    """Few key tiles and many products: dK and dV are formed in parts, which the workspace holds."""
    rows = 2 * B * Hq * ((Sq + 127) // 128 * 128) * 4
    assert sa.attn_bwd_workspace(B, Sq, Sk, Hq, Hkv, "cpu").numel() > rows
    kv_len = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=cuda_dev)
    q, k, v, d = make(cuda_dev, B, Sq, Sk, Hq, Hkv, seed=Sq)
    o, lse, got = check(q, k, v, d, causal=causal, kv_len=kv_len)
    again = sa.attn_bwd_bf16(d, q, k, v, o, lse, causal=causal, kv_len=kv_len)
    for a, b in zip(got, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,Sq,Sk,Hq,Hkv,lens", [(2, 300, 2, 4, 4, None), (1, 500, 3, 2, 1, None), (3, 77, 5, 2, 2, [5, 2, 4]),
                                                 (2, 90, 90, 4, 2, None), (1, 128, 128, 3, 3, [100])])
def test_few_keys(cuda_dev, B, Sq, Sk, Hq, Hkv, lens, causal):
    """With all keys in one tile the gradients do not carry O's rounding: train_ref's bounds without it."""
    kv_len = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=cuda_dev)
    q, k, v, d = make(cuda_dev, B, Sq, Sk, Hq, Hkv, seed=Sq + Sk)
    o, lse = sa.attn_fwd_bf16_lse(q, k, v, causal=causal, kv_len=kv_len)
    got = sa.attn_bwd_bf16(d, q, k, v, o, lse, causal=causal, kv_len=kv_len)
    torch.cuda.synchronize()
    sa.attn_get_device_status()
    ref = Reference(q, k, v, None, causal, kv_len)
    ref.o_tol = 0 * ref.o_tol
    # delta is a sum of up to 128 FP32 products p dp, each p off by its own bound
    ref.backward(d)
    dp = ref.dp = (d.double().permute(0, 2, 1, 3) @ ref.v.transpose(-1, -2)).abs()
    e_delta = (ref.p * dp * (ref.e_p + 2.0 ** -16)).sum(-1, keepdim=True)
    more = ref.p * e_delta
    tol = {"dq": ref.dq_tol + (ref.scale * more @ ref.k.abs()).permute(0, 2, 1, 3),
           "dk": ref.dk_tol + ref.shared(ref.scale * more.transpose(-1, -2) @ ref.q.abs()), "dv": ref.dv_tol}
    far = {name: worst(t, getattr(ref, name), tol[name]) for name, t in zip(("dq", "dk", "dv"), got)}
    print(far, [float((t.double() - getattr(ref, n)).norm() / getattr(ref, n).norm().clamp_min(1e-30))
                for n, t in zip(("dq", "dk", "dv"), got)])
    assert max(far.values()) <= 1, far


@pytest.mark.parametrize("offset", [0.5, 4.0])
def test_keys_with_a_mean(cuda_dev, offset):
    """Keys with channels of their own mean, `offset` times their spread: a row of dS has the sum 0, so that the mean
    does not come into dQ, but for the rounding of the parts in the tile that makes up for the others'.  Errors of
    rounding are at most u / sqrt(3) of their value in the mean square: dQ's own, those of its terms, and offset^2 of
    those of 128 keys of 1200; 1.1 for the offsets drawn.  (All keys' would be 0.0106 with 4.)"""
    g = torch.Generator(device=cuda_dev).manual_seed(5)
    q, k, v, d = make(cuda_dev, 1, 1200, 1200, 2, 2, seed=44)
    k = (k.float() + offset * torch.randn(2, 128, generator=g, device=cuda_dev)).to(torch.bfloat16)
    o, lse, got = check(q, k, v, d)
    ref = Reference(q, k, v)
    ref.backward(d)
    err = float((got[0].double() - ref.dq).norm() / ref.dq.norm())
    print(err)
    assert err <= 1.1 * 2.0 ** -8 * math.sqrt((2 + offset ** 2 * 128 / 1200) / 3)


def test_key_counts_out_of_range_are_clamped(cuda_dev):
    q, k, v, d = make(cuda_dev, 3, 150, 140, 4, 2, seed=9)
    wild = torch.tensor([-7, 10 ** 9, 133], dtype=torch.int32, device=cuda_dev)
    tame = torch.tensor([0, 140, 133], dtype=torch.int32, device=cuda_dev)
    for causal in (False, True):
        a = check(q, k, v, d, causal=causal, kv_len=tame)
        o, lse = sa.attn_fwd_bf16_lse(q, k, v, causal=causal, kv_len=wild)
        b = sa.attn_bwd_bf16(d, q, k, v, o, lse, causal=causal, kv_len=wild)
        assert torch.equal(o, a[0]) and torch.equal(lse, a[1])
        for x, y in zip(a[2], b):
            assert torch.equal(x, y)


def test_more_heads_than_a_grid_dimension(cuda_dev):
    """70000 (batch entry, head) pairs of a few rows each, against four of them at a time."""
    B, H = 700, 100
    q, k, v, d = make(cuda_dev, B, 5, 3, H, H, seed=10)
    o, lse = sa.attn_fwd_bf16_lse(q, k, v, causal=True)
    got = (o, lse.transpose(1, 2), *sa.attn_bwd_bf16(d, q, k, v, o, lse, causal=True))
    for b in (0, 1, 327, 654, 655, 656, B - 1):
        part = [t[b:b + 1, :, 60:64] for t in (q, k, v, d)]
        po, plse = sa.attn_fwd_bf16_lse(*part[:3], causal=True)
        want = (po, plse.transpose(1, 2), *sa.attn_bwd_bf16(part[3], *part[:3], po, plse, causal=True))
        for x, y in zip(got, want):
            assert torch.equal(x[b:b + 1, :, 60:64], y)
    sa.attn_get_device_status()


def test_strides_past_32_bits(cuda_dev):
    """Batch entries 2^31 and more elements apart, of the inputs and of every output."""
    B, Sq, Sk, H, far = 2, 200, 300, 2, (1 << 31) + 1024
    store = torch.empty(far + (1 << 20), dtype=torch.bfloat16, device=cuda_dev)
    used = 0

    def spread(t):
        nonlocal used
        S, heads = t.shape[1], t.shape[2]
        out = store.as_strided((B, S, heads, 128), (far, heads * 128, 128, 1), used)
        used += S * heads * 128
        out.copy_(t)
        return out

    tensors = make(cuda_dev, B, Sq, Sk, H, H, seed=11)
    q, k, v, d = (spread(t) for t in tensors)
    o = spread(torch.zeros_like(tensors[0]))
    grads = [spread(torch.zeros_like(t)) for t in tensors[:3]]
    _, lse = sa.attn_fwd_bf16_lse(q, k, v, causal=True, out=o)
    sa.attn_bwd_bf16(d, q, k, v, o, lse, causal=True, dq=grads[0], dk=grads[1], dv=grads[2])
    wo, wlse, want = check(*tensors, causal=True)
    assert used <= 1 << 20 and torch.equal(o, wo) and torch.equal(lse, wlse)
    for x, y in zip(grads, want):
        assert torch.equal(x, y)


def test_one_tensor_as_queries_keys_and_values(cuda_dev):
    """Within the bounds.  A row's own key has nearly all of its probability here (scores of 11 against 1), so that
    dp - delta is of the size of the rounding of O in delta, and dQ of that of its error: the bounds count
    that (e_delta times |k|), a cosine of 0.9999 does not follow from them."""
    x, _, _, d = make(cuda_dev, 1, 260, 260, 3, 3, seed=12)
    check(x, x, x, d, causal=True, cosine=False)


def test_two_streams_at_once(cuda_dev):
    """Calls under way on two streams, each with its own outputs and workspace, give what they give alone."""
    cases = [make(cuda_dev, 1, 1500, 1500, 4, 2, seed=20 + i) for i in range(2)]
    alone = []
    for q, k, v, d in cases:
        o, lse = sa.attn_fwd_bf16_lse(q, k, v, causal=True)
        alone.append((o, lse, *sa.attn_bwd_bf16(d, q, k, v, o, lse, causal=True)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = []
        for (q, k, v, d), s in zip(cases, streams):
            o, lse = sa.attn_fwd_bf16_lse(q, k, v, causal=True, stream=s)
            got.append((o, lse, *sa.attn_bwd_bf16(d, q, k, v, o, lse, causal=True, stream=s)))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            for x, y in zip(a, b):
                assert torch.equal(x, y)
    sa.attn_get_device_status()
