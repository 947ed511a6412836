"""qk_norm_rope_bwd with weights and gradients left out, eps = 0 and expanded inputs, against its definition in 64 bits."""
import ctypes

import pytest
import torch

import rope_ref as ref
import sage_attention_forward_gb300 as sa

pytestmark = pytest.mark.gpu
TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def rows(seed, *shape, dtype, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * gain).to(dtype)


def strides(t):
    return (ctypes.c_int64 * 3)(*t.stride()[:3])


def backward(dq_out, dk_out, q, k, q_weight, k_weight, freq, eps, interleaved, wanted):
    """The C call, float32 weights; wanted: which of dq_weight and dk_weight are asked for (the others are NULL)."""
    B, S, Hq, N = q.shape
    L, dq, dk = sa.lib(), torch.empty_like(q), torch.empty_like(k)
    dw = [torch.empty(N, device=q.device) if w else None for w in wanted]
    ws = torch.empty(L.qk_norm_rope_bwd_workspace_size(B, S, Hq, k.shape[2], N), dtype=torch.uint8, device=q.device)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    held = [strides(t) for t in (dq_out, dk_out, q, k, dq, dk)]
    status = L.qk_norm_rope_bwd(
        dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), k.data_ptr(), ptr(q_weight), ptr(k_weight), dq.data_ptr(),
        dk.data_ptr(), *map(ptr, dw), B, S, Hq, k.shape[2], N, *held, eps, None, None, 1, ptr(freq), 2 * len(freq), interleaved,
        1.0, TYPES[q.dtype], 2, ws.data_ptr() if any(wanted) else None, ws.numel() if any(wanted) else 0,
        torch.cuda.current_stream().cuda_stream)
    assert status == 0, L.attn_last_error()
    return dq, dk, *dw


def check(got, x, dy, weights, freq, eps, interleaved):
    """got: dq, dk, dq_weight, dk_weight (a None is not looked at); x, dy: Q's and K's, on the CPU."""
    B, S, _, N = x[0].shape
    cos, sin = ref.cos_sin(freq.cpu(), None, B, S, 1.0)
    for i, name in enumerate("qk"):
        w = torch.ones(N, dtype=torch.float64) if weights[i] is None else weights[i].cpu().double()
        dx, bound, dw, dw_bound = ref.norm_rope_bwd(dy[i].double(), x[i].double(), w, eps, cos, sin, interleaved, 1.0)
        ref.near(got[i], dx, bound, "d" + name)
        if got[2 + i] is not None:
            ref.near(got[2 + i], dw, dw_bound, f"d{name}_weight")


# channels, rotated, interleaved, type: halves, neighbours, halves that are no whole pieces, by the channel
MAPS = [(128, 128, False, torch.bfloat16), (128, 64, True, torch.bfloat16), (128, 90, False, torch.float16),
        (77, 30, False, torch.bfloat16), (64, 64, False, torch.float32)]


@pytest.mark.parametrize("weighted,wanted", [((1, 1), (0, 1)), ((1, 1), (1, 0)), ((1, 1), (0, 0)), ((0, 1), (0, 1)),
                                             ((1, 0), (1, 0))])
@pytest.mark.parametrize("N,R,interleaved,dtype", MAPS)
def test_weights_and_gradients_left_out(N, R, interleaved, dtype, weighted, wanted, cuda_dev):
    """Q's and K's weights far apart, several units a warp: each side's gradients are formed with its own weights."""
    B, S, Hq, Hk = 1, 3001, 6, 5
    freq = sa.rope_frequencies(R, device=cuda_dev)[0]
    x = rows(1, B, S, Hq, N, dtype=dtype), rows(2, B, S, Hk, N, dtype=dtype)
    dy = rows(3, B, S, Hq, N, dtype=dtype, gain=0.1), rows(4, B, S, Hk, N, dtype=dtype, gain=0.1)
    weights = [(gain + rows(5 + i, N, dtype=torch.float32, gain=0.2)).to(cuda_dev) if weighted[i] else None
               for i, gain in enumerate((1.0, 9.0))]
    dev = [t.to(cuda_dev) for t in (*dy, *x)]
    got = backward(*dev, *weights, freq, 1e-5, interleaved, wanted)
    check(got, x, dy, weights, freq, 1e-5, interleaved)
    for _ in range(5):
        again = backward(*dev, *weights, freq, 1e-5, interleaved, wanted)
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(again, got))
    if weighted == wanted:
        bound = sa.qk_norm_rope_bwd(*dev, *weights, freq, eps=1e-5, interleaved=interleaved)
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(bound, got))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("heads", [(1, 3), (3, 5), (5, 1), (7, 2)])
@pytest.mark.parametrize("N,R,interleaved", [(128, 128, False), (128, 90, False), (80, 32, True), (64, 64, False), (58, 58, True),
                                             (160, 64, False), (61, 40, False)])
def test_eps_of_zero(N, R, interleaved, heads, dtype, cuda_dev):
    """Rows that are not zeros have finite results, however many of a warp's places have no head."""
    B, S = 2, 7
    freq = sa.rope_frequencies(R, device=cuda_dev)[0]
    x = [rows(20 + i, B, S, H, N, dtype=dtype) for i, H in enumerate(heads)]
    dy = [rows(22 + i, B, S, H, N, dtype=dtype, gain=0.1) for i, H in enumerate(heads)]
    weights = [(1 + rows(24 + i, N, dtype=torch.float32, gain=0.2)).to(cuda_dev) for i in range(2)]
    dev = [t.to(cuda_dev) for t in (*dy, *x)]
    check(sa.qk_norm_rope_bwd(*dev, *weights, freq, eps=0.0, interleaved=interleaved), x, dy, weights, freq, 0.0, interleaved)
    cos, sin = ref.cos_sin(freq.cpu(), None, B, S, 1.0)
    for t, y, w in zip(x, sa.qk_norm_rope_fwd(*dev[2:], *weights, freq, eps=0.0, interleaved=interleaved), weights):
        ref.near(y, *ref.norm_rope(t.double(), w.cpu().double(), 0.0, cos, sin, interleaved, 1.0), "y")


def test_eps_of_zero_and_a_row_of_zeros(cuda_dev):
    """Zeros come out, and the other rows' part of dw is what it is without that row."""
    freq = sa.rope_frequencies(128, device=cuda_dev)[0]
    x = rows(30, 1, 9, 3, 128, dtype=torch.float32).to(cuda_dev)
    dy = rows(31, 1, 9, 3, 128, dtype=torch.float32).to(cuda_dev)
    w = torch.ones(128, device=cuda_dev)
    x[0, 4] = 0
    y = sa.qk_norm_rope_fwd(x, None, w, None, freq, eps=0.0)[0]
    assert not y[0, 4].any() and torch.isfinite(y).all()
    dx, _, dw, _ = sa.qk_norm_rope_bwd(dy, None, x, None, w, None, freq, eps=0.0)
    dy[0, 4] = 0
    other, _, dw_other, _ = sa.qk_norm_rope_bwd(dy, None, x, None, w, None, freq, eps=0.0)
    seen = [s for s in range(9) if s != 4]
    assert torch.equal(dw, dw_other) and torch.equal(dx[0, seen], other[0, seen]) and torch.isfinite(dx).all()


def test_gradients_that_must_be_given(cuda_dev):
    x, w = torch.ones((1, 2, 2, 64), device=cuda_dev), torch.ones(64, device=cuda_dev)
    for dq_out, dk_out, k in ((None, x, x), (x, None, x), (None, None, None), (x, x, None)):
        with pytest.raises(ValueError, match="dq_out|dk_out"):
            sa.qk_norm_rope_bwd(dq_out, dk_out, x, k, w, None, None)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N,R", [(128, 128), (128, 90), (77, 30)])
def test_expanded_gradients_and_inputs(N, R, interleaved, cuda_dev):
    """Strides of 0 (a gradient that a sum or a mean hands on, one row for all heads) give the bits of the same tensor written out."""
    B, S, H = 2, 5, 3
    freq = sa.rope_frequencies(R, device=cuda_dev)[0]
    w = (1 + rows(40, N, dtype=torch.float32, gain=0.2)).to(cuda_dev)
    x, y = (rows(41 + i, B, S, H, N, dtype=torch.bfloat16).to(cuda_dev) for i in range(2))
    one = rows(43, N, dtype=torch.bfloat16).to(cuda_dev)
    shapes = [one.expand(B, S, H, N), x[:, :1].expand(B, S, H, N), x[:, :, 1:2].expand(B, S, H, N), x[:1].expand(B, S, H, N)]
    same = lambda a, b: all(p is q is None or torch.equal(p, q) for p, q in zip(a, b))  # noqa: E731
    for t in shapes:
        assert t.stride(3) == 1 and 0 in t.stride()
        full = t.clone(memory_format=torch.contiguous_format)
        assert same(sa.rope_bwd(t, y, freq, interleaved=interleaved), sa.rope_bwd(full, y, freq, interleaved=interleaved))
        for a, b in (((t, y, x, y), (full, y, x, y)), ((y, x, t, y), (y, x, full, y)), ((t, t, t, t), (full, full, full, full))):
            assert same(sa.qk_norm_rope_bwd(*a, w, w, freq, interleaved=interleaved),
                        sa.qk_norm_rope_bwd(*b, w, w, freq, interleaved=interleaved))
