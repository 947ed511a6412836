"""Outputs of the training calls that share memory with an input or with one another are refused wherever they start;
slices of one buffer whose rows lie between one another's are not (CPU: the check is on the host, before anything of
the GPU is touched)."""
import ctypes
import random

import pytest
import torch

import sage_attention_forward_gb300 as sa

I64x3 = ctypes.c_int64 * 3
ARG = 1
BASE = 1 << 30   # where the tensors' storage is taken to be


def at(t):
    return BASE + 2 * t.storage_offset()


def st(t):
    return I64x3(*t.stride()[:3])


def store(n):
    return torch.empty(n, dtype=torch.bfloat16, device="meta")


def forward(q, k, v, o):
    B, Sq, Hq, D = q.shape
    return sa.lib().attn_fwd_bf16_lse(at(q), at(k), at(v), at(o), 1 << 20, B, Sq, k.shape[1], Hq, k.shape[2], D, st(q),
                                      st(k), st(v), st(o), 0.1, 0, None, None)


def backward(d, q, k, v, o, dq, dk, dv):
    B, Sq, Hq, D = q.shape
    return sa.lib().attn_bwd_bf16(at(d), at(q), at(k), at(v), at(o), 1 << 20, at(dq), at(dk), at(dv), B, Sq, k.shape[1], Hq,
                                  k.shape[2], D, *(st(t) for t in (d, q, k, v, o, dq, dk, dv)), 0.1, 0, None, 1 << 20,
                                  1 << 40, None)


def norm(x, y):
    return sa.lib().layer_norm_fwd(at(x), None, None, at(y), 1 << 20, 1 << 20, *x.shape, st(x), st(y), 1e-6, 0, 0, None)


def norm_backward(dy, x, dx):
    return sa.lib().layer_norm_bwd(at(dy), at(x), None, 1 << 20, 1 << 20, at(dx), None, None, *x.shape, st(dy), st(x),
                                   st(dx), 0, 0, None, 0, None)


def slots(B, S, H, n, D=128):
    """n tensors [B, S, H, D] as slices of one buffer [B, S, n, H, D]."""
    x = store(B * S * n * H * D).view(B, S, n, H, D)
    return [x[:, :, i] for i in range(n)]


def test_slices_of_one_buffer():
    q, k, v, o, d, dq, dk, dv = slots(2, 100, 3, 8)
    assert forward(q, k, v, o) != ARG
    assert backward(d, q, k, v, o, dq, dk, dv) != ARG
    for bad in (q, k, v):
        assert forward(q, k, v, bad) == ARG
    for bad in (d, q, k, v, o, dk, dv):
        assert backward(d, q, k, v, o, bad, dk, dv) == ARG
    assert norm(q, k) != ARG and norm(q, q) != ARG
    assert norm_backward(q, k, v) != ARG and norm_backward(q, k, q) != ARG and norm_backward(q, k, k) != ARG


def test_views_that_start_elsewhere():
    x = store(2 * 101 * 4 * 128).view(2, 101, 4, 128)
    other = store(1 << 30)[1 << 29:][:2 * 100 * 4 * 128].view(2, 100, 4, 128)
    k, v, d, o, dk, dv = (store(1 << 30)[(1 << 29) + i * (1 << 20):][:2 * 100 * 4 * 128].view(2, 100, 4, 128)
                          for i in range(1, 7))
    q, late = x[:, :100], x[:, 1:]       # the same rows, one later
    assert forward(q, k, v, late) == ARG and "overlap" in sa.lib().attn_last_error().decode()
    assert forward(q, k, v, other) != ARG
    assert backward(d, q, k, v, o, late, dk, dv) == ARG
    assert norm(q, late) == ARG and norm_backward(q, k, late) == ARG and norm_backward(k, q, late) == ARG
    heads = store(2 * 100 * 5 * 128).view(2, 100, 5, 128)
    assert forward(heads[:, :, :4], k, v, heads[:, :, 1:]) == ARG      # three heads of four
    # in place, but with the rows in another order
    square = store(64 * 64 * 2 * 128).view(64, 64, 2, 128)
    assert norm(square, square.transpose(0, 1)) == ARG
    assert norm_backward(square.transpose(0, 1), store(1 << 30)[1 << 29:][:square.numel()].view(square.shape), square) == ARG


def test_last_and_first_rows_next_to_each_other():
    x = store(4 * 50 * 2 * 128).view(4, 50, 2, 128)
    assert norm(x[:2], x[2:]) != ARG and norm(x[2:], x[:2]) != ARG
    assert norm(x[:3], x[1:]) == ARG
    by_row = x.permute(1, 0, 2, 3)
    assert norm(by_row[:, :2], by_row[:, 2:]) != ARG
    # batch entries of one between those of the other
    assert norm(x[::2], x[1::2]) != ARG
    # every second row as one tensor, all of the later ones as another: they share some
    assert norm(x[:1, :25], x[:1, 1::2]) == ARG


def test_random_layouts_against_the_bytes():
    """Small tensors of random strides and starts: the answer is that of marking their bytes."""
    rng = random.Random(7)
    seen = set()
    for _ in range(3000):
        shape = [rng.randint(1, 4) for _ in range(3)] + [8]
        views, taken = [], []
        for _ in range(2):
            order = rng.sample(range(3), 3)
            stride, step = [0, 0, 0], 8 * rng.randint(1, 3)
            for i in order:
                stride[i] = step
                step = step * shape[i] + 8 * rng.randint(0, 2)
            start = 8 * rng.randint(0, 40)
            views.append(store(1 << 16).as_strided(shape, (*stride, 1), start))
            rows = torch.arange(1 << 16).as_strided(shape, (*stride, 1), start)
            taken.append(rows)
        common = bool(torch.isin(taken[0], taken[1]).any())
        same = torch.equal(taken[0], taken[1])
        got = norm(*views) == ARG
        assert got == (common and not same), (shape, [v.stride() for v in views], [v.storage_offset() for v in views])
        seen.add((common, same))
    assert seen >= {(True, False), (False, False)}


@pytest.mark.parametrize("far", [1 << 37, (1 << 38) - 8])
def test_strides_beyond_any_memory(far):
    status = sa.lib().layer_norm_fwd(BASE, None, None, BASE + 256, 1 << 20, 1 << 20, 1 << 10, 1 << 10, 1 << 10, 128,
                                I64x3(far, far, far), I64x3(far, far, far), 1e-6, 0, 0, None)
    assert status not in (0, ARG)
