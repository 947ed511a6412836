"""The 64-bit attention gradient that the GPU tests compare with, against differences of the
64-bit forward and against itself with a mistake put in (CPU)."""
import pytest
import torch

from train_ref import Reference, worst


def inputs(seed, B, Sq, Sk, Hq, Hkv, D=16):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    return r(B, Sq, Hq, D), r(B, Sk, Hkv, D), r(B, Sk, Hkv, D), r(B, Sq, Hq, D)


@pytest.mark.parametrize("causal,lens", [(False, None), (True, None), (False, [3, 0]), (True, [2, 7])])
@pytest.mark.parametrize("Sq,Sk", [(5, 7), (7, 5), (1, 1)])
def test_gradient_matches_differences(causal, lens, Sq, Sk):
    q, k, v, dout = inputs(1, 2, Sq, Sk, 4, 2)
    n = None if lens is None else torch.tensor(lens)
    f = lambda q, k, v: float((Reference(q, k, v, 0.3, causal, n).out() * dout).sum())  # noqa: E731
    grads = Reference(q, k, v, 0.3, causal, n).backward(dout)
    h = 1e-5
    for at, grad in enumerate(grads):
        d = inputs(2 + at, 2, Sq, Sk, 4, 2)[at]
        args = [q, k, v]
        up, down = list(args), list(args)
        up[at], down[at] = args[at] + h * d, args[at] - h * d
        # central difference: h^2 / 6 of a third derivative of order 10, and 1e-15 / h of cancellation
        assert abs((f(*up) - f(*down)) / (2 * h) - float((grad * d).sum())) < 1e-7


@pytest.mark.parametrize("which", ["delta", "scale", "mask"])
def test_bounds_catch_a_planted_mistake(which):
    q, k, v, dout = inputs(5, 1, 40, 60, 2, 1, 128)
    ref = Reference(q, k, v, causal=True)
    ref.backward(dout)
    bad = Reference(q, k, v, causal=which != "mask")
    if which == "scale":      # ds never multiplied by the scale
        dq = bad.backward(dout)[0] / bad.scale
    elif which == "delta":
        d = dout.permute(0, 2, 1, 3)
        ds = bad.p * (d @ bad.v.transpose(-1, -2))
        dq = (bad.scale * ds @ bad.k).permute(0, 2, 1, 3)
    else:
        dq = bad.backward(dout)[0]
    assert worst(ref.dq, ref.dq, ref.dq_tol) == 0.0
    assert worst(dq, ref.dq, ref.dq_tol) > 3
