"""The row-by-row error model (train_rows.py) on the host: results rounded once pass it, and a mistake in a single row, key
or remainder tile of a long problem does not, which the elementwise worst-case bounds of train_ref.py let through (CPU)."""
import pytest
import torch

from train_ref import Reference
from train_rows import FACTOR, worst_rows


def problem(Sq, Sk, Hq=2, Hkv=1, causal=False):
    g = torch.Generator().manual_seed(Sq + Sk)
    r = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)   # noqa: E731
    q, k, v, d = r(1, Sq, Hq, 128), r(1, Sk, Hkv, 128), r(1, Sk, Hkv, 128), r(1, Sq, Hq, 128)
    ref = Reference(q, k, v, causal=causal)
    ref.backward(d)
    results = {"o": ref.out(), "dq": ref.dq, "dk": ref.dk, "dv": ref.dv}
    return ref, d, {n: t.to(torch.bfloat16) for n, t in results.items()}


def parts(ref, d):
    """p and ds [B, Hq, Sq, Sk], and ds without delta."""
    dp = d.double().permute(0, 2, 1, 3) @ ref.v.transpose(-1, -2)
    return ref.p, ref.p * (dp - (ref.p * dp).sum(-1, keepdim=True)), ref.p * dp


@pytest.mark.parametrize("Sq,Sk,causal", [(1000, 1000, True), (1000, 1000, False), (3, 6000, False), (700, 130, False),
                                          (40, 60, True)])
def test_results_rounded_once_pass(Sq, Sk, causal):
    ref, d, got = problem(Sq, Sk, causal=causal)
    far = worst_rows(got, ref, d)
    # a rounding's largest error is sqrt(3) times its mean square one
    assert max(far.values()) <= 3 ** 0.5, far


@pytest.mark.parametrize("Sq,Sk", [(1000, 1000), (700, 900), (3, 6000)])
@pytest.mark.parametrize("mistake", ["no delta", "x 1.3", "last keys", "first keys", "zero"])
def test_one_row_of_dq(Sq, Sk, mistake):
    ref, d, got = problem(Sq, Sk, causal=Sq == 1000)
    p, ds, raw = parts(ref, d)
    row, head = Sq - 1, 1
    x = ds[0, head, row].clone()
    if mistake == "no delta":
        x = raw[0, head, row]
    elif mistake == "x 1.3":
        x = 1.3 * x
    elif mistake == "last keys":
        x[-32:] = 0
    elif mistake == "first keys":
        x[:32] = 0
    else:
        x = 0 * x
    got["dq"][0, row, head] = (ref.scale * x @ ref.k[0, head]).to(torch.bfloat16)
    far = worst_rows(got, ref, d)
    assert far["dq"] > FACTOR and max(far[n] for n in ("o", "dk", "dv")) < FACTOR


@pytest.mark.parametrize("Sq,Sk", [(1000, 1000), (900, 700), (6000, 3)])
@pytest.mark.parametrize("mistake", ["x 1.3", "last queries", "no delta", "other head missing"])
def test_one_key_of_dk_and_dv(Sq, Sk, mistake):
    ref, d, got = problem(Sq, Sk)
    p, ds, raw = parts(ref, d)
    key = Sk - 1
    a, b = p[0, :, :, key].clone(), ds[0, :, :, key].clone()
    if mistake == "x 1.3":
        a, b = 1.3 * a, 1.3 * b
    elif mistake == "last queries":
        # (of 6000 queries on 3 keys that many come to no more than the rounding)
        a[:, -Sq // 8:] = 0
        b[:, -Sq // 8:] = 0
    elif mistake == "no delta":
        b = raw[0, :, :, key]
    else:
        a[1], b[1] = 0, 0
    got["dv"][0, key, 0] = torch.einsum("hi,hid->d", a, d.double()[0].transpose(0, 1)).to(torch.bfloat16)
    got["dk"][0, key, 0] = (ref.scale * torch.einsum("hi,hid->d", b, ref.q[0])).to(torch.bfloat16)
    far = worst_rows(got, ref, d)
    assert far["dk"] > FACTOR and max(far["o"], far["dq"]) < FACTOR
    assert mistake == "no delta" or far["dv"] > FACTOR


@pytest.mark.parametrize("mistake", ["x 1.02", "last keys"])
def test_one_row_of_o(mistake):
    ref, d, got = problem(700, 900)
    x = ref.p[0, 1, 699].clone()
    if mistake == "last keys":
        x[-4:] = 0
    else:
        x = 1.02 * x
    got["o"][0, 699, 1] = (x @ ref.v[0, 1]).to(torch.bfloat16)
    assert worst_rows(got, ref, d)["o"] > FACTOR
