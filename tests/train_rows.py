"""What the training kernels' roundings come to, row by row: the expected error, in the mean square, of each row of O and
dQ and of each key's dK and dV (test helper, not a test file).  train_ref's elementwise bounds add up worst cases over
channels and keys and leave a wrong row of many keys room; an error of independent roundings is far below them.

A rounding to BF16 is off by at most u = 2^-8 of its value, so by at most u / sqrt(3) in the mean square over even
positions in a step (r2 = u^2 / 3 below).  What is rounded:
  O      each p before P V, and the result:            r2 (sum_j p_j^2 |v_j|^2 + |o|^2)
  dV     each p before P^T dO, and the result:         r2 (sum_i p_ij^2 |dO_i|^2 + |dv|^2)
  dQ     each ds before dS K, and the result.  Delta comes from the O that was rounded, which moves it by
             e = dO . (o as given - o)
         (known, not a matter of chance), and every ds of the row by -e p_j.  The sum of the row's rounded ds is taken
         off again: in proportion to p from the first 128 keys and, where another key has more than half of
         the probability, from that one with the weight 1.  With w the mean of those keys so weighted and W the
         sum of the weights, a key beyond the first 128 comes in as (k_j - w) times the rounding of
         p_j (dp_j - delta - e), one of the first 128 as k_j times that of p_j (dp_j - delta - e + e / W), and e
         itself as e (sum_j p_j k_j - w).
  dK     each ds before dS^T Q, and the result.  Its delta is the row's corrected one, which has the sum of the
         roundings of the ds beyond the first 128 keys in it; that comes in times p_ij.
FP32 is counted by 2^-20 of |dO| |v| in dp, 2^-19 (1 + scale |q| |k|) relative in p, and 2^-17 of the sum of
magnitudes in each sum."""
from __future__ import annotations

import torch

R2 = 2.0 ** -16 / 3
HALF = 0.51        # a key with more of a row's probability takes part of the row's rest
FACTOR = 4.0       # errors are asserted up to this many times the expected one


def expected(ref, dout, o):
    """ref: a Reference; o [B, Sq, Hq, D]: what the backward was given.  Expected squared errors of the rows of o and dq
    [B, Sq, Hq], and of dk and dv [B, Sk, Hkv]."""
    ref.backward(dout)
    d = dout.double().permute(0, 2, 1, 3)
    p, q, k, v, scale = ref.p, ref.q, ref.k, ref.v, ref.scale
    n2 = lambda t: t.square().sum(-1)                 # noqa: E731
    rows = lambda t: t.permute(0, 2, 1)               # noqa: E731
    keys = lambda t: ref.shared(t)                    # noqa: E731
    dp = d @ v.transpose(-1, -2)
    delta = (p * dp).sum(-1, keepdim=True)
    lone = (ref.lim == 1)[:, None, :, None]           # ds is exactly 0 there
    e = (d * (o.double().permute(0, 2, 1, 3) - ref.o)).sum(-1, keepdim=True)
    first = torch.arange(p.shape[-1], device=p.device) < 128
    weight = torch.where(first, p, (p > HALF).to(p.dtype))
    total = weight.sum(-1, keepdim=True)
    some = total > 1e-6
    total = torch.where(some, total, 1.0)
    w = torch.where(some, weight @ k / total, 0.0)
    ds = torch.where(lone, 0.0, p * (dp - delta))
    ds_q = torch.where(lone, 0.0, p * (dp - delta - e + torch.where(first & some, e / total, 0.0)))
    rel = 2.0 ** -19 * (1 + scale * n2(q).sqrt()[..., None] * n2(k).sqrt()[..., None, :])
    size = n2(d).sqrt()[..., None] * n2(v).sqrt()[..., None, :]
    fp32 = torch.where(lone, 0.0, (rel * ds).square() + (2.0 ** -20 * p * size).square())
    # |k_j - w|^2, and |k_j|^2 for the first keys
    off = n2(k)[..., None, :] + torch.where(first, 0.0, n2(w)[..., None] - 2 * w @ k.transpose(-1, -2)).clamp_min(
        -n2(k)[..., None, :])
    dq2 = ((R2 * ds_q.square() * off).sum(-1) + (fp32 @ n2(k)[..., None])[..., 0]
           + torch.where(lone, 0.0, e * (p @ k - w)).square().sum(-1) + n2(2.0 ** -17 * ds.abs() @ k.abs()))
    moved = torch.where(first, 0.0, R2 * ds_q.square()).sum(-1, keepdim=True)   # of dK's delta, squared
    dk2 = R2 * ds.square() + fp32 + torch.where(lone, 0.0, p.square() * moved)
    return {
        "o": rows(R2 * (p.square() @ n2(v)[..., None])[..., 0] + R2 * n2(ref.o)
                  + n2((2.0 ** -17 + rel.amax(-1, keepdim=True)) * (p @ v.abs()))),
        "dq": rows(scale ** 2 * dq2) + R2 * n2(ref.dq),
        "dk": (keys(scale ** 2 * dk2.transpose(-1, -2) @ n2(q)[..., None])[..., 0] + R2 * n2(ref.dk)
               + n2(2.0 ** -17 * keys(scale * ds.abs().transpose(-1, -2) @ q.abs()))),
        "dv": (keys((p.square() * (R2 + rel.square())).transpose(-1, -2) @ n2(d)[..., None])[..., 0]
               + R2 * n2(ref.dv) + n2(2.0 ** -17 * keys(p.transpose(-1, -2) @ d.abs()))),
    }


def worst_rows(got, ref, dout):
    """got: results by the names o (which the others came from), dq, dk, dv.  The largest row error of each in units of
    the expected one."""
    squares = expected(ref, dout, got["o"])
    want = {"o": ref.out(), "dq": ref.dq, "dk": ref.dk, "dv": ref.dv}
    far = {}
    for name, t in got.items():
        x = (t.double() - want[name]).square().sum(-1).sqrt() / (squares[name].sqrt() + 1e-30)
        far[name] = float(torch.nan_to_num(x, nan=float("inf")).max())
    return far
