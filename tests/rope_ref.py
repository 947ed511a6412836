"""The rotation of Q and K, and their norm with it, in 64 bits, with a bound on each output's error.

Angles come from the table's integers by integer arithmetic, so that they are exact for any position.  Bounds are counted
in u = 2^-24 (half a step of binary32) and in half a step of the output's type:

  cosine, sine   the fraction of a turn off by 2^-31 turns, then rounded to binary32 (half turns below 1: 2^-25, so
                 pi 2^-25 of angle), sincospi within 2 units in the last place, the product with the magnitude: 8 u
  a pair         (|a| + |b|) (8 u + 2 u) m for two products and a sum
  r              a sum of squares over 16 channels a lane and 5 steps between lanes (21 u), its square root halves that,
                 rsqrt 2 units in the last place (4 u), eps and the mean (1 u): 16 u
"""
import math

import torch

U = 2.0 ** -24


def cos_sin(freq, pos, B, S, magnitude):
    """freq: int64 [R / 2]; pos: integers [B or 1, S, axes] or None.  -> float64 [B, S, 1, R / 2] twice."""
    out = torch.empty((B, S, 1, len(freq)), dtype=torch.float64)
    table = [(int(f) % 2 ** 64) for f in freq.tolist()]
    for b in range(B):
        for s in range(S):
            for i, f in enumerate(table):
                if pos is None:
                    at = s
                else:
                    row = pos[b % pos.shape[0], s]
                    at = int(row[min(f & 3, len(row) - 1)])
                turn = at * (f & ~3) % 2 ** 64
                out[b, s, 0, i] = (turn - 2 ** 64 if turn >= 2 ** 63 else turn) / 2.0 ** 64
    return torch.cos(2 * math.pi * out) * magnitude, torch.sin(2 * math.pi * out) * magnitude


def parts(R, interleaved):
    return (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))


def rotate(x, cos, sin, interleaved):
    R = 2 * cos.shape[-1]
    a, b = parts(R, interleaved)
    y = x.clone()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def spread(x, R, interleaved, magnitude):
    """|a| + |b| times the magnitude in both places of each pair; |x| where a channel passes."""
    a, b = parts(R, interleaved)
    y = x.abs()
    both = (y[..., a] + y[..., b]) * abs(magnitude)
    y[..., a], y[..., b] = both, both
    return y


def half_step(y, dtype):
    return y.abs() * torch.finfo(dtype).eps / 2 + torch.finfo(dtype).smallest_normal


def rope(x, cos, sin, interleaved, magnitude):
    """y and its bound; sin negated for the backward."""
    y = rotate(x, cos, sin, interleaved)
    return y, 10 * U * spread(x, 2 * cos.shape[-1], interleaved, magnitude)


def norm_rope(x, w, eps, cos, sin, interleaved, magnitude):
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    z = x * r * w
    y = rotate(z, cos, sin, interleaved)
    return y, (16 + 2 + 10) * U * spread(z, 2 * cos.shape[-1], interleaved, magnitude)


def norm_rope_bwd(dy, x, w, eps, cos, sin, interleaved, magnitude):
    """dx, dw and their bounds."""
    R, N = 2 * cos.shape[-1], x.shape[-1]
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    xhat = x * r
    g = rotate(dy, cos, -sin, interleaved)
    gs = spread(dy, R, interleaved, magnitude)     # 10 u of it for g
    gw = g * w
    dot = (gw * xhat).sum(-1, keepdim=True) / N
    dx = r * (gw - xhat * dot)
    size = (gs * w.abs() * xhat.abs()).sum(-1, keepdim=True) / N
    # g w: 10 u + 1; the dot's terms 10 + 1 + 17 + 1, its sum 21 + 1 u; xhat 17, dx's own steps 16 + 3
    err = r * U * ((11 + 19) * gs * w.abs() + xhat.abs() * ((29 + 22) + 17 + 19 + 1) * size)
    rows = x[..., 0].numel()
    dw = (g * xhat).sum((0, 1, 2))
    # terms 10 + 17 + 1 u, and one rounding for each of up to `rows` sums (fewer: the rows are divided)
    return dx, err, dw, (28 + min(rows, 4096) + 32) * U * (gs * xhat.abs()).sum((0, 1, 2))


def near(got, want, bound, name):
    """Each output within its bound and half a step of its type."""
    off = (got.double().cpu() - want).abs() - bound - half_step(want + bound.sign() * bound, got.dtype)
    worst = float(off.max()) if off.numel() else -1.0
    assert not torch.isnan(got).any(), f"{name}: NaN"
    assert worst <= 0, f"{name}: {worst} past its bound at {int(off.argmax())} of {tuple(off.shape)}"
