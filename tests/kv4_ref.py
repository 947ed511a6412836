"""The K/V cache in 4 bits and attention over it, on the CPU: codes and scales by exact arithmetic, records byte by byte as
the header lays them out, attention in 64 bits with a bound on each output's error."""
import math

import numpy as np
import torch

RECORD = 2304


def quantise(x):
    """BF16 [..., 128] -> integer codes in [-8, 7] [..., 128] and scales float64 [..., 4] (all exact in 64 bits: the quotient
    of two 8-bit significands is at least 2^-10 from half an integer where it is none, and ties are exact)."""
    g = x.double().reshape(*x.shape[:-1], 4, 32)
    top, low = g.amax(-1), g.amin(-1)
    ext = torch.where(top >= -low, top, low)
    ext = torch.where(ext.abs() < 2.0 ** -100, 0.0, ext)
    scale = torch.where(ext == 0, 0.0, -ext / 8)      # (+0)
    safe = torch.where(scale == 0, 1.0, scale)
    code = torch.round(g / safe[..., None]).clamp(-8, 7)
    code = torch.where(scale[..., None] == 0, 0.0, code)
    return code.flatten(-2).to(torch.int64), scale


def values(x):
    code, scale = quantise(x)
    return code.double() * scale.repeat_interleave(32, -1)


def put(record, j, which, code, scale):
    """Token j's codes [128] and scales [4] of K (0) or V (1) into a record (uint8 [2304])."""
    word = record[:2048].view(np.uint32)
    half = record[:2048].view(np.uint16)
    c = (np.asarray(code, dtype=np.int64) + 8).astype(np.uint32)
    if which == 0:
        for t in range(4):
            for g in range(4):
                word[16 * j + 4 * t + g] = sum(int(c[32 * g + 8 * t + i]) << (4 * i) for i in range(8))
    else:
        for r in range(8):
            at = (1024 + 512 * (j // 8) + 16 * (4 * r + j % 8 // 2) + 8 * (j % 2)) // 2
            for g in range(4):
                half[at + g] = sum(int(c[32 * g + 4 * r + i]) << (4 * i) for i in range(4))
    bits = torch.as_tensor(scale).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    record[2048:].view(np.uint16)[8 * j + 4 * which:8 * j + 4 * which + 4] = bits


def write(cache, table, start, count, k, v):
    """kv4_write on a numpy cache [pages, heads, tiles, 2304]."""
    pages, heads, tiles, _ = cache.shape
    size = 16 * tiles
    for b in range(k.shape[0]):
        for i in range(min(max(count[b], 0), k.shape[1])):
            at = start[b] + i
            if at < 0 or at >= table.shape[1] * size:
                continue
            page = int(table[b, at // size])
            if not 0 <= page < pages:
                continue
            for h in range(heads):
                for which, x in ((0, k), (1, v)):
                    code, scale = quantise(x[b, i, h])
                    put(cache[page, h, at % size // 16], at % 16, which, code.numpy(), scale)


def steps(x):
    return quantise(x)[1].repeat_interleave(32, -1)


def held(k, v):
    """What attention takes of K and V: the values that the codes stand for, and the scales by channel."""
    return values(k), values(v), steps(k), steps(v)


def attention(q, k, v, step, v_step, seen, scale):
    """One request: q [Sq, Hq, 128]; k, v, step and v_step as held() gives them, [n, Hkv, 128]; seen [Sq, n].  -> O, lse,
    their bounds.

      scores   products with 256 + code for half of the channels and 16 + code for the others (at most 271; what the constants
               and the codes' bias of 8 add is taken off again) over 128 channels in FP32, sums of 16 channels rounded or
               cut within 2^-22 of their parts, a few of them: 2^-21 280 sum |q step|; Q's FP16, of a row whose largest
               magnitude is at least 1, off by at most 2^-25: 2^-24 max|q| sum |k|
      P        scale and rounding to FP16: half a step, 2^-11 of the value, + 2^-22; below 2^-14 (the largest scale being at
               least 2^6 there, for a probability of 1) up to 2^-25 a key, of a code of at most 8: n 2^-28 max(step_v);
               its exponential 2^-21; sums 2^-18
    """
    G = q.shape[1] // k.shape[1]
    v_step = float(v_step.abs().max()) if v_step.numel() else 0.0
    q = q.double()
    k, v, step = (t.repeat_interleave(G, 1) for t in (k, v, step))
    s = torch.einsum("shd,nhd->hsn", q, k) * scale
    hidden = ~seen[None].expand_as(s)
    s = s.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse)[..., None])
    o = torch.einsum("hsn,nhd->shd", p, v)
    off = scale * (280 * 2.0 ** -21 * torch.einsum("shd,nhd->hsn", q.abs(), step.abs())
                   + 2.0 ** -24 * q.abs().amax(-1).T[..., None] * k.abs().sum(-1).T[:, None])
    off = off + s.abs().nan_to_num(posinf=0.0) * 2.0 ** -21
    off = off.masked_fill(hidden, 0.0).amax(-1) if s.shape[-1] else torch.zeros_like(lse)
    size = torch.einsum("hsn,nhd->shd", p, v.abs())
    bound = size * (2.0 ** -11 + 2.0 ** -18 + 2 * off.T[..., None])
    bound = bound + v.shape[0] * 2.0 ** -28 * v_step
    return o, lse, bound, off + 2.0 ** -17 + lse.abs().nan_to_num(posinf=0.0) * 2.0 ** -22


def check(got, got_lse, want, lse, bound, lse_bound):
    half = (want.abs() + bound) * 2.0 ** -8 + 2.0 ** -130
    worst = float(((got.double().cpu() - want).abs() - bound - half).max())
    assert worst <= 0, f"O is {worst} past its bound"
    got_lse = got_lse.double().cpu()
    empty = torch.isinf(lse)
    assert torch.equal(torch.isinf(got_lse), empty) and (got_lse[empty] < 0).all()
    assert ((got_lse - lse).abs()[~empty] <= lse_bound[~empty]).all(), "lse"
