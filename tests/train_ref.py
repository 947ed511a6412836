"""Attention forward with row statistics and its backward in 64 bits, with elementwise error
bounds for the kernels (test helper, not a test file).

Bounds, from the kernels' arithmetic (u = 2^-8, half a BF16 step; everything else is FP32):
  scores    a sum of 128 FP32 products in any order, each addition off by at most 2^-23 of the
            partial sums: e_s <= 2^-16 scale sum_d |q_d k_d|, and the scaling and the base-2
            exponential add 2^-20 of the probability and 2^-22 |s|.
  lse       e_lse <= max_j e_s + 2^-21 (1 + |lse|) + (66 + Sk / 128) 2^-24 (the sum of the
            probabilities: 64 additions in a tile's accumulator, one per tile).
  O         each p rounded to BF16 (u), p itself off by e_p = e_s + 2^-20, one rounding of O:
            (u + 2 max e_p) A|V| + u |O|,  A|V| = sum_j p_j |v_j|.
  p (bwd)   relative e_s + e_lse + 2^-20.
  dV        sum_i p |dO| (u + e_p) + u |dV|.
  delta     sum_d |dO_d| times O's own bound, and 2^-16 sum_d |dO_d O_d|.  (Formed from the sum of a row's rounded
            dS instead, it is off by u sum_j |ds| <= u sum_j p (|dp| + |delta|), which is no more: sum_j p |dp| <=
            |dO| A|V|, and |delta| <= |dO| |O|.)
  dp        2^-16 sum_d |dO_d v_d|.
  ds        p (e_delta + e_dp) + |ds| (u + e_p).
  dQ, dK    scale times the sums of ds's bound times |K|, |Q|, and u of the result.  In dQ a row that sees more
            than 128 keys has the sum of its ds's errors, whose bound is the sum of theirs, taken off
            again in the first 128, in proportion to p: that bound times the mean of |K| there.
The FP32 sums over rows or keys add at most 2^-23 per addition of the sum of magnitudes, which
2^-12 of it covers up to 2000 terms; that is added to u everywhere as `acc`.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -8
ACC = 2.0 ** -12


def limits(B, Sq, Sk, causal, kv_len):
    """[B, Sq] keys that each query sees (negative values clamped to 0)."""
    n = torch.full((B,), Sk, dtype=torch.int64) if kv_len is None else kv_len.long().cpu().clamp(0, Sk)
    out = n[:, None].expand(B, Sq).clone()
    if causal:
        out = torch.minimum(out, torch.arange(Sq)[None] + 1 + Sk - Sq).clamp_min(0)
    return out


class Reference:
    """One head layout: q, dout [B, Sq, Hq, D], k, v [B, Sk, Hkv, D], any dtype and device."""

    def __init__(self, q, k, v, scale=None, causal=False, kv_len=None):
        B, Sq, Hq, D = q.shape
        Sk, Hkv = k.shape[1], k.shape[2]
        self.scale = 1.0 / math.sqrt(D) if scale is None else scale
        self.group, self.Hkv = Hq // Hkv, Hkv
        lim = limits(B, Sq, Sk, causal, kv_len).to(q.device)
        self.seen = (torch.arange(Sk, device=q.device)[None, None] < lim[..., None])[:, None]   # [B, 1, Sq, Sk]
        self.lim = lim
        real = self.seen.any(dim=2)[:, 0]                                                   # [B, Sk]
        # keys that nobody sees may hold anything: they are zeros here
        keep = real[:, :, None, None]
        self.q = q.double().permute(0, 2, 1, 3)
        self.k = self.heads(torch.where(keep, k, torch.zeros_like(k)))
        self.v = self.heads(torch.where(keep, v, torch.zeros_like(v)))
        s = self.scale * self.q @ self.k.transpose(-1, -2)
        s = torch.where(self.seen, s, torch.full_like(s, -math.inf))
        top = s.amax(-1, keepdim=True)
        top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
        e = torch.exp(s - top)
        total = e.sum(-1, keepdim=True)
        self.lse = (top + total.log())[..., 0]                                             # [B, Hq, Sq]
        self.p = e / torch.where(total == 0, torch.ones_like(total), total)
        self.o = self.p @ self.v                                                           # [B, Hq, Sq, D]
        # error bounds
        e_s = 2.0 ** -16 * self.scale * self.q.abs() @ self.k.abs().transpose(-1, -2)
        e_s = e_s + 2.0 ** -22 * torch.where(self.seen, s, torch.zeros_like(s)).abs()
        lse = torch.where(torch.isinf(self.lse), torch.zeros_like(self.lse), self.lse)
        self.lse_tol = (torch.where(self.seen, e_s, torch.zeros_like(e_s)).amax(-1) + 2.0 ** -21 * (1 + lse.abs())
                        + (66 + Sk / 128) * 2.0 ** -24)
        self.e_p = e_s + self.lse_tol[..., None] + 2.0 ** -20
        worst = torch.where(self.seen, self.e_p, torch.zeros_like(self.e_p)).amax(-1, keepdim=True)
        self.o_tol = (U + 2 * worst + ACC) * (self.p @ self.v.abs()) + U * self.o.abs() + 1e-37

    def heads(self, t):
        """[B, S, Hkv, D] -> [B, Hq, S, D] in 64 bits."""
        return t.double().permute(0, 2, 1, 3).repeat_interleave(self.group, dim=1)

    def shared(self, t):
        """[B, Hq, S, D] summed over the query heads of a key head -> [B, S, Hkv, D]."""
        B, Hq, S, D = t.shape
        return t.reshape(B, self.Hkv, self.group, S, D).sum(2).permute(0, 2, 1, 3)

    def out(self):
        return self.o.permute(0, 2, 1, 3)

    def backward(self, dout):
        d = dout.double().permute(0, 2, 1, 3)
        dp = d @ self.v.transpose(-1, -2)
        delta = (self.p * dp).sum(-1, keepdim=True)
        ds = self.p * (dp - delta)
        self.dq = (self.scale * ds @ self.k).permute(0, 2, 1, 3)
        self.dk = self.shared(self.scale * ds.transpose(-1, -2) @ self.q)
        self.dv = self.shared(self.p.transpose(-1, -2) @ d)
        e_delta = (d.abs() * self.o_tol).sum(-1, keepdim=True) + 2.0 ** -16 * (d * self.o).abs().sum(-1, keepdim=True)
        e_dp = 2.0 ** -16 * d.abs() @ self.v.abs().transpose(-1, -2)
        rel = U + self.e_p + ACC
        e_ds = self.p * (e_delta + e_dp) * (1 + self.e_p) + ds.abs() * rel
        lone = (self.lim == 1)[:, None, :, None]   # ds is exactly 0 there
        e_ds = torch.where(lone, torch.zeros_like(e_ds), e_ds)
        self.dq_tol = (self.scale * e_ds @ self.k.abs()).permute(0, 2, 1, 3) + U * self.dq.abs() + 1e-37
        if self.p.shape[-1] > 128:
            p0 = self.p[..., :128]
            mean = (p0 @ self.k[..., :128, :].abs()) / p0.sum(-1, keepdim=True).clamp_min(1e-6)
            spread = self.scale * e_ds.sum(-1, keepdim=True) * mean
            self.dq_tol += torch.where(self.lim[:, None, :, None] > 128, spread, 0 * spread).permute(0, 2, 1, 3)
        self.dk_tol = self.shared(self.scale * e_ds.transpose(-1, -2) @ self.q.abs()) + U * self.dk.abs() + 1e-37
        self.dv_tol = self.shared((self.p * rel).transpose(-1, -2) @ d.abs()) + U * self.dv.abs() + 1e-37
        return self.dq, self.dk, self.dv


def worst(got, want, tol):
    """Largest error in units of its bound; inf where got is not finite."""
    d = (got.double() - want).abs() / tol
    return float(torch.nan_to_num(d, nan=math.inf).max())
