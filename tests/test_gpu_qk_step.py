"""A training step of attention's inputs as a user runs it: norm and rotation of Q and K where the fused projection left them,
attention, and the gradients back to the projection's output and the norm's weights, against autograd in 64 bits."""
import math

import pytest
import torch

import sage_attention_forward_gb300 as sa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hk,R,interleaved,causal", [(3, 3, 128, True, False), (4, 2, 64, False, True), (2, 1, 90, False, True)])
def test_training_step(Hq, Hk, R, interleaved, causal, cuda_dev):
    B, S, eps = 2, 150, 1e-5
    freq, m = sa.rope_frequencies(R, scaling={"kind": "yarn", "factor": 2, "length": 64}, device=cuda_dev)
    g = torch.Generator().manual_seed(Hq + R)
    qkv = torch.randn((B, S, Hq + 2 * Hk, 128), generator=g).to(torch.bfloat16)
    qw, kw = (1 + 0.2 * torch.randn(128, generator=g) for _ in range(2))
    do = (torch.randn((B, S, Hq, 128), generator=g) * 0.1).to(torch.bfloat16)
    pos = torch.arange(S, dtype=torch.int32)

    d = qkv.to(cuda_dev)
    q, k, v = d[:, :, :Hq], d[:, :, Hq:Hq + Hk], d[:, :, Hq + Hk:]
    how = {"eps": eps, "interleaved": interleaved, "magnitude": m}
    w = (qw.to(cuda_dev), kw.to(cuda_dev))
    qr, kr = sa.qk_norm_rope_fwd(q, k, *w, freq, pos.to(cuda_dev), **how)
    o, lse = sa.attn_fwd_bf16_lse(qr, kr, v, causal=causal)
    dqr, dkr, dv = sa.attn_bwd_bf16(do.to(cuda_dev), qr, kr, v, o, lse, causal=causal)
    dqkv = torch.empty_like(d)
    dq, dk, dqw, dkw = sa.qk_norm_rope_bwd(dqr, dkr, q, k, *w, freq, pos.to(cuda_dev), dq=dqkv[:, :, :Hq],
                                           dk=dqkv[:, :, Hq:Hq + Hk], **how)
    dqkv[:, :, Hq + Hk:] = dv

    x = qkv.double().requires_grad_()
    ws = [t.double().requires_grad_() for t in (qw, kw)]
    turns = torch.tensor([f / 2.0 ** 64 for f in freq.tolist()], dtype=torch.float64)
    angle = 2 * math.pi * pos.double()[:, None, None] * turns
    c, s = angle.cos() * m, angle.sin() * m

    def turned(t, w):
        t = t / (t.square().mean(-1, keepdim=True) + eps).sqrt() * w
        a, b = (t[..., :R:2], t[..., 1:R:2]) if interleaved else (t[..., :R // 2], t[..., R // 2:R])
        y = (a * c - b * s, b * c + a * s)
        head = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
        return torch.cat([head, t[..., R:]], -1)

    q64, k64, v64 = turned(x[:, :, :Hq], ws[0]), turned(x[:, :, Hq:Hq + Hk], ws[1]), x[:, :, Hq + Hk:]
    k64, v64 = (t.repeat_interleave(Hq // Hk, 2) for t in (k64, v64))
    z = torch.einsum("bihd,bjhd->bhij", q64, k64) / math.sqrt(128)
    if causal:
        z = z.masked_fill(torch.ones((S, S), dtype=torch.bool).triu(1), -math.inf)
    out = torch.einsum("bhij,bjhd->bihd", z.softmax(-1), v64)
    want = torch.autograd.grad((out * do.double()).sum(), (x, *ws))
    # Roundings of up to 2^-8 of a value: Q' and K', P, dS, O, dQ', dK', the result, eight in a row at most and independent of
    # one another: within 8 x 2^-8 of the norm in the worst case
    for name, got, ref in (("o", o, out.detach()), ("dqkv", dqkv, want[0]), ("dqw", dqw, want[1]), ("dkw", dkw, want[2])):
        rel = float((got.double().cpu() - ref).norm() / ref.norm())
        assert rel < 8 * 2.0 ** -8, (name, rel)
