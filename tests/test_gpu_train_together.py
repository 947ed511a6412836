"""The training operators as a transformer layer uses them: layer norm of Q and K where a fused projection
left them, attention forward, attention backward, layer norm backward into the projection's gradient.

The reference is the chain in 64 bits.  It starts from the normalised Q and K as the kernel rounded
them (checked on their own), since that rounding is the operator's output type.  dQ and dK then are off by at
most train_ref's bounds E; through layer norm's backward, which is linear in its gradient, dx is off by
  rstd (|w| E + mean(|w| E) + |xhat| mean(|w| E |xhat|)),  dweight by sum |xhat| E,  dbias by sum E,
to which that kernel's own bounds come (test_gpu_layer_norm.py), taken at gradients up to |dy| + E."""
import pytest
import torch

import sage_attention_forward_gb300 as sa
from test_gpu_layer_norm import E as E32, U, check_fwd, worst
from train_ref import Reference

pytestmark = pytest.mark.gpu

EPS = 1e-6


class Layer:
    """Buffers of one layer: everything that a captured graph writes stays where it is."""

    def __init__(self, dev, B, S, Hq, Hkv, seed):
        g = torch.Generator(device=dev).manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
        self.sizes = (B, S, Hq, Hkv)
        self.x = (r(B, S, Hq + 2 * Hkv, 128) + 0.3).to(torch.bfloat16)
        self.dout = (0.1 * r(B, S, Hq, 128)).to(torch.bfloat16)
        self.w = [(1 + 0.2 * r(128)), (1 + 0.2 * r(128)).to(torch.bfloat16)]
        self.b = [0.2 * r(128), (0.2 * r(128)).to(torch.bfloat16)]
        self.dx = torch.full_like(self.x, float("nan"))

    def parts(self, t):
        _, _, Hq, Hkv = self.sizes
        return t[:, :, :Hq], t[:, :, Hq:Hq + Hkv], t[:, :, Hq + Hkv:]

    def step(self, causal, kv_len):
        xq, xk, v = self.parts(self.x)
        gq, gk, gv = self.parts(self.dx)
        q, *sq = sa.layer_norm_fwd(xq, self.w[0], self.b[0], EPS)
        k, *sk = sa.layer_norm_fwd(xk, self.w[1], self.b[1], EPS)
        o, lse = sa.attn_fwd_bf16_lse(q, k, v, causal=causal, kv_len=kv_len)
        # dV goes straight to its place; dQ and dK go there through layer norm's backward, in place
        sa.attn_bwd_bf16(self.dout, q, k, v, o, lse, causal=causal, kv_len=kv_len, dq=gq, dk=gk, dv=gv)
        _, dwq, dbq = sa.layer_norm_bwd(gq, xq, self.w[0], *sq, dx=gq)
        _, dwk, dbk = sa.layer_norm_bwd(gk, xk, self.w[1], *sk, dx=gk)
        return (q, *sq), (k, *sk), o, lse, [dwq, dwk], [dbq, dbk]


def norm_backward(dy, tol, x, mean, rstd, w, got_dx, got_dw, got_db):
    """dy and its bound `tol` in 64 bits through layer norm's backward, against the kernel's results."""
    X, W, r = x.double(), w.double(), rstd.double()[..., None]
    N, rows = X.shape[-1], X[..., 0].numel()
    xh = (X - mean.double()[..., None]) * r
    avg = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    g = dy * W
    want = r * (g - avg(g) - xh * avg(g * xh))
    # the gradient comes in rounded, and off by tol
    e = tol * W.abs()
    far = r * (e + avg(e) + xh.abs() * avg(e * xh.abs()))
    big = g.abs() + e
    e_xh = 2 * E32 * (xh.abs() + r * (X - mean.double()[..., None]).abs())
    own = r * ((N + 3) * E32 * avg(big) + xh.abs() * ((N + 5) * E32 * avg(big * xh.abs()) + avg(big * e_xh))
               + e_xh * avg(big * xh.abs()) + 8 * E32 * (big + avg(big) + xh.abs() * avg(big * xh.abs())))
    u = U[got_dx.dtype]
    out = {"dx": worst(got_dx, want, (far + own) * (1 + u) + u * want.abs() + 1e-38)}
    lead = (0, 1, 2)
    for name, t, f, e_f in (("dw", got_dw, xh, e_xh), ("db", got_db, torch.ones_like(xh), 0 * xh)):
        s = (dy * f).sum(lead)
        size = ((dy.abs() + tol) * f.abs()).sum(lead)
        bound = (tol * f.abs()).sum(lead) + ((dy.abs() + tol) * e_f).sum(lead) + (rows + 8) * E32 * size
        out[name] = worst(t, s, bound * (1 + U[t.dtype]) + U[t.dtype] * s.abs() + 1e-38)
    return out


@pytest.mark.parametrize("B,S,Hq,Hkv,causal,lens", [(2, 333, 6, 2, True, [333, 130]), (1, 128, 2, 2, False, None),
                                                    (3, 40, 4, 1, True, [0, 1, 40]), (1, 700, 3, 3, False, [513])])
def test_layer_step(cuda_dev, B, S, Hq, Hkv, causal, lens):
    layer = Layer(cuda_dev, B, S, Hq, Hkv, 7 * S)
    kv_len = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=cuda_dev)
    (q, *sq), (k, *sk), o, lse, dw, db = layer.step(causal, kv_len)
    torch.cuda.synchronize()
    sa.attn_get_device_status()
    xq, xk, v = layer.parts(layer.x)
    check_fwd(xq, layer.w[0], layer.b[0], EPS, (q, *sq))
    check_fwd(xk, layer.w[1], layer.b[1], EPS, (k, *sk))
    ref = Reference(q, k, v, None, causal, kv_len)
    ref.backward(layer.dout)
    far = {"o": worst(o, ref.out(), ref.o_tol.permute(0, 2, 1, 3))}
    gq, gk, gv = layer.parts(layer.dx)
    far["v"] = worst(gv, ref.dv, ref.dv_tol)
    far["q"] = norm_backward(ref.dq, ref.dq_tol, xq, *sq, layer.w[0], gq, dw[0], db[0])
    far["k"] = norm_backward(ref.dk, ref.dk_tol, xk, *sk, layer.w[1], gk, dw[1], db[1])
    print(far)
    assert max([far["o"], far["v"], *far["q"].values(), *far["k"].values()]) <= 1, far


def test_layer_step_captured(cuda_dev):
    """The step in a graph, replayed on new inputs, gives the eager step's bits."""
    layer, other = Layer(cuda_dev, 2, 200, 4, 2, 1), Layer(cuda_dev, 2, 200, 4, 2, 2)
    kv_len = torch.tensor([200, 77], dtype=torch.int32, device=cuda_dev)
    layer.step(True, kv_len)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        _, _, o, lse, dw, db = layer.step(True, kv_len)
    for name in ("x", "dout"):
        getattr(layer, name).copy_(getattr(other, name))
    for i in range(2):
        layer.w[i].copy_(other.w[i])
        layer.b[i].copy_(other.b[i])
    layer.dx.fill_(float("nan"))
    graph.replay()
    _, _, o2, lse2, dw2, db2 = other.step(True, kv_len)
    torch.cuda.synchronize()
    sa.attn_get_device_status()
    for a, b in zip([o, lse, *dw, *db, layer.dx], [o2, lse2, *dw2, *db2, other.dx]):
        assert torch.equal(a, b)
