"""layer_norm_fwd and layer_norm_bwd against their formulas in 64 bits.

Bounds, from the kernels' arithmetic (FP32, u = half a step of the result's type, e = 2^-24):
  mean   a sum of N in any order: N e sum|x| / N, and a rounding of 1 / N
  var    sums of squares of x - mean (each off by e |x - mean| and the mean's error): relative
         (N + 8) e, plus the square of the mean's error; rstd is off by half of that, relatively
  y      |w| (e_xhat) + u |y|,  e_xhat = |xhat| (e_rstd + 4 e) + rstd (e_mean + e |x|)
  dx     rstd times the bound of the bracket: the two means of N terms at N e of their magnitudes,
         xhat's bound with |g| and |xhat|, 8 e of the terms; and u |dx|.  mean and rstd are inputs, so
         that the reference takes them as given
  dw     sum over the rows of |dy| e_xhat + (rows + 8) e |dy xhat|, and u of the result; db the like
(In practice sums are trees, far inside the N e of a chain.)"""
import pytest
import torch

import sage_attention_forward_gb300 as sa

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25, torch.float32: 1e-38}   # half the smallest step


def worst(got, want, tol):
    d = (got.double() - want).abs() / tol
    return float(torch.nan_to_num(d, nan=float("inf")).max()) if d.numel() else 0.0


def make(dev, shape, dtype, wtype, seed, offset=0.5):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = (torch.randn(shape, generator=g, device=dev) * (torch.rand(shape[-1], generator=g, device=dev) + 0.5) + offset)
    dy = torch.randn(shape, generator=g, device=dev) * 0.3
    w = 1 + 0.3 * torch.randn(shape[-1], generator=g, device=dev)
    b = 0.3 * torch.randn(shape[-1], generator=g, device=dev)
    return x.to(dtype), dy.to(dtype), w.to(wtype), b.to(wtype)


def check_fwd(x, w, b, eps, got):
    y, mean, rstd = got
    N = x.shape[-1]
    X = x.double()
    m = X.mean(-1)
    c = X - m[..., None]
    var = c.square().mean(-1)
    r = 1 / torch.sqrt(var + eps)
    e_m = (N + 2) * E * X.abs().mean(-1) + 1e-300
    assert worst(mean, m, e_m) <= 1
    # (var is not below eps's part: relative to var + eps)
    e_var = ((N + 8) * E * var + 2 * e_m * c.abs().mean(-1) + (e_m + E * X.abs().amax(-1)) ** 2) / (var + eps)
    e_r = 0.5 * e_var * (1 + e_var) + 4 * E
    assert worst(rstd, r, r * e_r) <= 1
    xh = c * r[..., None]
    e_xh = xh.abs() * (e_r + 4 * E)[..., None] + (r * (1 + e_r))[..., None] * (e_m[..., None] + E * X.abs())
    W = 1.0 if w is None else w.double()
    B = 0.0 if b is None else b.double()
    want = xh * W + B
    aw = 1.0 if w is None else w.double().abs()
    ab = 0.0 if b is None else b.double().abs()
    tol = aw * (e_xh + 2 * E * xh.abs()) + 2 * E * ab + U[y.dtype] * want.abs() * (1 + 2.0 ** -8) + TINY[y.dtype]
    assert worst(y, want, tol) <= 1


def check_bwd(dy, x, w, mean, rstd, got):
    dx, dw, db = got
    N, rows = x.shape[-1], x[..., 0].numel()
    X, D, m, r = x.double(), dy.double(), mean.double()[..., None], rstd.double()[..., None]
    xh = (X - m) * r
    e_xh = 2 * E * (xh.abs() + r * (X - m).abs())
    W = torch.ones(N, dtype=torch.float64, device=x.device) if w is None else w.double()
    g = D * W
    a, c = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    want = r * (g - a - xh * c)
    e_a = (N + 3) * E * g.abs().mean(-1, keepdim=True)
    e_c = (N + 5) * E * (g * xh).abs().mean(-1, keepdim=True) + (g.abs() * e_xh).mean(-1, keepdim=True)
    terms = g.abs() + a.abs() + (xh * c).abs()
    tol = r * (e_a + xh.abs() * e_c + e_xh * c.abs() + 8 * E * terms) + U[x.dtype] * want.abs() * (1 + 2.0 ** -8) + TINY[x.dtype]
    assert worst(dx, want, tol) <= 1
    if dw is None:
        return
    lead = tuple(range(x.dim() - 1))
    for t, term, extra in ((dw, D * xh, D.abs() * e_xh), (db, D, 0 * D)):
        s = term.sum(lead) if lead else term
        mag = term.abs().sum(lead) if lead else term.abs()
        ex = extra.sum(lead) if lead else extra
        assert worst(t, s, (rows + 8) * E * mag + ex + U[t.dtype] * s.abs() * (1 + 2.0 ** -8) + TINY[t.dtype]) <= 1


TYPES = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float16, torch.float16),
         (torch.float16, torch.float32), (torch.float32, torch.float32)]


@pytest.mark.parametrize("dtype,wtype", TYPES)
@pytest.mark.parametrize("rows,N", [(1, 1), (3, 2), (5, 7), (130, 8), (33, 64), (1000, 65), (77, 128), (5000, 128),
                                    (300, 129), (257, 256), (50, 500), (64, 512), (31, 513), (400, 1000), (9, 2048),
                                    (700, 4099), (6, 5120), (3, 8192), (2, 8193), (5, 12288), (400, 16384), (3, 16383)])
def test_sizes(cuda_dev, rows, N, dtype, wtype):
    x, dy, w, b = make(cuda_dev, (rows, N), dtype, wtype, rows + N)
    got = sa.layer_norm_fwd(x, w, b, eps=1e-5)
    check_fwd(x, w, b, 1e-5, got)
    back = sa.layer_norm_bwd(dy, x, w, got[1], got[2])
    check_bwd(dy, x, w, got[1], got[2], back)
    again = sa.layer_norm_bwd(dy, x, w, got[1], got[2])
    assert all(torch.equal(p, q) for p, q in zip(back, again))


@pytest.mark.parametrize("N", [128, 96, 33])
def test_strided_heads(cuda_dev, N):
    """Q's heads as a slice of a fused projection, results into slices of wider buffers."""
    B, S, H = 2, 150, 3
    qkv, dq, w, b = make(cuda_dev, (B, S, 3, H, N), torch.bfloat16, torch.float32, 1)
    x, dy = qkv[:, :, 1], dq[:, :, 0]
    y, mean, rstd = sa.layer_norm_fwd(x, w, b)
    check_fwd(x, w, b, 1e-6, (y, mean, rstd))
    wide = torch.full((B, H, S, N + 8), 7.0, dtype=torch.bfloat16, device=cuda_dev).permute(0, 2, 1, 3)
    y2, _, _ = sa.layer_norm_fwd(x, w, b, out=wide[..., :N])
    assert torch.equal(y2, y) and bool((wide[..., N:] == 7).all())
    dx, dw, db = sa.layer_norm_bwd(dy, x, w, mean, rstd)
    check_bwd(dy, x, w, mean, rstd, (dx, dw, db))
    sa.layer_norm_bwd(dy, x, w, mean, rstd, dx=wide[..., :N])
    assert torch.equal(wide[..., :N], dx) and bool((wide[..., N:] == 7).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [128, 1024])
def test_alignment_and_broadcast(cuda_dev, N, dtype):
    """Pointers off the 16-byte grid, odd row strides, a row read again and again (stride 0)."""
    base, dbase, w, b = make(cuda_dev, (40, N + 3), dtype, dtype, 2)
    x, dy, w, b = base[:, 1:N + 1], dbase[:, 3:], w[1:N + 1].clone(), b[1:N + 1].clone()
    y, mean, rstd = sa.layer_norm_fwd(x, w, b)
    check_fwd(x, w, b, 1e-6, (y, mean, rstd))
    check_bwd(dy, x, w, mean, rstd, sa.layer_norm_bwd(dy, x, w, mean, rstd))
    one = dy[:1].expand(40, N)
    check_bwd(one, x, w, mean, rstd, sa.layer_norm_bwd(one, x, w, mean, rstd))
    rep = x[:1].expand(40, N)
    y2, m2, r2 = sa.layer_norm_fwd(rep, w, b)
    assert torch.equal(y2, y[:1].expand(40, N)) and torch.equal(m2, mean[:1].expand(40))


def test_without_weight_and_bias(cuda_dev):
    x, dy, w, b = make(cuda_dev, (50, 200), torch.bfloat16, torch.bfloat16, 3)
    got = sa.layer_norm_fwd(x)
    check_fwd(x, None, None, 1e-6, got)
    back = sa.layer_norm_bwd(dy, x, None, got[1], got[2])
    assert back[1] is None and back[2] is None
    check_bwd(dy, x, None, got[1], got[2], back)
    check_fwd(x, w, None, 1e-6, sa.layer_norm_fwd(x, w))
    check_fwd(x, None, b, 1e-6, sa.layer_norm_fwd(x, None, b))
    dw, db = torch.empty(200, device=cuda_dev), torch.empty(200, device=cuda_dev)
    check_bwd(dy, x, None, got[1], got[2], sa.layer_norm_bwd(dy, x, None, got[1], got[2], dweight=dw, dbias=db))


def test_large_mean(cuda_dev):
    """Rows whose mean is a thousand times their spread keep their variance."""
    x, dy, w, b = make(cuda_dev, (64, 640), torch.float32, torch.float32, 4, offset=1000.0)
    check_fwd(x, w, b, 1e-6, sa.layer_norm_fwd(x, w, b))


def test_in_place(cuda_dev):
    x, dy, w, b = make(cuda_dev, (300, 384), torch.bfloat16, torch.bfloat16, 5)
    y, mean, rstd = sa.layer_norm_fwd(x, w, b)
    dx, dw, db = sa.layer_norm_bwd(dy, x, w, mean, rstd)
    d2 = dy.clone()
    got = sa.layer_norm_bwd(d2, x, w, mean, rstd, dx=d2)
    assert all(torch.equal(p, q) for p, q in zip(got, (dx, dw, db)))
    x2 = x.clone()
    assert torch.equal(sa.layer_norm_fwd(x2, w, b, out=x2)[0], y)


def test_many_rows(cuda_dev):
    x, dy, w, b = make(cuda_dev, (200001, 24), torch.bfloat16, torch.float32, 6)
    got = sa.layer_norm_fwd(x, w, b)
    check_fwd(x, w, b, 1e-6, got)
    check_bwd(dy, x, w, got[1], got[2], sa.layer_norm_bwd(dy, x, w, got[1], got[2]))


def test_no_rows(cuda_dev):
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=cuda_dev)
    w = torch.ones(64, dtype=torch.bfloat16, device=cuda_dev)
    y, mean, rstd = sa.layer_norm_fwd(x, w, w)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dw, db = sa.layer_norm_bwd(x, x, w, mean, rstd, dweight=torch.ones_like(w), dbias=torch.ones_like(w))
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())


def test_streams_and_graph(cuda_dev):
    x, dy, w, b = make(cuda_dev, (999, 1000), torch.bfloat16, torch.bfloat16, 7)

    def step(stream=None):
        y, mean, rstd = sa.layer_norm_fwd(x, w, b, stream=stream)
        return (y,) + sa.layer_norm_bwd(dy, x, w, mean, rstd, stream=stream)

    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    other = step(s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = step()
    x.mul_(1.5)
    graph.replay()
    now = step()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(caught, now)) and not torch.equal(now[1], want[1])


def test_gradient_matches_differences(cuda_dev):
    """The kernel's gradients against central differences of the 64-bit forward."""
    x, dy, w, b = make(cuda_dev, (20, 48), torch.float32, torch.float32, 8)
    _, mean, rstd = sa.layer_norm_fwd(x, w, b, eps=1e-5)
    grads = sa.layer_norm_bwd(dy, x, w, mean, rstd)

    def f(x, w, b):
        c = x - x.mean(-1, keepdim=True)
        y = c / torch.sqrt(c.square().mean(-1, keepdim=True) + 1e-5) * w + b
        return float((y * dy.double()).sum())

    args = [t.double() for t in (x, w, b)]
    g = torch.Generator(device=cuda_dev).manual_seed(9)
    for at, grad in enumerate(grads):
        d = torch.randn(grad.shape, generator=g, device=cuda_dev, dtype=torch.float64)
        up, down = list(args), list(args)
        up[at], down[at] = args[at] + 1e-5 * d, args[at] - 1e-5 * d
        # h^2 of a third derivative of order 1e3; FP32 gradients: 48 terms' 2^-24 each over 960 values of order 1
        assert abs((f(*up) - f(*down)) / 2e-5 - float((grad.double() * d).sum())) < 1e-3


@pytest.mark.parametrize("N", [128, 130, 1000, 9000])
def test_strides_past_32_bits(cuda_dev, N):
    """Rows 2^31 and more elements apart in the inputs and outputs."""
    far = (1 << 31) + 64
    store = torch.empty(far + (1 << 18), dtype=torch.bfloat16, device=cuda_dev)
    x, dy, w, b = make(cuda_dev, (2, 3, N), torch.bfloat16, torch.float32, 77)
    pitch = (N + 15) // 16 * 16   # (whole 16-byte pieces where N allows them)
    at = [0]

    def spread(t):
        out = store.as_strided(t.shape, (far, pitch, 1), at[0])
        at[0] += 3 * pitch
        return out.copy_(t)

    sx, sdy, sy, sdx = spread(x), spread(dy), spread(torch.zeros_like(x)), spread(torch.zeros_like(x))
    assert at[0] <= 1 << 18
    _, mean, rstd = sa.layer_norm_fwd(sx, w, b, 1e-5, out=sy)
    _, dw, db = sa.layer_norm_bwd(sdy, sx, w, mean, rstd, dx=sdx)
    torch.cuda.synchronize()
    check_fwd(x, w, b, 1e-5, (sy, mean, rstd))
    check_bwd(dy, x, w, mean, rstd, (sdx, dw, db))


def test_infinities_stay_in_their_row(cuda_dev):
    """A row of NaN or infinities changes no other row's y and dx, also where rows share a warp."""
    for N in (64, 128, 2000):
        x, dy, w, b = make(cuda_dev, (67, N), torch.bfloat16, torch.bfloat16, 78)
        bad = x.clone()
        bad[5] = float("nan")
        bad[33, 1] = float("inf")
        keep = torch.ones(67, dtype=torch.bool, device=cuda_dev)
        keep[5] = keep[33] = False
        y, mean, rstd = sa.layer_norm_fwd(x, w, b)
        by, bmean, brstd = sa.layer_norm_fwd(bad, w, b)
        dx, _, _ = sa.layer_norm_bwd(dy, x, w, mean, rstd)
        bdx, _, _ = sa.layer_norm_bwd(dy, bad, w, bmean, brstd)
        for good, other in ((y, by), (mean, bmean), (rstd, brstd), (dx, bdx)):
            assert torch.equal(good[keep], other[keep])
        assert bool(by[5].isnan().all()) and bool(by[33].isnan().any())


@pytest.mark.parametrize("dtype,wtype", TYPES)
@pytest.mark.parametrize("rows,N,gap,start", [(1, 513, 0, 0), (1, 1773, 0, 3), (7, 259, 0, 1), (7, 515, 1, 0), (900, 1773, 0, 5),
                                              (1300, 1001, 3, 1), (300, 6345, 0, 0), (40, 8177, 2, 7), (20, 8191, 0, 1),
                                              (2000, 517, 8, 2), (9, 1022, 0, 1)])
def test_rows_off_16_bytes(cuda_dev, rows, N, gap, start, dtype, wtype):
    """Rows that start and end anywhere, with NaN between them and around the tensor: nothing of it comes into the
    results, and what lies between and around the outputs' rows stays as it was."""
    x, dy, w, b = make(cuda_dev, (rows, N), dtype, wtype, rows + N)
    pitch, size = N + gap, start + rows * (N + gap) + 16

    def spread(t):
        store = torch.full((size,), float("nan"), dtype=dtype, device=cuda_dev)
        view = store.as_strided((rows, N), (pitch, 1), start)
        if t is not None:
            view.copy_(t)
        return store, view

    (_, vx), (_, vdy), (sy, vy), (sdx, vdx) = spread(x), spread(dy), spread(None), spread(None)
    _, mean, rstd = sa.layer_norm_fwd(vx, w, b, 1e-5, out=vy)
    check_fwd(x, w, b, 1e-5, (vy, mean, rstd))
    _, dw, db = sa.layer_norm_bwd(vdy, vx, w, mean, rstd, dx=vdx)
    check_bwd(dy, x, w, mean, rstd, (vdx, dw, db))
    for store, view in ((sy, vy), (sdx, vdx)):
        view.fill_(float("nan"))
        assert bool(store.isnan().all())
    # in place, and the same bits again
    _, again, _ = sa.layer_norm_bwd(vdy, vx, w, mean, rstd, dx=vdy)
    assert torch.equal(dw, again)
    check_bwd(dy, x, w, mean, rstd, (vdy, dw, db))
    sa.layer_norm_fwd(vx, w, b, 1e-5, out=vx)
    check_fwd(x, w, b, 1e-5, (vx, mean, rstd))
    sa.attn_get_device_status()


@pytest.mark.parametrize("N", [8200, 12288, 14080, 14084, 16384])
@pytest.mark.parametrize("rows", [5, 700])
def test_wide_rows_of_32_bits(cuda_dev, rows, N):
    """Two rows of x and dy in shared memory, up to what it holds, and past that."""
    x, dy, w, b = make(cuda_dev, (rows, N), torch.float32, torch.float32, N)
    y, mean, rstd = sa.layer_norm_fwd(x, w, b, 1e-6)
    check_fwd(x, w, b, 1e-6, (y, mean, rstd))
    check_bwd(dy, x, w, mean, rstd, sa.layer_norm_bwd(dy, x, w, mean, rstd))
    sa.attn_get_device_status()


@pytest.mark.parametrize("dtype,wtype", TYPES)
@pytest.mark.parametrize("N", [8192, 8200, 9000, 10240, 10248])
def test_where_the_forms_change(cuda_dev, N, dtype, wtype):
    """Around the largest rows of each form of the ring."""
    x, dy, w, b = make(cuda_dev, (321, N), dtype, wtype, N)
    y, mean, rstd = sa.layer_norm_fwd(x, w, b, 1e-6)
    check_fwd(x, w, b, 1e-6, (y, mean, rstd))
    check_bwd(dy, x, w, mean, rstd, sa.layer_norm_bwd(dy, x, w, mean, rstd))
    sa.attn_get_device_status()
