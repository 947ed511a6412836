"""What the training entry points refuse: on the host, before anything of the GPU is touched, through the
C ABI and through the Python binding (CPU-only tests)."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

import sage_attention_forward_gb300 as sa

I64x3 = ctypes.c_int64 * 3
FAKE = 0x10000   # an aligned non-null address; validation never dereferences it
OK, ARG, ALIGN, UNSUPPORTED = 0, 1, 2, 3
BF16, F16, F32 = 0, 1, 2


def strides(t):
    return None if t is None else I64x3(*t)


ATTN = dict(q=FAKE, k=FAKE, v=FAKE, o=2 * FAKE, lse=FAKE, B=2, Sq=256, Sk=128, Hq=4, Hkv=2, D=128,
            q_str=(256 * 512, 512, 128), k_str=(128 * 256, 256, 128), v_str=(128 * 256, 256, 128),
            o_str=(256 * 512, 512, 128), scale=0.088, causal=0, kv_len=None)


def call_fwd(**kw):
    a = SimpleNamespace(**{**ATTN, **kw})
    return sa.lib().attn_fwd_bf16_lse(a.q, a.k, a.v, a.o, a.lse, a.B, a.Sq, a.Sk, a.Hq, a.Hkv, a.D, strides(a.q_str),
                                      strides(a.k_str), strides(a.v_str), strides(a.o_str), a.scale, a.causal,
                                      a.kv_len, None)


def call_bwd(**kw):
    more = dict(dout=FAKE, dq=16 * FAKE, dk=17 * FAKE, dv=18 * FAKE, dout_str=ATTN["q_str"], dq_str=ATTN["q_str"],
                dk_str=ATTN["k_str"], dv_str=ATTN["k_str"], ws=FAKE, ws_bytes=1 << 40)
    a = SimpleNamespace(**{**ATTN, **more, **kw})
    return sa.lib().attn_bwd_bf16(a.dout, a.q, a.k, a.v, a.o, a.lse, a.dq, a.dk, a.dv, a.B, a.Sq, a.Sk, a.Hq, a.Hkv,
                                  a.D, strides(a.dout_str), strides(a.q_str), strides(a.k_str), strides(a.v_str),
                                  strides(a.o_str), strides(a.dq_str), strides(a.dk_str), strides(a.dv_str), a.scale,
                                  a.causal, a.kv_len, a.ws, a.ws_bytes, None)


ATTN_CASES = [
    (dict(D=64), UNSUPPORTED),
    (dict(B=0), OK),
    (dict(Hq=0, Hkv=0, q=None, k=None, v=None), OK),
    (dict(B=-1), ARG),
    (dict(Sq=0), ARG),
    (dict(Sk=0), ARG),
    (dict(Sk=(1 << 30) + 1), ARG),
    (dict(Hq=3), ARG),                 # not a multiple of Hkv
    (dict(Hq=0), ARG),
    (dict(Hkv=0), ARG),
    (dict(causal=2), ARG),
    (dict(scale=-1.0), ARG),
    (dict(scale=float("nan")), ARG),
    (dict(scale=float("inf")), ARG),
    (dict(kv_len=FAKE + 2), ALIGN),
    (dict(q=None), ARG),
    (dict(v=FAKE + 8), ALIGN),
    (dict(lse=None), ARG),
    (dict(lse=FAKE + 4), ALIGN),
    (dict(k_str=None), ARG),
    (dict(k_str=(128 * 256, 260, 128)), ALIGN),
    (dict(k_str=(128 * 256, 0, 128)), ARG),
    (dict(v_str=(128 * 256, -256, 128)), ARG),
    (dict(o_str=(256 * 512, 512, 4)), ALIGN),
    (dict(B=65536, Hq=16384, Hkv=16384), ARG),   # 2^31 tiles: beyond the grid
    (dict(B=300, Hq=300, Hkv=300, q=None), ARG),   # 90000 heads are accepted (then the NULL q is reported)
]


@pytest.mark.parametrize("call", [call_fwd, call_bwd])
@pytest.mark.parametrize("kw,status", ATTN_CASES)
def test_attention_arguments(call, kw, status):
    assert call(**kw) == status
    if status:
        assert sa.lib().attn_last_error().decode() != ""


@pytest.mark.parametrize("kw,status", [
    (dict(dout=None), ARG),
    (dict(dout=FAKE + 2), ALIGN),
    (dict(dq=None), ARG),
    (dict(dk=18 * FAKE + 8), ALIGN),
    (dict(dv_str=None), ARG),
    (dict(dq_str=(256 * 512, 0, 128)), ARG),
    (dict(ws=None), ARG),
    (dict(ws=FAKE + 8), ALIGN),
    (dict(ws_bytes=1), ARG),
    (dict(dq=FAKE), ARG),               # q's memory: dK is still to be formed from it
    (dict(dk=FAKE), ARG),
    (dict(dv=17 * FAKE), ARG),          # dK's memory
])
def test_attention_backward_arguments(kw, status):
    assert call_bwd(**kw) == status


@pytest.mark.parametrize("name", "qkv")
def test_attention_forward_over_its_input(name):
    assert call_fwd(**{name: 2 * FAKE}) == ARG


def test_attention_workspace_size():
    size = sa.lib().attn_bwd_bf16_workspace_size
    assert size(0, 4, 4, 2, 2) == 0 and size(1, 4, 4, 2, 0) == 0
    # two floats for each row of each query head, rows padded to whole tiles; few key tiles and heads take more
    assert size(2, 129, 5000, 128, 64) == 2 * 2 * 128 * 256 * 4
    assert size(2, 1290, 64, 6, 3) > 2 * 2 * 6 * 1408 * 4
    assert size(64, 1 << 20, 128, 64, 64) == 2 * 64 * 64 * (1 << 20) * 4   # beyond 32 bits
    assert call_bwd(ws_bytes=2 * 2 * 4 * 256 * 4 - 1) == ARG


NORM = dict(x=FAKE, w=FAKE, b=FAKE, y=2 * FAKE, mean=FAKE, rstd=FAKE, B=2, S=64, H=3, N=128,
            x_str=(64 * 384, 384, 128), y_str=(64 * 384, 384, 128), eps=1e-6, dtype=BF16, w_dtype=BF16)


def call_norm_fwd(**kw):
    a = SimpleNamespace(**{**NORM, **kw})
    return sa.lib().layer_norm_fwd(a.x, a.w, a.b, a.y, a.mean, a.rstd, a.B, a.S, a.H, a.N, strides(a.x_str),
                                   strides(a.y_str), a.eps, a.dtype, a.w_dtype, None)


def call_norm_bwd(**kw):
    more = dict(dy=FAKE, dx=2 * FAKE, dw=FAKE, db=FAKE, dy_str=NORM["x_str"], dx_str=NORM["x_str"], ws=FAKE,
                ws_bytes=1 << 40)
    a = SimpleNamespace(**{**NORM, **more, **kw})
    return sa.lib().layer_norm_bwd(a.dy, a.x, a.w, a.mean, a.rstd, a.dx, a.dw, a.db, a.B, a.S, a.H, a.N,
                                   strides(a.dy_str), strides(a.x_str), strides(a.dx_str), a.dtype, a.w_dtype, a.ws,
                                   a.ws_bytes, None)


@pytest.mark.parametrize("call", [call_norm_fwd, call_norm_bwd])
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), ARG),
    (dict(dtype=-1), ARG),
    (dict(dtype=BF16, w_dtype=F16), ARG),
    (dict(dtype=F32, w_dtype=BF16), ARG),
    (dict(B=-1), ARG),
    (dict(N=0), ARG),
    (dict(N=16385), ARG),
    (dict(B=1 << 15, S=1 << 15, H=2), ARG),      # 2^31 rows
    (dict(B=1 << 30, S=1 << 30, H=1 << 30), ARG),
    (dict(x=None), ARG),
    (dict(x=FAKE + 1), ALIGN),
    (dict(x=FAKE + 2, dtype=F32, w_dtype=F32), ALIGN),
    (dict(x_str=None), ARG),
    (dict(x_str=(64 * 384, -384, 128)), ARG),
    (dict(x_str=(1 << 38, 384, 128)), ARG),
    (dict(w=FAKE + 1), ALIGN),
    (dict(w=FAKE + 2, w_dtype=F32), ALIGN),
    (dict(mean=None), ARG),
    (dict(rstd=FAKE + 2), ALIGN),
])
def test_layer_norm_arguments(call, kw, status):
    assert call(**kw) == status
    assert sa.lib().attn_last_error().decode() != ""


@pytest.mark.parametrize("kw,status", [
    (dict(eps=-1e-6), ARG),
    (dict(eps=float("nan")), ARG),
    (dict(eps=float("inf")), ARG),
    (dict(y=None), ARG),
    (dict(b=FAKE + 1), ALIGN),
    (dict(y_str=(64 * 384, 0, 128)), ARG),       # rows on one another
    (dict(B=0), OK),
    (dict(H=0, x=None, y=None), OK),
])
def test_layer_norm_forward_arguments(kw, status):
    assert call_norm_fwd(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), ARG),
    (dict(dx=None), ARG),
    (dict(dx_str=(64 * 384, 384, 0)), ARG),
    (dict(dw=None), ARG),                        # one without the other
    (dict(db=None), ARG),
    (dict(dw=FAKE + 1), ALIGN),
    (dict(ws=None), ARG),
    (dict(ws=FAKE + 4), ALIGN),
    (dict(ws_bytes=1), ARG),
    (dict(S=0, dw=None, db=None), OK),
])
def test_layer_norm_backward_arguments(kw, status):
    assert call_norm_bwd(**kw) == status


def test_layer_norm_workspace_size():
    size = sa.lib().layer_norm_bwd_workspace_size
    assert size(0, 4, 4, 128) == 0 and size(1, 1, 1, 16385) == 0 and size(1 << 30, 1 << 30, 1 << 30, 8) == 0
    for N in (1, 7, 128, 5120, 16384):
        for rows in (1, 33, 5000, 1 << 30):
            assert size(1, rows, 1, N) == size(rows, 1, 1, N) > 0
            assert size(1, rows, 1, N) % (2 * 4 * N) == 0   # rows of partial sums, weight's and bias's


# ------------------------------------------------------------------ the binding's own checks
def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_tensors_must_be_on_a_gpu():
    q = bf16(1, 8, 2, 128)
    with pytest.raises(ValueError, match="CUDA"):
        sa.attn_fwd_bf16_lse(q, q, q)
    with pytest.raises(ValueError, match="CUDA"):
        sa.attn_bwd_bf16(q, q, q, q, q, torch.zeros(1, 2, 8))
    with pytest.raises(ValueError, match="CUDA"):
        sa.layer_norm_fwd(q)
    with pytest.raises(ValueError, match="CUDA"):
        sa.layer_norm_bwd(q, q, None, q[..., 0].float(), q[..., 0].float())


def test_ranks_and_types():
    with pytest.raises(ValueError, match="B, S, H, D"):
        sa.attn_fwd_bf16_lse(bf16(8, 128), bf16(8, 128), bf16(8, 128))
    with pytest.raises(ValueError, match="one to four"):
        sa.layer_norm_fwd(torch.zeros(()))
    with pytest.raises(ValueError, match="one to four"):
        sa.layer_norm_fwd(torch.zeros(1, 1, 1, 1, 1))
    with pytest.raises(ValueError, match="bfloat16, float16 or float32"):
        sa.layer_norm_fwd(torch.zeros(4, dtype=torch.float64))


def test_stride_arrays():
    t = bf16(2, 4, 3, 128)
    assert list(sa._strides("a b", t, t.permute(0, 2, 1, 3))) == [1536, 384, 128, 1, 1536, 128, 384, 1]
    with pytest.raises(ValueError, match="b must have unit channel stride"):
        sa._strides("a b", t, t.transpose(2, 3))
    assert list(sa._norm_strides("x", t[0, 0])) == [0, 0, 128, 1]
    assert list(sa._norm_strides("x", bf16(4, 2)[:, :1])) == [0, 0, 2, 1]
    with pytest.raises(ValueError, match="x must have unit channel stride"):
        sa._norm_strides("x", t.transpose(2, 3))
