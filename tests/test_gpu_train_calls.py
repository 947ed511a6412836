"""Calls of the training operators that the documentation allows and the other tests do not make."""
import pytest
import torch

import sage_attention_forward_gb300 as sa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,N", [(700, 128), (300, 129), (400, 1000), (900, 1773), (700, 5120), (320, 9000), (200, 12288),
                                    (40, 16384)])
def test_layer_norm_gradient_over_its_input(cuda_dev, rows, N, dtype):
    """dx in x's place: the same bits as in a tensor of its own."""
    g = torch.Generator(device=cuda_dev).manual_seed(N)
    x, dy = (torch.randn((rows, N), generator=g, device=cuda_dev).to(dtype) for _ in range(2))
    w = torch.randn(N, generator=g, device=cuda_dev).to(dtype)
    _, mean, rstd = sa.layer_norm_fwd(x, w, w)
    want = sa.layer_norm_bwd(dy, x, w, mean, rstd)
    x2 = x.clone()
    got = sa.layer_norm_bwd(dy, x2, w, mean, rstd, dx=x2)
    torch.cuda.synchronize()
    sa.attn_get_device_status()
    assert got[0] is x2 and all(torch.equal(a, b) for a, b in zip(got, want))


def test_streams_by_handle(cuda_dev):
    """A stream as torch's object, as its handle, as another library's object, and the default stream's handle."""
    class Other:
        def __init__(self, handle):
            self.cuda_stream = handle

    g = torch.Generator(device=cuda_dev).manual_seed(3)
    q, k, v, d = (torch.randn((1, 200, 2, 128), generator=g, device=cuda_dev).to(torch.bfloat16) for _ in range(4))
    s = torch.cuda.Stream()
    results = []
    for stream in (None, s, s.cuda_stream, Other(s.cuda_stream), 0):
        torch.cuda.synchronize()
        y, mean, rstd = sa.layer_norm_fwd(q, stream=stream)
        o, lse = sa.attn_fwd_bf16_lse(y, k, v, stream=stream)
        grads = sa.attn_bwd_bf16(d, y, k, v, o, lse, stream=stream)
        dx, _, _ = sa.layer_norm_bwd(grads[0], q, None, mean, rstd, stream=stream)
        torch.cuda.synchronize()
        results.append((y, mean, rstd, o, lse, *grads, dx))
    for r in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, results[0]))


@pytest.mark.parametrize("value", [0.0, -30.0, -1e4, 40.0, float("inf"), float("nan")])
@pytest.mark.parametrize("Sq,Sk", [(300, 700), (500, 128), (5, 3)])
def test_an_lse_of_another_call(cuda_dev, Sq, Sk, value):
    """Not the forward's: the gradients may be anything then, but they come, and the next call's are right."""
    g = torch.Generator(device=cuda_dev).manual_seed(4)
    r = lambda *s: torch.randn(s, generator=g, device=cuda_dev).to(torch.bfloat16)   # noqa: E731
    q, k, v, d = r(2, Sq, 4, 128), r(2, Sk, 2, 128), r(2, Sk, 2, 128), r(2, Sq, 4, 128)
    o, lse = sa.attn_fwd_bf16_lse(q, k, v)
    want = sa.attn_bwd_bf16(d, q, k, v, o, lse)
    sa.attn_bwd_bf16(d, q, k, v, o, torch.full_like(lse, value))
    got = sa.attn_bwd_bf16(d, q, k, v, o, lse)
    torch.cuda.synchronize()
    sa.attn_get_device_status()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
