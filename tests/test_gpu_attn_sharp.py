"""attn_bwd_bf16 where a key has nearly all of a row's probability: dP - delta is then of the size of what O's rounding
leaves in delta, and dQ is small.  Each row's error stays within a few times what its roundings come to
(train_rows.py), with that key in the first tile of 128, beyond it, on the diagonal, and in the last tile."""
import pytest
import torch

import sage_attention_forward_gb300 as sa
from train_ref import Reference
from train_rows import FACTOR, worst_rows

pytestmark = pytest.mark.gpu


def check(q, k, v, d, causal=False, kv_len=None):
    o, lse = sa.attn_fwd_bf16_lse(q, k, v, causal=causal, kv_len=kv_len)
    dq, dk, dv = sa.attn_bwd_bf16(d, q, k, v, o, lse, causal=causal, kv_len=kv_len)
    again = sa.attn_bwd_bf16(d, q, k, v, o, lse, causal=causal, kv_len=kv_len)
    torch.cuda.synchronize()
    sa.attn_get_device_status()
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dv), again))
    ref = Reference(q, k, v, None, causal, kv_len)
    far = worst_rows({"o": o, "dq": dq, "dk": dk, "dv": dv}, ref, d)
    rel = {n: float((t.double() - getattr(ref, n)).norm() / getattr(ref, n).norm())
           for n, t in (("dq", dq), ("dk", dk), ("dv", dv))}
    print(far, rel)
    assert max(far.values()) <= FACTOR, far
    return ref, rel


def make(dev, B, Sq, Sk, Hq, Hkv, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=dev)   # noqa: E731
    return r(B, Sq, Hq, 128), r(B, Sk, Hkv, 128), r(B, Sk, Hkv, 128), 0.1 * r(B, Sq, Hq, 128)


def bf(*tensors):
    return tuple(t.to(torch.bfloat16) for t in tensors)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("S", [260, 1000])
def test_queries_equal_to_keys(cuda_dev, S, causal):
    x, _, _, d = bf(*make(cuda_dev, 1, S, S, 3, 3, 12))
    _, rel = check(x, x, x, d, causal=causal)
    # the whole of it: the roundings of dS and of the result are u / sqrt(3) each, 0.0032 together; twice that
    assert rel["dq"] < 0.0065


@pytest.mark.parametrize("gain", [2.0, 4.0, 8.0, 16.0])
@pytest.mark.parametrize("mean", [0.0, 2.0])
def test_sharp_rows(cuda_dev, gain, mean):
    q, k, v, d = make(cuda_dev, 1, 300, 2048, 4, 2, 13)
    k = k + mean * torch.randn(2, 128, generator=torch.Generator(device=cuda_dev).manual_seed(1), device=cuda_dev)
    check(*bf(gain * q, k, v, d))


@pytest.mark.parametrize("at", [0, 127, 128, 700, 1299])
@pytest.mark.parametrize("share", [0.1, 0.2, 0.3])
def test_a_key_that_all_rows_look_at(cuda_dev, at, share):
    """With a share of 0.1 to 0.3 of that key in every query it has about half, most and all of the probability."""
    q, k, v, d = make(cuda_dev, 2, 300, 1300, 4, 2, 14)
    k[:, at] *= 3
    q = q + share * k[:, at].repeat_interleave(2, dim=1)[:, None]
    lens = torch.tensor([1300, at + 1], dtype=torch.int32, device=cuda_dev)
    check(*bf(q, k, v, d), kv_len=lens)


def test_strided_keys(cuda_dev):
    """The key's row is read where K's strides say."""
    g = torch.Generator(device=cuda_dev).manual_seed(15)
    x = torch.randn((2, 400, 3, 2, 128), generator=g, device=cuda_dev).to(torch.bfloat16)
    x[:, :, 1] = x[:, :, 0].flip(1)
    d = (0.1 * torch.randn((2, 400, 2, 128), generator=g, device=cuda_dev)).to(torch.bfloat16)
    ref, _ = check(x[:, :, 0], x[:, :, 1], x[:, :, 2], d)
    assert float((ref.p[..., 128:].amax(-1) > 0.5).double().mean()) > 0.5
    heads_first = x.permute(2, 0, 3, 1, 4).contiguous().permute(1, 3, 0, 2, 4)   # [.., S, 3, H, D] by heads
    check(heads_first[:, :, 0], heads_first[:, :, 1], heads_first[:, :, 2], d)


def test_keys_past_32_bits(cuda_dev):
    """K's rows 2^31 and more elements after its first: the same bits as from a tensor of its own."""
    x, _, _, d = bf(*make(cuda_dev, 2, 300, 300, 2, 2, 16))
    far = (1 << 31) + 256
    store = torch.empty(far + x[0].numel(), dtype=torch.bfloat16, device=cuda_dev)
    k = store.as_strided(x.shape, (far, *x.stride()[1:]), 0)
    k.copy_(x)
    o, lse = sa.attn_fwd_bf16_lse(x, k, x)
    got = sa.attn_bwd_bf16(d, x, k, x, o, lse)
    want = sa.attn_bwd_bf16(d, x, x, x, *sa.attn_fwd_bf16_lse(x, x, x))
    torch.cuda.synchronize()
    sa.attn_get_device_status()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ref = Reference(x, x, x)
    assert float((ref.p[:, :, 128:, 128:].amax(-1) > 0.5).double().mean()) > 0.5
