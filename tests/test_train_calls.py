"""Calls of the training operators that the binding has to refuse by itself, since the library never sees what is wrong
with them (CPU: tensors without data, the library's own checks behind them)."""
import pytest
import torch

import sage_attention_forward_gb300 as sa


@pytest.fixture
def on_meta(monkeypatch):
    """Takes tensors without data for tensors of the current device."""
    monkeypatch.setattr(sa, "_cuda_index", lambda name, t: t.get_device())
    monkeypatch.setattr(sa, "_elsewhere", lambda dev, stream: False)
    monkeypatch.setattr(sa, "_current_stream", lambda dev: 0)


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def norm_tensors(*shape):
    stats = [meta(*shape[:-1], dtype=torch.float32) for _ in range(2)]
    return meta(*shape), meta(*shape), *stats


@pytest.mark.parametrize("shape", [((1 << 32) + 3, 8), (1 << 31, 4), (2, (1 << 32) + 1, 1, 16), (3, (1 << 32) + 128)])
def test_layer_norm_sizes_past_32_bits(on_meta, shape):
    x, y, mean, rstd = norm_tensors(*shape)
    with pytest.raises(ValueError, match="2\\^31"):
        sa.layer_norm_fwd(x, out=y, mean=mean, rstd=rstd)
    with pytest.raises(ValueError, match="2\\^31"):
        sa.layer_norm_bwd(y, x, None, mean, rstd, dx=meta(*shape))
    with pytest.raises(ValueError, match="2\\^31"):
        sa.layer_norm_bwd_workspace(shape, "meta")


@pytest.mark.parametrize("B,Sq,Sk,Hq,Hkv", [(1, (1 << 32) + 5, 7, 1, 1), (1, 5, (1 << 32) + 7, 1, 1),
                                            ((1 << 32) + 1, 5, 7, 1, 1), (1, 5, 7, (1 << 32) + 2, (1 << 32) + 2)])
def test_attention_sizes_past_32_bits(on_meta, B, Sq, Sk, Hq, Hkv):
    q, k = meta(B, Sq, Hq, 128), meta(B, Sk, Hkv, 128)
    lse = meta(B, Hq, Sq, dtype=torch.float32)
    with pytest.raises(ValueError, match="2\\^31"):
        sa.attn_fwd_bf16_lse(q, k, k, out=q, lse=lse)
    with pytest.raises(ValueError, match="2\\^31"):
        sa.attn_bwd_bf16(q, q, k, k, q, lse, dq=q, dk=k, dv=k, workspace=meta(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="2\\^31"):
        sa.attn_bwd_workspace(B, Sq, Sk, Hq, Hkv, "meta")


def test_ordinary_sizes_reach_the_library(on_meta):
    """(What these tests take the place of: the library is called, and reports the missing data.)"""
    x, y, mean, rstd = norm_tensors(6, 8)
    with pytest.raises(sa.AttnError, match="x is NULL"):
        sa.layer_norm_fwd(x, out=y, mean=mean, rstd=rstd)
    q = meta(1, 5, 2, 128)
    with pytest.raises(sa.AttnError, match="q is NULL"):
        sa.attn_fwd_bf16_lse(q, q, q, out=q, lse=meta(1, 2, 5, dtype=torch.float32))


class OtherDevicesStream:
    """What the binding looks at of a stream, without a GPU."""
    device = torch.device("cuda", 1)
    cuda_stream = 4096


@pytest.mark.parametrize("call", ["layer_norm_fwd", "layer_norm_bwd", "attn_fwd_bf16_lse", "attn_bwd_bf16"])
def test_a_stream_of_another_device(monkeypatch, call):
    """torch makes a stream's device current with it, and the call would run on some stream of the tensors' device."""
    monkeypatch.setattr(sa, "_cuda_index", lambda name, t: 0)
    monkeypatch.setattr(sa, "_expect", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "Stream", OtherDevicesStream)
    q = meta(1, 5, 2, 128)
    lse = meta(1, 2, 5, dtype=torch.float32)
    args = {"layer_norm_fwd": (q,), "layer_norm_bwd": (q, q, None, lse, lse), "attn_fwd_bf16_lse": (q, q, q),
            "attn_bwd_bf16": (q, q, q, q, q, lse)}[call]
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        getattr(sa, call)(*args, stream=OtherDevicesStream())
