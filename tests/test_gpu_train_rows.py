"""O, dQ, dK and dV of the training kernels row by row against what their roundings come to (train_rows.py): a wrong row,
key or remainder tile among many shows, where worst-case bounds over all keys leave it room."""
import math

import pytest
import torch

from test_gpu_attn_sharp import check
from test_gpu_attn_train import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,Sq,Sk,Hq,Hkv", [
    (1, 1, 1, 1, 1), (1, 1, 129, 2, 1), (1, 130, 1, 1, 1), (2, 2, 3, 2, 2), (1, 129, 127, 2, 2), (2, 200, 300, 6, 2),
    (1, 513, 257, 4, 1), (1, 257, 700, 3, 3), (1, 1000, 1000, 2, 2), (3, 384, 640, 8, 1), (1, 1111, 1025, 4, 2)])
def test_shapes(cuda_dev, B, Sq, Sk, Hq, Hkv, causal):
    check(*make(cuda_dev, B, Sq, Sk, Hq, Hkv, seed=Sq + Sk), causal=causal)


@pytest.mark.parametrize("Sq,Sk,Hq,Hkv,causal", [(6000, 130, 2, 1, False), (3, 6000, 2, 1, True), (64, 5000, 4, 4, False),
                                                 (4000, 257, 4, 1, True), (2500, 2500, 2, 1, True)])
def test_long_axes(cuda_dev, Sq, Sk, Hq, Hkv, causal):
    check(*make(cuda_dev, 1, Sq, Sk, Hq, Hkv, seed=Sq), causal=causal)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Sq,Sk,lens", [(300, 300, [300, 1, 0, 129]), (70, 520, [128, 127, 129, 520]), (1, 300, [1, 0, 300, 200]),
                                        (900, 1000, [1000, 999, 513, 640])])
def test_key_counts_and_garbage_padding(cuda_dev, Sq, Sk, lens, causal):
    q, k, v, d = make(cuda_dev, len(lens), Sq, Sk, 4, 2, seed=7)
    n = torch.tensor(lens, dtype=torch.int32, device=cuda_dev)
    for b, x in enumerate(lens):
        k[b, x:] = math.nan
        v[b, x:] = math.inf
    check(q, k, v, d, causal=causal, kv_len=n)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,Sq,Sk,Hq,Hkv,lens", [(3, 300, 300, 64, 64, [300, 1, 0]), (1, 2000, 130, 4, 2, None),
                                                 (5, 100, 700, 40, 20, [0, 700, 0, 129, 640])])
def test_many_items_and_divided_sums(cuda_dev, B, Sq, Sk, Hq, Hkv, lens, causal):
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=cuda_dev)
    check(*make(cuda_dev, B, Sq, Sk, Hq, Hkv, seed=30 + B), causal=causal, kv_len=n)


@pytest.mark.parametrize("offset", [0.5, 4.0])
def test_keys_and_values_with_a_mean(cuda_dev, offset):
    g = torch.Generator(device=cuda_dev).manual_seed(5)
    q, k, v, d = make(cuda_dev, 1, 1200, 1200, 2, 2, seed=44)
    mean = lambda: offset * torch.randn(2, 128, generator=g, device=cuda_dev)   # noqa: E731
    check(q, (k.float() + mean()).to(torch.bfloat16), v, d)
    check(q, k, (v.float() + mean()).to(torch.bfloat16), d)
