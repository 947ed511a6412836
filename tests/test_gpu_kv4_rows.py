"""attn_fwd_kv4 where a row's numbers are special: queries that are no numbers."""
import math

import pytest
import torch

import kv4_ref as ref
import sage_attention_forward_gb300 as sa
from test_gpu_kv4 import filled, ints, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq", [4, 8, 16])                # 4, 8 and 16 queries a key head
@pytest.mark.parametrize("lens", [(40, 5), (6000, 300)])  # a head within one warp's work, and in pieces that are joined
def test_a_query_that_is_no_number(Hq, lens, cuda_dev):
    """Its row is NaN, in O and in lse (a merge by lse would drop a row of -inf); the others are what they are without it."""
    cache, table, *kv = filled(10, lens, 1, 16, cuda_dev)
    q = rows(11, 2, 1, Hq, 128).to(cuda_dev)
    bad = q.clone()
    bad[0, 0, 1, 5], bad[1, 0, 2, 127] = math.nan, math.inf
    o, lse = sa.attn_fwd_kv4(bad, cache, table, ints(*lens).to(cuda_dev))
    for b, h in ((0, 1), (1, 2)):
        assert torch.isnan(o[b, 0, h]).all() and torch.isnan(lse[b, h, 0])
        keep = [i for i in range(Hq) if i != h]
        seen = torch.ones((1, lens[b]), dtype=torch.bool)
        want = ref.attention(q[b, :, keep].cpu(), *(t[b, :lens[b]] for t in kv), seen, 128 ** -0.5)
        ref.check(o[b, :, keep], lse[b, keep], *want)


@pytest.mark.parametrize("gains", [(1.0, 2.0 ** -16, 2.0 ** -32, 2.0 ** -64), (2.0 ** -40, 2.0 ** 60, 0.0, 1.0)])
@pytest.mark.parametrize("Hq", [4, 8, 16])
@pytest.mark.parametrize("lens", [(40, 5), (6000, 300)])
def test_groups_of_values_of_unlike_sizes(lens, Hq, gains, cuda_dev):
    """V's groups of 32 channels have scales of their own: what one holds is no matter of another's size."""
    B, n, most = len(lens), max(lens), -(-max(lens) // 16)
    size = torch.tensor(gains, dtype=torch.float64).repeat_interleave(32)
    k, v = rows(20, B, n, 1, 128), (rows(21, B, n, 1, 128, dtype=torch.float64) * size).to(torch.bfloat16)
    table, cache = torch.arange(B * most, dtype=torch.int32).view(B, most).to(cuda_dev), sa.kv4_cache(B * most, 1, 16, cuda_dev)
    sa.kv4_write(k.to(cuda_dev), v.to(cuda_dev), cache, table, ints(*[0] * B).to(cuda_dev), ints(*lens).to(cuda_dev))
    kv, q = ref.held(k, v), rows(22, B, 1, Hq, 128).to(cuda_dev)
    o, lse = sa.attn_fwd_kv4(q, cache, table, ints(*lens).to(cuda_dev))
    for b, m in enumerate(lens):
        seen = torch.ones((1, m), dtype=torch.bool)
        for g in range(4):
            part = slice(32 * g, 32 * g + 32)
            kb, vb, ks, vs = (t[b, :m] for t in kv)
            want = ref.attention(q[b].cpu(), kb, vb[..., part], ks, vs[..., part], seen, 128 ** -0.5)
            ref.check(o[b][..., part], lse[b], *want)
