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
