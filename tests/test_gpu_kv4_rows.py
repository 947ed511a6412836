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


def tight(q, k, v, step, v_step, seen, scale):
    """O, lse and their bounds for queries of whole numbers up to 127 (scaled by a power of two): every product with a code and every
    sum of a group, the constants 264 and 24 and all, is a whole multiple of one unit below 2^24 (32 x 271 x 127 < 2^20.1), exact in
    FP32 in any order.  What is left of a score's error, u = 2^-24: three additions of the groups' sums and their four products,
    fused (4 u of the sum of |q k|), the factor of query, scale and log2 e (rounded: 2 u, and its product: 1 u), and the difference
    to the reference maximum (1 u of each): 9 u sum |q k|, times the scale.  exp2 within 2^-22.  P as tests/kv4_ref.py has it."""
    G = q.shape[1] // k.shape[1]
    q = q.double()
    kk, vv, st = (t.repeat_interleave(G, 1) for t in (k, v, v_step))
    s = torch.einsum("shd,nhd->hsn", q, kk) * scale
    s = s.masked_fill(~seen[None], -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None])
    o = torch.einsum("hsn,nhd->shd", p, vv)
    off = (scale * 9 * 2.0 ** -24 * torch.einsum("shd,nhd->hsn", q.abs(), kk.abs())).masked_fill(~seen[None], 0.0).amax(-1)
    size = torch.einsum("hsn,nhd->shd", p, vv.abs())
    bound = size * (2.0 ** -11 + 2.0 ** -18 + 2 * off.T[..., None]) + v.shape[0] * 2.0 ** -28 * float(st.abs().max())
    return o, lse, bound, off + 2.0 ** -19 + lse.abs() * 2.0 ** -22


@pytest.mark.parametrize("Hq", [4, 8, 16])
@pytest.mark.parametrize("gain,scale", [(1.0, 0.001), (1.0, 0.0884), (2.0 ** -7, 0.0884), (1.0, 0.3), (2.0 ** 10, 2.0 ** -12)])
def test_scores_of_whole_queries(gain, scale, Hq, cuda_dev):
    """Flat and sharp rows (scores up to some hundreds apart), within about 10^-6 of the largest scores."""
    lens = (90, 700)
    cache, table, *kv = filled(40, lens, 1, 16, cuda_dev)
    g = torch.Generator().manual_seed(41)
    q = (torch.randint(-127, 128, (2, 1, Hq, 128), generator=g).double() * gain).to(torch.bfloat16)
    o, lse = sa.attn_fwd_kv4(q.to(cuda_dev), cache, table, ints(*lens).to(cuda_dev), softmax_scale=scale)
    for b, n in enumerate(lens):
        ref.check(o[b], lse[b], *tight(q[b], *(t[b, :n] for t in kv), torch.ones((1, n), dtype=torch.bool), scale))


@pytest.mark.parametrize("size", [3e38, 1e33, 2.0 ** -97])
@pytest.mark.parametrize("Hq", [4, 8, 16])
@pytest.mark.parametrize("lens", [(40, 5), (6000, 300)])
def test_values_at_the_ends_of_the_range(lens, Hq, size, cuda_dev):
    """Sums over many keys pass what FP32 holds where their mean does not; the other end has no bits to spare."""
    B, n, most = len(lens), max(lens), -(-max(lens) // 16)
    k, v = rows(50, B, n, 1, 128), rows(51, B, n, 1, 128, dtype=torch.float64).abs().clamp(0.05, 1.0)
    v = (v * size).to(torch.bfloat16)
    table, cache = torch.arange(B * most, dtype=torch.int32).view(B, most).to(cuda_dev), sa.kv4_cache(B * most, 1, 16, cuda_dev)
    sa.kv4_write(k.to(cuda_dev), v.to(cuda_dev), cache, table, ints(*[0] * B).to(cuda_dev), ints(*lens).to(cuda_dev))
    kv, q = ref.held(k, v), rows(52, B, 1, Hq, 128).to(cuda_dev)
    o, lse = sa.attn_fwd_kv4(q, cache, table, ints(*lens).to(cuda_dev))
    assert torch.isfinite(o).all()
    for b, m in enumerate(lens):
        seen = torch.ones((1, m), dtype=torch.bool)
        ref.check(o[b], lse[b], *ref.attention(q[b].cpu(), *(t[b, :m] for t in kv), seen, 128 ** -0.5))
