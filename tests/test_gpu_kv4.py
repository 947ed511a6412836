"""kv4_write, kv4_read and attn_fwd_kv4 on the GPU against tests/kv4_ref.py."""
import math

import numpy as np
import pytest
import torch

import kv4_ref as ref
import sage_attention_forward_gb300 as sa

pytestmark = pytest.mark.gpu


def rows(seed, *shape, gain=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * gain).to(dtype)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32)


def pages(seed, B, most, extra=3):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(B * most + extra, generator=g)[:B * most].to(torch.int32).view(B, most)


# S, kv heads, page size, pages a request, starts, counts
WRITES = [
    (1, 1, 16, 2, (0, 15, 16, 31), None),              # a token at a record's ends
    (1, 3, 32, 1, (5, 40, -1), None),                  # past the table's end, before the first token
    (40, 2, 16, 4, (0, 3, 30), (40, 0, 29)),           # padding, a request without tokens
    (17, 1, 48, 3, (47, -5), (99, 17)),                # across pages; more than there are; from before the first token
    (64, 2, 64, 1, (0, 1), (-3, 64)),
    (8, 1, 16, 1, (2 ** 31 - 4, -2 ** 31), None),
]


@pytest.mark.parametrize("case", WRITES, ids=str)
def test_write_and_read(case, cuda_dev):
    S, H, size, most, start, count = case
    B = len(start)
    k, v = rows(1, B, S, H, 128), rows(2, B, S, H, 128, gain=0.01)
    k[..., 7] *= 30                                    # a channel that stands out
    k[0, 0, 0, 32:64] = 0                              # a group of zeros, one too small, ties, subnormal values beside it
    k[0, 0, 0, 64:96] = 2.0 ** -110
    v[0, 0, 0, :32] = torch.arange(32).to(torch.bfloat16) / 2 - 8
    v[0, 0, 0, 32:64] = 2.0 ** -99
    v[0, 0, 0, 40:50] = 1e-40
    v[0, 0, 0, 64:96], v[0, 0, 0, 70], v[0, 0, 0, 80] = 1.0, -3e38, 3e38
    table = pages(3, B, most)
    table[-1, 0] = -1 if most > 1 else table[-1, 0]
    table[0, -1] = 10 ** 6 if most > 2 else table[0, -1]
    cache = torch.randint(0, 256, (B * most + 3, H, size // 16, 2304), dtype=torch.uint8)
    want = cache.numpy().copy()
    ref.write(want, table.numpy(), start, count or (S,) * B, k, v)
    got, dev_table, dev_start = cache.to(cuda_dev), table.to(cuda_dev), ints(*start).to(cuda_dev)
    dev_count = None if count is None else ints(*count).to(cuda_dev)
    sa.kv4_write(k.to(cuda_dev), v.to(cuda_dev), got, dev_table, dev_start, dev_count)
    wrong = np.argwhere(got.cpu().numpy() != want)
    assert len(wrong) == 0, f"{len(wrong)} bytes, the first at {wrong[:8].tolist()}"
    read = sa.kv4_read(got, dev_table, dev_start, S, dev_count)
    for x, y in zip((k, v), read):
        exact = ref.values(x)
        for b in range(B):
            for i in range(S):
                at = start[b] + i
                there = i < (count or (S,) * B)[b] and 0 <= at < most * size and 0 <= int(table[b, at // size]) < len(want)
                assert torch.equal(y[b, i].cpu(), exact[b, i].to(torch.bfloat16) if there else torch.zeros_like(x[b, i]))


def test_pieces_of_a_record_join(cuda_dev):
    """A prompt written token by token, and in pieces on the way, leaves the bytes of one call."""
    k, v = rows(4, 1, 50, 2, 128).to(cuda_dev), rows(5, 1, 50, 2, 128).to(cuda_dev)
    table = pages(6, 1, 4).to(cuda_dev)
    whole, parts = sa.kv4_cache(7, 2, 16), sa.kv4_cache(7, 2, 16)
    sa.kv4_write(k, v, whole, table, ints(3).to(cuda_dev))
    at = 0
    for n in (1, 1, 20, 5, 1, 22):
        sa.kv4_write(k[:, at:at + n], v[:, at:at + n], parts, table, ints(3 + at).to(cuda_dev))
        at += n
    assert at == 50 and torch.equal(whole, parts)


def filled(seed, lens, H, size, dev, garbage=True):
    """A cache of requests of these lengths (unwritten bytes are anything), the table, and what the codes stand for."""
    B, most = len(lens), max(1, -(-max(lens) // size))
    k, v = rows(seed, B, max(max(lens), 1), H, 128), rows(seed + 1, B, max(max(lens), 1), H, 128)
    k += rows(seed + 2, H, 128, gain=0.5)
    table = pages(seed + 3, B, most).to(dev)
    cache = sa.kv4_cache(B * most + 3, H, size, dev)
    if garbage:
        cache.fill_(255)                               # codes of 7, scales of NaN
    sa.kv4_write(k.to(dev), v.to(dev), cache, table, ints(*[0] * B).to(dev), ints(*lens).to(dev))
    return cache, table, *ref.held(k, v)


def verify(got, q, lens, kv, causal, scale=1 / math.sqrt(128), gone=None):
    Sq = q.shape[1]
    for b, n in enumerate(lens):
        seen = torch.ones((Sq, n), dtype=torch.bool)
        if causal:
            seen = torch.arange(n)[None] < n - Sq + 1 + torch.arange(Sq)[:, None]
        if gone is not None:
            seen &= ~gone[b][:n]
        o, lse, bound, lse_bound = ref.attention(q[b].cpu(), *(t[b, :n] for t in kv), seen, scale)
        ref.check(got[0][b], got[1][b], o, lse, bound, lse_bound)


# lengths, queries, query heads, key heads, page size, causal
CASES = [
    ((1,), 1, 1, 1, 16, True),
    ((0, 5), 1, 4, 2, 16, True),                       # a request without a key
    ((15, 16, 17, 33), 1, 8, 8, 16, True),
    ((100, 3, 64), 1, 8, 1, 32, True),                 # eight heads on one key head
    ((70, 2, 0, 31), 4, 7, 1, 16, True),               # 28 rows: two tiles; rows before the first key
    ((70, 2, 0, 31), 4, 7, 1, 16, False),
    ((1000, 1), 1, 32, 8, 64, True),                   # unequal shares
    ((129,) * 9, 2, 4, 1, 128, True),
    ((700,), 5, 12, 4, 16, True),                      # 15 of 16 columns
    ((300, 20), 40, 6, 2, 48, True),                   # 120 rows a key head
    ((5000, 4999), 1, 2, 2, 16, True),                 # one head over many CTAs
    ((37, 1, 250, 0, 90) * 30, 1, 4, 2, 16, True),     # more requests than a CTA's threads
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}-" + "-".join(map(str, c[1:])))
def test_attention(case, cuda_dev):
    lens, Sq, Hq, H, size, causal = case
    cache, table, *kv = filled(10, lens, H, size, cuda_dev)
    q = rows(20, len(lens), Sq, Hq, 128, gain=2.0).to(cuda_dev)
    got = sa.attn_fwd_kv4(q, cache, table, ints(*lens).to(cuda_dev), causal=causal)
    verify(got, q, lens, kv, causal)


@pytest.mark.parametrize("gain,scale", [(1e-3, None), (1e4, 1e-4), (1e-30, 1e28), (1e30, 1e-30), (1.0, 0.0), (60.0, 0.3)])
def test_sizes_of_queries_and_scales(gain, scale, cuda_dev):
    lens = (90, 33)
    cache, table, *kv = filled(30, lens, 2, 16, cuda_dev)
    q = rows(31, 2, 2, 4, 128, gain=gain).to(cuda_dev)
    q[0, 0, 0] = 0
    got = sa.attn_fwd_kv4(q, cache, table, ints(*lens).to(cuda_dev), softmax_scale=scale)
    verify(got, q, lens, kv, True, scale=128 ** -0.5 if scale is None else scale)


def test_growing_and_falling_scores(cuda_dev):
    """A reference maximum that is raised again and again, and one that the first record sets."""
    n = 600
    for rising in (True, False):
        at = torch.arange(n).double() / n * 6
        k = (at if rising else at.flip(0))[:, None].expand(n, 128).to(torch.bfloat16)[None, :, None].contiguous()
        v = rows(41, 1, n, 1, 128)
        table, cache = pages(42, 1, 38).to(cuda_dev), sa.kv4_cache(41, 1, 16)
        sa.kv4_write(k.to(cuda_dev), v.to(cuda_dev), cache, table, ints(0).to(cuda_dev))
        q = torch.ones((1, 1, 3, 128), dtype=torch.bfloat16, device=cuda_dev)
        got = sa.attn_fwd_kv4(q, cache, table, ints(n).to(cuda_dev))
        verify(got, q, (n,), ref.held(k, v), True)


@pytest.mark.parametrize("sizes", [(0.0, 0.0), (1e-28, 1e-20), (1e-20, 1e20), (1e20, 1e-20), (1e30, 1e30)])
def test_sizes_of_values(sizes, cuda_dev):
    """Values that grow and fall along the context, tiny, huge and zero ones."""
    n, lens = 300, (300, 77)
    k, v = rows(45, 2, n, 2, 128), rows(46, 2, n, 2, 128, dtype=torch.float64)
    step = torch.linspace(0, 1, n, dtype=torch.float64)[None, :, None, None]
    v = (v * (sizes[0] ** (1 - step) * sizes[1] ** step if sizes[0] else 0 * step)).to(torch.bfloat16)
    table, cache = pages(47, 2, 19).to(cuda_dev), sa.kv4_cache(41, 2, 16)
    sa.kv4_write(k.to(cuda_dev), v.to(cuda_dev), cache, table, ints(0, 0).to(cuda_dev))
    for Hq in (2, 12, 20):   # each form: 4, 8 and 16 queries
        q = rows(48 + Hq, 2, 1, Hq, 128).to(cuda_dev)
        got = sa.attn_fwd_kv4(q, cache, table, ints(*lens).to(cuda_dev))
        verify(got, q, lens, ref.held(k, v), True)


def test_pages_that_are_none(cuda_dev):
    """Their keys are not seen: holes anywhere, a request of nothing but holes."""
    lens = (200, 64, 90)
    cache, table, *kv = filled(50, lens, 2, 16, cuda_dev)
    table[0, 3], table[0, 12], table[0, 7] = -1, 2 ** 31 - 1, cache.shape[0]
    table[1] = -7
    gone = torch.zeros((3, 208), dtype=torch.bool)
    for page in (3, 12, 7):
        gone[0, 16 * page:16 * page + 16] = True
    gone[1] = True
    q = rows(51, 3, 3, 4, 128).to(cuda_dev)
    got = sa.attn_fwd_kv4(q, cache, table, ints(*lens).to(cuda_dev))
    verify(got, q, lens, kv, True, gone=gone)
    assert not got[0][1].any() and (got[1][1] == -math.inf).all()


def test_lengths_beyond_the_table_and_below_zero(cuda_dev):
    cache, table, *kv = filled(60, (32, 32, 32), 1, 16, cuda_dev)
    q = rows(61, 3, 1, 2, 128).to(cuda_dev)
    got = sa.attn_fwd_kv4(q, cache, table, ints(32, 2 ** 31 - 1, -5).to(cuda_dev))
    verify(got, q, (32, 32, 0), kv, True)


def test_strides_streams_and_graphs(cuda_dev):
    lens = (300, 41)
    n = ints(*lens).to(cuda_dev)
    cache, table, *kv = filled(70, lens, 2, 32, cuda_dev)
    q = rows(71, 2, 3, 8, 128).to(cuda_dev)
    want = sa.attn_fwd_kv4(q, cache, table, n)
    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))  # noqa: E731
    # heads before tokens; a table's row inside a wider one; outputs in a slice
    wide = torch.full((2, 99), -1, dtype=torch.int32, device=cuda_dev)
    wide[:, 5:5 + table.shape[1]] = table
    view = wide[:, 5:5 + table.shape[1]]
    out = torch.zeros((2, 8, 7, 128), dtype=torch.bfloat16, device=cuda_dev)
    got = sa.attn_fwd_kv4(q.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3), cache, view, n,
                          out=out.permute(0, 2, 1, 3)[:, 2:5])
    assert same(got, want) and not out[:, :, :2].any() and not out[:, :, 5:].any()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sa.attn_fwd_kv4(q, cache, table, n, stream=side)
    side.synchronize()
    assert same(got, want)
    # a captured step: a token is written, then seen; replayed as the request grows
    k, v = rows(72, 2, 1, 2, 128).to(cuda_dev), rows(73, 2, 1, 2, 128).to(cuda_dev)
    at, now = ints(299, 40).to(cuda_dev), ints(300, 41).to(cuda_dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sa.kv4_write(k, v, cache, table, at)
        step = sa.attn_fwd_kv4(q[:, :1], cache, table, now)
    eager = cache.clone()
    for _ in range(5):
        graph.replay()
        sa.kv4_write(k, v, eager, table, at)
        assert torch.equal(cache, eager) and same(step, sa.attn_fwd_kv4(q[:, :1], eager, table, now))
        at += 1
        now += 1
        k.mul_(-1.5)


def test_thousands_of_requests(cuda_dev):
    """More requests than a warp looks at together, many without a key; some of them checked."""
    g = torch.Generator().manual_seed(75)
    lens = tuple(torch.randint(-20, 60, (3000,), generator=g).clamp(min=0).tolist())
    B, H, size = len(lens), 1, 16
    k, v = rows(76, B, 60, H, 128), rows(77, B, 60, H, 128)
    table = pages(78, B, 4).to(cuda_dev)
    cache, n = sa.kv4_cache(B * 4 + 3, H, size, cuda_dev), ints(*lens).to(cuda_dev)
    sa.kv4_write(k.to(cuda_dev), v.to(cuda_dev), cache, table, torch.zeros_like(n), n)
    q = rows(79, B, 1, 2, 128).to(cuda_dev)
    o, lse = sa.attn_fwd_kv4(q, cache, table, n)
    some = list(range(0, B, 43)) + [B - 1]
    verify((o[some], lse[some]), q[some], [lens[b] for b in some], [t[some] for t in ref.held(k, v)], True)
    empty = (n == 0).nonzero()[:, 0]
    assert not o[empty].any() and (lse[empty] == -math.inf).all()


def test_two_calls_at_once(cuda_dev):
    """On two streams, each with its own workspace, again and again: the bits of one call alone."""
    problems = []
    for seed, lens, H in ((110, (2000, 7, 650), 2), (120, (333, 4000), 1)):
        cache, table, *_ = filled(seed, lens, H, 32, cuda_dev)
        q, n = rows(seed + 9, len(lens), 2, 4, 128).to(cuda_dev), ints(*lens).to(cuda_dev)
        problems.append((q, cache, table, n))
    want = [sa.attn_fwd_kv4(*p) for p in problems]
    streams = [torch.cuda.Stream() for _ in problems]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [sa.attn_fwd_kv4(*p, stream=s) for p, s in zip(problems, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_many_rounds_give_the_same_bits(cuda_dev):
    lens = (3000, 5, 800)
    cache, table, *_ = filled(80, lens, 2, 64, cuda_dev)
    q, n = rows(81, 3, 2, 8, 128).to(cuda_dev), ints(*lens).to(cuda_dev)
    want = sa.attn_fwd_kv4(q, cache, table, n)
    for _ in range(10):
        got = sa.attn_fwd_kv4(q, cache, table, n)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_cache_past_2_to_the_31_bytes(cuda_dev):
    H, size = 4, 64
    num = 2 ** 32 // (H * size // 16 * 2304) + 8      # 4 GB
    cache = torch.empty((num, H, size // 16, 2304), dtype=torch.uint8, device=cuda_dev)
    lens = (100, 65)
    table = torch.tensor([[num - 1, num // 2 + 3], [num - 2, 0]], dtype=torch.int32, device=cuda_dev)
    k, v = rows(90, 2, 100, H, 128), rows(91, 2, 100, H, 128)
    start = ints(0, 0).to(cuda_dev)
    sa.kv4_write(k.to(cuda_dev), v.to(cuda_dev), cache, table, start, ints(*lens).to(cuda_dev))
    got = sa.kv4_read(cache, table, start, 100, ints(*lens).to(cuda_dev))
    for x, y in zip((k, v), got):
        for b, n in enumerate(lens):
            assert torch.equal(y[b, :n].cpu(), ref.values(x[b, :n]).to(torch.bfloat16)) and not y[b, n:].any()
    q = rows(92, 2, 1, 8, 128).to(cuda_dev)
    verify(sa.attn_fwd_kv4(q, cache, table, ints(*lens).to(cuda_dev)), q, lens, ref.held(k, v), True)


def test_a_prompt_in_pieces(cuda_dev):
    """Norm, rotation, cache and attention together: a prompt through the BF16 attention, its keys into the cache, then a
    token at a time; and a second piece of a prompt on the cache's values read back."""
    B, n, Hq, H = 1, 75, 4, 2
    freq, m = sa.rope_frequencies(128, scaling={"kind": "yarn", "factor": 4, "length": 64}, device=cuda_dev)
    qkv = rows(100, B, n + 3, Hq + 2 * H, 128).to(cuda_dev)
    w = (1 + rows(101, 128, dtype=torch.float32, gain=0.1)).to(cuda_dev)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:]
    place = torch.arange(n + 3, dtype=torch.int32, device=cuda_dev)
    q, k = sa.qk_norm_rope_fwd(q, k, w, w, freq, place, magnitude=m)
    v = v.contiguous()
    cache, table = sa.kv4_cache(8, H, 16), pages(102, 1, 5).to(cuda_dev)
    sa.kv4_write(k[:, :n], v[:, :n], cache, table, ints(0).to(cuda_dev))
    kv = ref.held(k.cpu(), v.cpu())
    for i in range(n, n + 3):
        sa.kv4_write(k[:, i:i + 1], v[:, i:i + 1], cache, table, ints(i).to(cuda_dev))
        got = sa.attn_fwd_kv4(q[:, i:i + 1], cache, table, ints(i + 1).to(cuda_dev))
        verify(got, q[:, i:i + 1], (i + 1,), kv, True)
    kr, vr = sa.kv4_read(cache, table, ints(0).to(cuda_dev), n + 3)
    a, lse = sa.attn_fwd_bf16_lse(q[:, 40:], kr, vr, causal=True)
    b, other = sa.attn_fwd_kv4(q[:, 40:], cache, table, ints(n + 3).to(cuda_dev))
    # two forms of one result: K and V's values rounded to BF16 (2^-8 each) and P in both
    assert (a.float() - b.float()).abs().max() < 0.05 and (lse - other).abs().max() < 0.05
