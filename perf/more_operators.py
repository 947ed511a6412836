"""What the operators between a projection and attention are measured on: rotary positions, the norm of queries and
keys with the rotation in the same pass (each with its backward pass), and a K/V cache in 4 bits with the attention
that reads it.

`run` computes an operator in its plain form (elementary torch operations in 32 bits, angles in 64) or, with `own`
set, through this package's calls.  `exact` is the operator's definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6
D = 128                        # channels of a head in the cache
GROUP = 32                     # channels that share a scale
TILE = 16                      # tokens of a record of the cache: K codes, V codes, scales
RECORD = TILE * 2 * (D // 2 + 2 * (D // GROUP))
# the most work that a drawn case takes: values of Q and K, and tokens times key heads in the cache
MOST_VALUES = 76112 * 80 * 128
MOST_CACHED = 8 * 131072 * 8


# ------------------------------------------------------------------ cases
def rotation(name, op, B, S, Hq, Hk, N, R, dtype, interleaved=False, axes="", start=0, scaling="none", weight="bf16",
             fused=False):
    """N channels a head, the first R of them rotated.  axes: channels of each position axis ("": one axis, from
    `start` on).  fused: Q and K are slices of a fused projection [B, S, 3, H, N]."""
    return {"name": name, "op": op, "B": B, "S": S, "Hq": Hq, "Hk": Hk, "N": N, "R": R, "dtype": dtype,
            "interleaved": interleaved, "axes": axes, "start": start, "scaling": scaling, "weight": weight,
            "fused": fused}


def cached(name, op, B, S, Hq, Hk, longest, page, ragged=False, causal=True):
    """S new tokens of each of B requests whose caches hold up to `longest` tokens, the new ones included."""
    return {"name": name, "op": op, "B": B, "S": S, "Hq": Hq, "Hk": Hk, "longest": longest, "page": page,
            "ragged": ragged, "causal": causal}


def listed():
    return [
        # one decoding step of a batch: a token of each request, positions far into a context beyond the trained one
        rotation("rope fwd decode", "rope_fwd", 64, 1, 32, 8, 128, 128, "bf16", start=100000, scaling="bands"),
        # Q and K of a video model's layer (Wan at 720p): frame, row and column positions
        rotation("rope fwd video", "rope_fwd", 1, 76112, 40, 40, 128, 128, "bf16", interleaved=True, axes="44,42,42"),
        # the gradient where only part of a head of 80 channels is rotated
        rotation("rope bwd partial", "rope_bwd", 2, 4001, 32, 8, 80, 32, "fp16", scaling="linear"),
        # the smallest workload of the benchmark
        rotation("norm rope fwd tiny", "norm_fwd", 1, 512, 2, 2, 128, 128, "bf16", fused=True),
        # FLUX at 1024^2: text and image tokens, Q and K where the fused projection left them
        rotation("norm rope fwd flux1024", "norm_fwd", 1, 4608, 24, 24, 128, 128, "bf16", interleaved=True,
                 axes="16,56,56", fused=True),
        # the same layer at 2048^2 in training
        rotation("norm rope bwd flux2048", "norm_bwd", 1, 16896, 24, 24, 128, 128, "bf16", interleaved=True,
                 axes="16,56,56", weight="fp32", fused=True),
        # a causal language model's layer in 32 bits, shared key heads, an odd length, stretched positions
        rotation("norm rope bwd gqa", "norm_bwd", 2, 4001, 32, 8, 64, 64, "fp32", scaling="yarn", weight="fp32"),
        # a decoding step's new keys and values, and what the cache holds of them
        cached("cache append", "kv4_write", 128, 1, 8, 8, 2048, 16, ragged=True),
        # prompts of an odd length
        cached("cache prompt", "kv4_write", 4, 8191, 8, 8, 9000, 64),
        # one request, a few drafted tokens: launches and latency
        cached("cached attn tiny", "attn_kv4", 1, 4, 8, 2, 700, 16),
        # a serving batch of many lengths, one token each
        cached("cached attn batch", "attn_kv4", 64, 1, 32, 8, 8192, 64, ragged=True),
        # long contexts, one token each
        cached("cached attn long", "attn_kv4", 8, 1, 32, 8, 131072, 64),
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    op = rng.choice(["rope_fwd", "rope_bwd", "norm_fwd", "norm_bwd", "norm_bwd", "kv4_write", "attn_kv4", "attn_kv4",
                     "attn_kv4"])
    if op in ("kv4_write", "attn_kv4"):
        hk, b = spread(1, 16), spread(1, 128)
        longest = spread(1, max(1, min(131072, MOST_CACHED // (2 * b * hk))))
        new = spread(1, min(longest, 8192 if op == "kv4_write" else 8))
        case = cached("", op, b, new, hk * rng.choice([1, 2, 4, 7, 8]), hk, longest, rng.choice([16, 32, 64, 128]),
                      ragged=rng.random() < 0.6, causal=rng.random() < 0.8)
    else:
        n = rng.choice([128, 128, 64, 80, 96, 256, 2 * spread(2, 128), spread(3, 256)])
        r = n // 2 * 2 if rng.random() < 0.5 else 2 * rng.randint(1, n // 2)
        hk = spread(1, 16)
        hq = hk * rng.choice([1, 1, 2, 4, 8])
        s = spread(1, max(1, min(65536, MOST_VALUES // (4 * n * (hq + hk)))))
        b = rng.randint(1, 4) if s > 16 else spread(1, 128)
        axes = ""
        if r >= 6 and rng.random() < 0.4:
            part = r // 6 * 2
            axes = "%d,%d,%d" % (r - 2 * part, part, part)
        kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        case = rotation("", op, b, s, hq, hk, n, r, kind, interleaved=rng.random() < 0.5, axes=axes,
                        start=spread(1, 1 << 20) if rng.random() < 0.5 else 0,
                        scaling=rng.choice(["none", "linear", "bands", "yarn"]), weight=rng.choice([kind, "fp32"]),
                        fused=hq == hk and rng.random() < 0.5)
    del case["name"]
    return case


def lengths(case):
    """Tokens of each request's cache, the new ones included.  In a ragged batch of short contexts one has none."""
    n, new = case["longest"], case["S"]
    if not case["ragged"]:
        return [n] * case["B"]
    r = random.Random("%d %d %d" % (case["B"], n, new))
    counts = [r.randint(min(n, max(new, n // 16)), n) for _ in range(case["B"])]
    if case["op"] == "attn_kv4" and case["B"] > 1 and n < 64:
        counts[r.randrange(case["B"])] = 0
    return counts


def work(case):
    if case["op"] in ("kv4_write", "attn_kv4"):
        held = RECORD // TILE
        if case["op"] == "kv4_write":
            tokens = case["B"] * case["S"] * case["Hk"]
            return {"bytes": tokens * (2 * 4 * D + 2 * held), "flops": tokens * 2 * 8 * D}
        n = np.asarray(lengths(case), dtype=np.int64)
        seen = n[:, None] - (np.arange(case["S"])[::-1] if case["causal"] else np.zeros(case["S"], dtype=np.int64))
        rows = case["B"] * case["S"] * case["Hq"]
        return {"bytes": int(n.sum()) * case["Hk"] * held + rows * (4 * D + 4),
                "flops": 4 * D * int(np.maximum(seen, 0).sum()) * case["Hq"]}
    rows = case["B"] * case["S"] * (case["Hq"] + case["Hk"])
    e = SIZES[case["dtype"]]
    rotate = 3 * case["R"]
    if case["op"] == "norm_bwd":
        return {"bytes": 3 * rows * case["N"] * e, "flops": rows * (11 * case["N"] + rotate)}
    return {"bytes": 2 * rows * case["N"] * e,
            "flops": rows * (rotate + (4 * case["N"] if case["op"] == "norm_fwd" else 0))}


# ------------------------------------------------------------------ inputs
def sections(case):
    """Position axis of each rotated pair."""
    widths = [int(w) for w in case["axes"].split(",")] if case["axes"] else [case["R"]]
    return np.repeat(np.arange(len(widths)), np.asarray(widths) // 2), widths


def frequencies(case):
    """Radians a position of each pair, in 64 bits, and the factor of cosine and sine."""
    axis, widths = sections(case)
    inside = np.concatenate([np.arange(w // 2) / (w // 2) for w in widths])
    w = 10000.0 ** -inside
    if case["scaling"] == "linear":      # positions interpolated
        return w / 4.0, 1.0
    if case["scaling"] == "bands":       # long wavelengths stretched, short ones kept, a ramp between
        turns = 8192 * w / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        return w * keep + w / 8.0 * (1.0 - keep), 1.0
    if case["scaling"] == "yarn":
        turns = 4096 * w / (2 * math.pi)
        keep = np.clip((np.log(np.maximum(turns, 1e-30)) - math.log(1.0)) / (math.log(32.0) - math.log(1.0)), 0.0, 1.0)
        return w * keep + w / 16.0 * (1.0 - keep), 0.1 * math.log(16.0) + 1.0
    return w, 1.0


def places(case, g):
    """int32 positions: [B, S] of consecutive tokens, or [1, S, 3] of a grid of frames, rows and columns."""
    s = torch.arange(case["S"], device="cuda", dtype=torch.int32)
    if case["axes"]:
        side = max(1, int(math.sqrt(case["S"] / 4)))
        return torch.stack([s // (side * side), s // side % side, s % side], dim=-1)[None]
    first = torch.zeros((case["B"], 1), dtype=torch.int32, device="cuda")
    if case["start"]:
        first = torch.randint(0, case["start"], (case["B"], 1), generator=g, device="cuda", dtype=torch.int32)
    return first + s


def quantise(x):
    """Codes in [-8, 7] (32-bit values) and scales [..., 4] of BF16 rows [..., 128]."""
    x = x.float().unflatten(-1, (D // GROUP, GROUP))
    top, low = x.amax(-1), x.amin(-1)
    ext = torch.where(top >= -low, top, low)
    ext = torch.where(ext.abs() < 2.0 ** -100, torch.zeros_like(ext), ext)
    scale = ext * -0.125
    code = (x / torch.where(scale == 0, torch.ones_like(scale), scale)[..., None]).round_().clamp_(-8, 7)
    code = torch.where((scale == 0)[..., None], torch.zeros_like(code), code)
    return code.flatten(-2), scale


def byte_sources():
    """Where a record's 2048 code bytes take their low and their high 4 bits from: indexes into [K, V][16 tokens][128]."""
    at = np.zeros((2, 2048), dtype=np.int64)
    token, word, i = np.meshgrid(np.arange(TILE), np.arange(16), np.arange(8), indexing="ij")
    # K: a token's 64 bytes in four pieces of 16, a word of each group in every piece
    k_from = token * D + GROUP * (word % 4) + 8 * (word // 4) + i
    k_byte = token * 64 + word * 4 + i // 2
    # V: 8 bytes of each token in every piece, four channels of each group in every one
    piece, half, j = word // 2, word % 2, i
    v_from = TILE * D + token * D + GROUP * (2 * half + j // 4) + 4 * piece + j % 4
    v_byte = 1024 + token // 8 * 512 + (4 * piece + token % 8 // 2) * 16 + token % 2 * 8 + half * 4 + j // 2
    for src, byte in ((k_from, k_byte), (v_from, v_byte)):
        at[(i % 2).ravel(), byte.ravel()] = src.ravel()
    return at


def make_cache(case, k, v):
    """The cache of K and V [B, longest, Hk, 128], pages in mixed order, and the table [B, pages] of their places."""
    B, n, hk, page = case["B"], case["longest"], case["Hk"], case["page"]
    per = -(-n // page)
    pad = (0, 0, 0, 0, 0, per * page - n)
    parts, scales = [], []
    for x in (k, v):
        code, scale = quantise(torch.nn.functional.pad(x, pad))
        code = (code + 8).to(torch.uint8).view(B * per, page // TILE, TILE, hk, D)
        parts.append(code.permute(0, 3, 1, 2, 4).reshape(-1, TILE * D))
        scale = scale.to(torch.bfloat16).view(B * per, page // TILE, TILE, hk, D // GROUP)
        scales.append(scale.permute(0, 3, 1, 2, 4).reshape(-1, TILE, D // GROUP))
    low, high = (torch.from_numpy(a).to("cuda") for a in byte_sources())
    codes = torch.cat(parts, dim=1)
    packed = codes.index_select(1, low) | (codes.index_select(1, high) << 4)
    scales = torch.cat(scales, dim=-1).reshape(-1, TILE * 2 * (D // GROUP)).view(torch.uint8)
    return torch.cat([packed, scales], dim=1).view(B * per, hk, page // TILE, RECORD), per


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, gain=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device="cuda") * gain).to(dtype)

    B, S, Hq, Hk = (case[n] for n in ("B", "S", "Hq", "Hk"))
    if case["op"] in ("kv4_write", "attn_kv4"):
        counts = torch.tensor(lengths(case), dtype=torch.int32, device="cuda")
        spread = torch.rand((2, Hk, D), generator=g, device="cuda") + 0.5   # channels have spreads of their own
        pages = -(-case["longest"] // case["page"])
        order = torch.randperm(B * pages, generator=g, device="cuda")
        state = {"case": case, "table": order.to(torch.int32).view(B, pages), "len": counts}
        if case["op"] == "kv4_write":
            state["k"], state["v"] = ((torch.randn((B, S, Hk, D), generator=g, device="cuda") * w).to(torch.bfloat16)
                                      for w in spread)
            state["start"] = torch.clamp(counts - S, min=0)
            state["cache"] = torch.zeros((B * pages, Hk, case["page"] // TILE, RECORD), dtype=torch.uint8, device="cuda")
            return state
        k, v = ((torch.randn((B, case["longest"], Hk, D), generator=g, device="cuda") * w).to(torch.bfloat16)
                for w in spread)
        k += normal(Hk, D, gain=0.5)   # keys have channels of their own mean
        cache, pages = make_cache(case, k, v)
        state["cache"] = torch.empty_like(cache)
        state["cache"][order] = cache
        state["q"] = normal(B, S, Hq, D)
        return state
    N, t = case["N"], TYPES[case["dtype"]]
    if case["fused"]:
        qkv = normal(B, S, 3, Hq, N, dtype=t)
        q, k = qkv[:, :, 0], qkv[:, :, 1]
    else:
        q, k = normal(B, S, Hq, N, dtype=t), normal(B, S, Hk, N, dtype=t)
    w, magnitude = frequencies(case)
    axis, _ = sections(case)
    # turns a position in units of 2^-64, the axis in the two lowest bits
    turns = [(round(x / (2 * math.pi) * 2.0 ** 64) & ~3 | int(a)) for x, a in zip(w.tolist(), axis)]
    state = {"case": case, "q": q, "k": k, "magnitude": magnitude, "pos": places(case, g),
             "w": torch.tensor(w, dtype=torch.float64, device="cuda"),
             "axis": torch.tensor(axis, device="cuda"),
             "freq": torch.tensor(np.array(turns, dtype=np.uint64).view(np.int64), device="cuda")}
    if case["op"].startswith("norm"):
        kind = TYPES[case["weight"]]
        state["qw"], state["kw"] = ((1.0 + normal(N, gain=0.2, dtype=torch.float32)).to(kind) for _ in range(2))
    if case["op"].endswith("bwd"):
        state["dq"], state["dk"] = normal(B, S, Hq, N, gain=0.1, dtype=t), normal(B, S, Hk, N, gain=0.1, dtype=t)
    return state


# ------------------------------------------------------------------ plain forms
def cos_sin(state):
    """[B or 1, S, 1, R / 2] in 32 bits, from angles in 64."""
    pos, w = state["pos"].double(), state["w"]
    angle = pos.index_select(-1, state["axis"]) * w if state["case"]["axes"] else pos[..., None] * w
    m = state["magnitude"]
    return (angle.cos() * m).float()[:, :, None], (angle.sin() * m).float()[:, :, None]


def rotate(x, cos, sin, case):
    """x [..., N] in 32 bits."""
    R = case["R"]
    y = x.clone()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if case["interleaved"] else (slice(0, R // 2), slice(R // 2, R))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def plain_norm(x, w, cos, sin, case):
    f = x.float()
    r = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
    return rotate(f * r * w.float(), cos, sin, case).to(x.dtype)


def plain_norm_backward(dy, x, w, cos, sin, case):
    f = x.float()
    r = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
    xhat = f * r
    g = rotate(dy.float(), cos, -sin, case)
    gw = g * w.float()
    dx = (gw - xhat * (gw * xhat).mean(-1, keepdim=True)) * r
    return dx.to(x.dtype), (g * xhat).sum((0, 1, 2)).to(w.dtype)


def plain_values(x):
    code, scale = quantise(x)
    return (code * scale.repeat_interleave(GROUP, -1)).to(torch.bfloat16)


def unpack(state):
    """K and V in 32 bits, [B, Hk, pages * page, 128]."""
    case = state["case"]
    at = byte_sources()
    place = np.zeros(2 * TILE * D, dtype=np.int64)
    place[at[0]] = 2 * np.arange(2048)
    place[at[1]] = 2 * np.arange(2048) + 1
    byte, shift = torch.from_numpy(place // 2).to("cuda"), torch.from_numpy(place % 2 * 4).to(torch.uint8).to("cuda")
    rec = state["cache"][state["table"].long()]                     # [B, pages, Hk, tiles, RECORD]
    B, pages, hk, tiles, _ = rec.shape
    scale = rec[..., 2048:].contiguous().view(torch.bfloat16).float().view(B, pages, hk, tiles, TILE, 2, D // GROUP)
    code = rec.view(-1, RECORD).index_select(1, byte).bitwise_right_shift_(shift).bitwise_and_(15)
    code = code.view(B, pages, hk, tiles, 2, TILE, D // GROUP, GROUP)
    return [((code[..., i, :, :, :].float() - 8.0) * scale[..., i, :, None]).permute(0, 2, 1, 3, 4, 5, 6)
            .reshape(B, hk, pages * tiles * TILE, D) for i in range(2)]


def plain_attention(state):
    case = state["case"]
    B, S, Hq, Hk = (case[n] for n in ("B", "S", "Hq", "Hk"))
    k, v = unpack(state)
    q = state["q"].float().view(B, S, Hk, Hq // Hk, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, -1, D)
    s = torch.matmul(q * (1.0 / math.sqrt(D)), k.transpose(-1, -2)).view(B, Hk, S, Hq // Hk, -1)
    i = torch.arange(S, device="cuda")
    limit = state["len"][:, None] - (S - 1 - i if case["causal"] else 0 * i)
    hidden = torch.arange(s.shape[-1], device="cuda") >= limit[..., None]
    s = s.masked_fill_(hidden[:, None, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hk, -1, p.shape[-1]), v).view(B, Hk, S, Hq // Hk, D)
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + total.log()).squeeze(-1).permute(0, 1, 3, 2).reshape(B, Hq, S)
    return {"o": o.permute(0, 2, 1, 3, 4).reshape(B, S, Hq, D).to(torch.bfloat16), "lse": lse}


def run_own(state):
    import sage_attention_forward_gb300 as sa
    case, op = state["case"], state["case"]["op"]
    if op == "attn_kv4":
        o, lse = sa.attn_fwd_kv4(state["q"], state["cache"], state["table"], state["len"], causal=case["causal"])
        return {"o": o, "lse": lse}
    if op == "kv4_write":
        sa.kv4_write(state["k"], state["v"], state["cache"], state["table"], state["start"])
        k, v = sa.kv4_read(state["cache"], state["table"], state["start"], case["S"])
        return {"k": k, "v": v}
    how = {"interleaved": case["interleaved"], "magnitude": state["magnitude"]}
    if op == "rope_fwd":
        q, k = sa.rope_fwd(state["q"], state["k"], state["freq"], state["pos"], **how)
    elif op == "rope_bwd":
        q, k = sa.rope_bwd(state["dq"], state["dk"], state["freq"], state["pos"], **how)
    elif op == "norm_fwd":
        q, k = sa.qk_norm_rope_fwd(state["q"], state["k"], state["qw"], state["kw"], state["freq"], state["pos"],
                                   eps=EPS, **how)
    else:
        dq, dk, dqw, dkw = sa.qk_norm_rope_bwd(state["dq"], state["dk"], state["q"], state["k"], state["qw"],
                                               state["kw"], state["freq"], state["pos"], eps=EPS, **how)
        return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}
    return {"q": q, "k": k}


def run(state):
    if own:
        return run_own(state)
    case, op = state["case"], state["case"]["op"]
    if op == "attn_kv4":
        return plain_attention(state)
    if op == "kv4_write":
        return {"k": plain_values(state["k"]), "v": plain_values(state["v"])}
    cos, sin = cos_sin(state)
    if op == "norm_fwd":
        return {"q": plain_norm(state["q"], state["qw"], cos, sin, case),
                "k": plain_norm(state["k"], state["kw"], cos, sin, case)}
    if op == "norm_bwd":
        dq, dqw = plain_norm_backward(state["dq"], state["q"], state["qw"], cos, sin, case)
        dk, dkw = plain_norm_backward(state["dk"], state["k"], state["kw"], cos, sin, case)
        return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}
    back = op == "rope_bwd"
    q, k = (state["dq"], state["dk"]) if back else (state["q"], state["k"])
    sin = -sin if back else sin
    return {"q": rotate(q.float(), cos, sin, case).to(q.dtype), "k": rotate(k.float(), cos, sin, case).to(k.dtype)}


# ------------------------------------------------------------------ the definitions in 64 bits
def turned(x, state, sign):
    """x times e^(i sign angle) in pairs of channels, as complex numbers."""
    case = state["case"]
    half = case["R"] // 2
    pos = state["pos"].double()
    if pos.dim() == 2 and not case["axes"]:
        angle = torch.einsum("bs,r->bsr", pos, state["w"])
    else:
        angle = torch.stack([pos[0, :, a] for a in state["axis"].tolist()], dim=-1)[None] * state["w"]
    e = torch.polar(torch.full_like(angle, state["magnitude"]), sign * angle)[:, :, None]
    head = x[..., :case["R"]]
    if case["interleaved"]:
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], half, 2).contiguous()) * e
        out = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(head[..., :half].contiguous(), head[..., half:].contiguous()) * e
        out = torch.cat([z.real, z.imag], dim=-1)
    return torch.cat([out, x[..., case["R"]:]], dim=-1)


def exact_rotation(state):
    case, op = state["case"], state["case"]["op"]
    out = {}
    for n in ("q", "k"):
        if op == "rope_fwd":
            out[n] = turned(state[n].double(), state, 1.0)
        elif op == "rope_bwd":
            out[n] = turned(state["d" + n].double(), state, -1.0)
        else:
            x, w = state[n].double(), state[n + "w"].double()
            rms = ((x * x).sum(-1, keepdim=True) / case["N"] + EPS).sqrt()
            if op == "norm_fwd":
                out[n] = turned(x / rms * w, state, 1.0)
                continue
            g = turned(state["d" + n].double(), state, -1.0)
            out["d" + n] = g * w / rms - x * (g * w * x).sum(-1, keepdim=True) / (case["N"] * rms ** 3)
            out["d" + n + "w"] = torch.einsum("bshn,bshn->n", g, x / rms)
    return out


def exact_values(x):
    """Each value's nearest multiple (ties to even) of its group's step among -8 to 7 of them."""
    x = x.double().reshape(*x.shape[:-1], D // GROUP, GROUP)
    most, least = x.max(-1, keepdim=True).values, x.min(-1, keepdim=True).values
    step = torch.where(most + least >= 0, most, least) / -8.0
    step = torch.where(step.abs() < 2.0 ** -103, torch.full_like(step, math.inf), step)
    n = torch.round(x / step).clamp(-8.0, 7.0)
    return torch.where(n == 0, torch.zeros_like(x), n * step).flatten(-2)


def exact_attention(state):
    """One request and key head at a time; codes read from their places in a record by arithmetic."""
    case = state["case"]
    B, S, Hq, Hk = (case[n] for n in ("B", "S", "Hq", "Hk"))
    G = Hq // Hk
    o = torch.zeros((B, S, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, S), -math.inf, dtype=torch.float64, device="cuda")
    t = torch.arange(TILE, device="cuda")[:, None]
    c = torch.arange(D, device="cuda")[None]
    group, inside = c // GROUP, c % GROUP
    k_nibble = t * 128 + inside // 8 * 32 + group * 8 + inside % 8
    v_nibble = 2048 + t // 8 * 1024 + (inside // 4 * 4 + t % 8 // 2) * 32 + t % 2 * 16 + group * 4 + inside % 4
    for b, n in enumerate(lengths(case)):
        if n == 0:
            continue
        used = state["table"][b, :-(-n // case["page"])].long()
        for h in range(Hk):
            rec = state["cache"][used, h].reshape(-1, RECORD)
            steps = rec[:, 2048:].contiguous().view(torch.bfloat16).double().view(-1, TILE, 2, D // GROUP)
            k, v = (((rec[:, at.flatten() // 2].int() >> (at.flatten() % 2 * 4).int() & 15) - 8).double()
                    .view(-1, TILE, D) * steps[:, :, i, :].repeat_interleave(GROUP, -1)
                    for i, at in enumerate((k_nibble, v_nibble)))
            k, v = k.reshape(-1, D)[:n], v.reshape(-1, D)[:n]
            q = state["q"][b, :, h * G:(h + 1) * G].double()
            a = torch.einsum("sgd,nd->gsn", q, k) / math.sqrt(D)
            if case["causal"]:
                seen = torch.ones((S, n), dtype=torch.bool, device="cuda").tril(n - S)
                a = torch.where(seen, a, torch.full_like(a, -math.inf))
            z = torch.logsumexp(a, dim=-1)
            p = torch.nan_to_num(torch.exp(a - z[..., None]), nan=0.0)
            o[b, :, h * G:(h + 1) * G] = torch.einsum("gsn,nd->sgd", p, v)
            lse[b, h * G:(h + 1) * G] = z
    return {"o": o, "lse": lse}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "attn_kv4":
        return exact_attention(state)
    if case["op"] == "kv4_write":
        return {"k": exact_values(state["k"]), "v": exact_values(state["v"])}
    return exact_rotation(state)
