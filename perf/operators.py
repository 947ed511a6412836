"""What the training operators are measured on: attention's forward pass with the softmax statistics,
its backward pass, and layer norm's forward and backward pass.

`run` computes an operator in its plain form (elementary torch operations in 32 bits) or, with `own`
set, through this package's calls.  `exact` is the operator's definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

HEAD_DIM = 128
SCALE = 1.0 / math.sqrt(HEAD_DIM)
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# the most work that a drawn case takes: query-key pairs over all heads, and values of a layer norm
MOST_PAIRS = 16 * 16896 * 16896
MOST_VALUES = 76112 * 5120


def attention(name, op, B, Sq, Sk, Hq, Hkv, causal=False, kv_seed=-1):
    """kv_seed < 0: every key is real; else the batch entries' key counts are drawn from it."""
    return {"name": name, "op": op, "B": B, "Sq": Sq, "Sk": Sk, "Hq": Hq, "Hkv": Hkv, "causal": causal,
            "kv_seed": kv_seed}


def norm(name, op, B, S, H, N, dtype, weight="bf16", fused=False):
    """fused: x is a slice of a fused projection [B, S, 3, H, N], as Q is."""
    return {"name": name, "op": op, "B": B, "S": S, "H": H, "N": N, "dtype": dtype, "weight": weight, "fused": fused}


def listed():
    return [
        # the smallest workload of the benchmark: launches and the first tile's latency
        attention("attn fwd tiny", "attn_fwd", 1, 512, 512, 2, 2),
        # a causal language model's layer: shared key heads, an odd length, two prompts padded to one length
        attention("attn fwd causal gqa", "attn_fwd", 2, 4001, 4001, 32, 8, causal=True, kv_seed=3),
        # image tokens of FLUX at 1024^2 on padded text keys
        attention("attn fwd cross", "attn_fwd", 2, 4608, 512, 24, 24, kv_seed=5),
        # the same three kinds of layer in the backward pass
        attention("attn bwd tiny", "attn_bwd", 1, 512, 512, 2, 2),
        attention("attn bwd causal gqa", "attn_bwd", 2, 4001, 4001, 32, 8, causal=True, kv_seed=3),
        # many queries on few keys: the gradients of K and V are sums over a long axis
        attention("attn bwd cross", "attn_bwd", 1, 16896, 512, 24, 24, kv_seed=5),
        # joint attention of FLUX at 1024^2
        attention("attn bwd flux1024", "attn_bwd", 1, 4608, 4608, 24, 24),
        # the longest: FLUX at 2048^2 by length, 16 heads
        attention("attn bwd long", "attn_bwd", 1, 16896, 16896, 16, 16),
        # norm of each head's query channels, read where the fused projection left them
        norm("ln fwd qk", "ln_fwd", 1, 4608, 24, 128, "bf16", fused=True),
        # norm of a video model's tokens (Wan at 720p: 76112 tokens of 40 heads)
        norm("ln fwd tokens", "ln_fwd", 1, 76112, 1, 5120, "bf16"),
        norm("ln bwd qk", "ln_bwd", 1, 4608, 24, 128, "bf16", weight="fp32", fused=True),
        norm("ln bwd tokens", "ln_bwd", 1, 76112, 1, 5120, "bf16"),
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    op = rng.choice(["attn_fwd", "attn_bwd", "attn_bwd", "ln_fwd", "ln_bwd"])
    if op.startswith("ln"):
        n = spread(4, 16384)
        kind = rng.choice(["bf16", "fp16", "fp32"])
        rows = spread(1, max(1, min(131072, MOST_VALUES // n)))
        heads = rng.choice([1, 1, 2, 5])
        s = max(1, rows // heads)
        case = norm("", op, 1, s, heads, n, kind, weight=rng.choice([kind, "fp32"]), fused=rng.random() < 0.3)
    else:
        b, hkv, g = rng.randint(1, 4), spread(1, 16), rng.choice([1, 1, 2, 3, 8])
        sq, sk = spread(1, 16384), spread(1, 16384)
        if rng.random() < 0.5:
            sk = sq
        while b * hkv * g * sq * sk > MOST_PAIRS // 3:
            sq, sk = max(1, sq * 2 // 3), max(1, sk * 2 // 3)
        case = attention("", op, b, sq, sk, hkv * g, hkv, causal=rng.random() < 0.4,
                         kv_seed=rng.randrange(1000) if rng.random() < 0.5 else -1)
    del case["name"]
    return case


def key_counts(case):
    r = random.Random(case["kv_seed"])
    # short batches may have an entry without any key
    return [case["Sk"] if case["kv_seed"] < 0 else r.randint(case["Sk"] // 4 if case["Sk"] > 64 else int(b == 0), case["Sk"])
            for b in range(case["B"])]


def visible_pairs(case):
    """Query-key pairs that the masks leave, of one head over the batch."""
    i = np.arange(case["Sq"], dtype=np.int64)
    total = 0
    for n in key_counts(case):
        limit = np.minimum(n, i + 1 + case["Sk"] - case["Sq"]) if case["causal"] else np.full_like(i, n)
        total += int(np.maximum(limit, 0).sum())
    return total


def work(case):
    if case["op"].startswith("ln"):
        rows, n, e = case["B"] * case["S"] * case["H"], case["N"], 4 if case["dtype"] == "fp32" else 2
        w = 4 if case["weight"] == "fp32" else 2
        if case["op"] == "ln_fwd":
            return {"bytes": 2 * rows * n * e + 2 * n * w + 8 * rows, "flops": 8 * rows * n}
        return {"bytes": 3 * rows * n * e + 3 * n * w + 8 * rows, "flops": 14 * rows * n}
    queries, keys = case["B"] * case["Sq"] * case["Hq"], sum(key_counts(case)) * case["Hkv"]
    times = 1 if case["op"] == "attn_fwd" else 2
    return {"bytes": times * (4 * HEAD_DIM * queries + 4 * HEAD_DIM * keys) + 4 * queries,
            "flops": (4 if times == 1 else 10) * HEAD_DIM * visible_pairs(case) * case["Hq"]}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, gain=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device="cuda") * gain).to(dtype)

    if case["op"].startswith("ln"):
        B, S, H, N, t = case["B"], case["S"], case["H"], case["N"], TYPES[case["dtype"]]
        # activations have channels of their own mean and spread
        spread = torch.rand(N, generator=g, device="cuda") + 0.5
        x = torch.randn((B, S, 3 if case["fused"] else 1, H, N), generator=g, device="cuda") * spread + 0.25
        x = x.to(t)[:, :, 0]
        w = TYPES[case["weight"]]
        state = {"case": case, "x": x, "weight": (1.0 + normal(N, gain=0.2, dtype=torch.float32)).to(w),
                 "bias": normal(N, gain=0.2, dtype=w)}
        if case["op"] == "ln_bwd":
            state["dy"] = normal(B, S, H, N, gain=0.1, dtype=t)
            state["mean"], state["rstd"] = statistics(x)
        return state
    B, Sq, Sk, Hq, Hkv = (case[n] for n in ("B", "Sq", "Sk", "Hq", "Hkv"))
    if Sq == Sk and Hq == Hkv:
        # self-attention reads its operands where one fused projection wrote them
        qkv = normal(B, Sq, 3, Hq, HEAD_DIM)
        q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    else:
        q, k, v = normal(B, Sq, Hq, HEAD_DIM), normal(B, Sk, Hkv, HEAD_DIM), normal(B, Sk, Hkv, HEAD_DIM)
    k += normal(Hkv, HEAD_DIM, gain=0.5)   # keys have channels of their own mean
    n = None
    if case["kv_seed"] >= 0:
        n = torch.tensor(key_counts(case), dtype=torch.int32, device="cuda")
    state = {"case": case, "q": q, "k": k, "v": v, "kv_len": n}
    if case["op"] == "attn_bwd":
        state["do"] = normal(B, Sq, Hq, HEAD_DIM, gain=0.05)
        state["o"], state["lse"] = plain_forward(state)
    return state


def grouped(t, Hkv):
    """[B, S, H, D] -> 32-bit [B, Hkv, H / Hkv, S, D]."""
    B, S, H, D = t.shape
    return t.float().reshape(B, S, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4)


def hidden(state):
    """Truth values of the keys that a query does not see, to be broadcast over [B, Hkv, G, Sq, Sk]; None if there are none."""
    case = state["case"]
    j = torch.arange(case["Sk"], device="cuda")
    out = None
    if state["kv_len"] is not None:
        out = (j >= state["kv_len"][:, None]).view(case["B"], 1, 1, 1, case["Sk"])
    if case["causal"]:
        i = torch.arange(case["Sq"], device="cuda")[:, None]
        late = j > i + (case["Sk"] - case["Sq"])
        out = late if out is None else out | late
    return out


def plain_scores(state):
    q, k = grouped(state["q"], state["case"]["Hkv"]), grouped(state["k"], state["case"]["Hkv"])
    s = torch.matmul(q * SCALE, k.transpose(-1, -2))
    mask = hidden(state)
    return s if mask is None else s.masked_fill_(mask, -math.inf)


def plain_forward(state):
    case = state["case"]
    B, Sq, Hq, Hkv = case["B"], case["Sq"], case["Hq"], case["Hkv"]
    s = plain_scores(state)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, grouped(state["v"], Hkv)) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + total.log()).reshape(B, Hq, Sq)
    return o.permute(0, 3, 1, 2, 4).reshape(B, Sq, Hq, HEAD_DIM).to(torch.bfloat16), lse


def plain_backward(state):
    case = state["case"]
    B, Sq, Sk, Hq, Hkv = (case[n] for n in ("B", "Sq", "Sk", "Hq", "Hkv"))
    q, k, v, do = (grouped(state[n], Hkv) for n in ("q", "k", "v", "do"))
    lse = state["lse"].reshape(B, Hkv, Hq // Hkv, Sq, 1)
    p = plain_scores(state).sub_(torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)).exp_()
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    dp = torch.matmul(do, v.transpose(-1, -2))
    ds = dp.sub_((p * dp).sum(-1, keepdim=True)).mul_(p).mul_(SCALE)
    dq = torch.matmul(ds, k).permute(0, 3, 1, 2, 4).reshape(B, Sq, Hq, HEAD_DIM)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2)
    return {"dq": dq.to(torch.bfloat16), "dk": dk.transpose(1, 2).to(torch.bfloat16),
            "dv": dv.transpose(1, 2).to(torch.bfloat16)}


def statistics(x):
    x = x.float()
    mean = x.mean(-1)
    return mean, torch.rsqrt((x - mean[..., None]).square().mean(-1) + EPS)


def plain_norm(state):
    x = state["x"].float()
    mean, rstd = statistics(x)
    y = (x - mean[..., None]) * rstd[..., None] * state["weight"].float() + state["bias"].float()
    return {"y": y.to(state["x"].dtype), "mean": mean, "rstd": rstd}


def plain_norm_backward(state):
    x, dy, w = state["x"].float(), state["dy"].float(), state["weight"]
    xhat = (x - state["mean"][..., None]) * state["rstd"][..., None]
    g = dy * w.float()
    dx = (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True)) * state["rstd"][..., None]
    return {"dx": dx.to(state["x"].dtype), "dweight": (dy * xhat).sum((0, 1, 2)).to(w.dtype),
            "dbias": dy.sum((0, 1, 2)).to(w.dtype)}


def run(state):
    case = state["case"]
    if own:
        import sage_attention_forward_gb300 as sa
        if case["op"] == "attn_fwd":
            o, lse = sa.attn_fwd_bf16_lse(state["q"], state["k"], state["v"], causal=case["causal"],
                                          kv_len=state["kv_len"])
            return {"o": o, "lse": lse}
        if case["op"] == "attn_bwd":
            dq, dk, dv = sa.attn_bwd_bf16(state["do"], state["q"], state["k"], state["v"], state["o"], state["lse"],
                                          causal=case["causal"], kv_len=state["kv_len"])
            return {"dq": dq, "dk": dk, "dv": dv}
        if case["op"] == "ln_fwd":
            y, mean, rstd = sa.layer_norm_fwd(state["x"], state["weight"], state["bias"], eps=EPS)
            return {"y": y, "mean": mean, "rstd": rstd}
        dx, dweight, dbias = sa.layer_norm_bwd(state["dy"], state["x"], state["weight"], state["mean"], state["rstd"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if case["op"] == "attn_fwd":
        o, lse = plain_forward(state)
        return {"o": o, "lse": lse}
    if case["op"] == "attn_bwd":
        return plain_backward(state)
    return plain_norm(state) if case["op"] == "ln_fwd" else plain_norm_backward(state)


def exact(case, seed):
    """The definitions in 64 bits: attention one query head at a time."""
    state = prepare(case, seed)
    if case["op"].startswith("ln"):
        x = state["x"].double()
        w = state["weight"].double()
        mean = x.mean(-1)
        var = (x * x).mean(-1) - mean * mean   # 64 bits leave 1e-14 of the mean's square
        rstd = 1.0 / torch.sqrt(var + EPS)
        xhat = (x - mean.unsqueeze(-1)) * rstd.unsqueeze(-1)
        if case["op"] == "ln_fwd":
            return {"y": xhat * w + state["bias"].double(), "mean": mean, "rstd": rstd}
        dy = state["dy"].double()
        n = case["N"]
        a = (dy * w).sum(-1, keepdim=True) / n
        b = (dy * w * xhat).sum(-1, keepdim=True) / n
        return {"dx": rstd.unsqueeze(-1) * (dy * w - a - b * xhat), "dweight": torch.einsum("bshn,bshn->n", dy, xhat),
                "dbias": dy.reshape(-1, n).sum(0)}
    B, Sq, Sk, Hq, Hkv = (case[n] for n in ("B", "Sq", "Sk", "Hq", "Hkv"))
    out = {n: torch.zeros((B, Sq, Hq, HEAD_DIM), dtype=torch.float64, device="cuda") for n in ("o", "dq")}
    out |= {n: torch.zeros((B, Sk, Hkv, HEAD_DIM), dtype=torch.float64, device="cuda") for n in ("dk", "dv")}
    out["lse"] = torch.full((B, Hq, Sq), -math.inf, dtype=torch.float64, device="cuda")
    counts = key_counts(case)
    for b in range(B):
        n = counts[b]
        if n == 0:
            continue
        for h in range(Hq):
            g = h // (Hq // Hkv)
            q, k, v = state["q"][b, :, h].double(), state["k"][b, :n, g].double(), state["v"][b, :n, g].double()
            t = q @ k.T / math.sqrt(HEAD_DIM)
            if case["causal"]:
                seen = torch.ones((Sq, n), dtype=torch.bool, device="cuda").tril(Sk - Sq)
                t = torch.where(seen, t, torch.full_like(t, -math.inf))
            lse = torch.logsumexp(t, dim=1)
            p = torch.nan_to_num(torch.exp(t - lse[:, None]), nan=0.0)
            del t
            if case["op"] == "attn_fwd":
                out["lse"][b, h], out["o"][b, :, h] = lse, p @ v
                continue
            do = state["do"][b, :, h].double()
            out["dv"][b, :n, g] += p.T @ do
            ds = do @ v.T
            ds -= (ds * p).sum(1, keepdim=True)
            ds *= p
            del p
            out["dq"][b, :, h] = ds @ k / math.sqrt(HEAD_DIM)
            out["dk"][b, :n, g] += ds.T @ q / math.sqrt(HEAD_DIM)
    return {n: out[n] for n in (("o", "lse") if case["op"] == "attn_fwd" else ("dq", "dk", "dv"))}
