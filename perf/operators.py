"""Grouped-query attention over a paged key-value cache: the cases its three
operators are measured on, with the operators in plain form and in 64 bits.

    append   new tokens' keys and values go into a paged cache, keys and
             queries turned by their positions on the way (gqa_cache_append)
    decode   the last T tokens of every sequence attend to the paged cache
             (gqa_decode_attn)
    prompt   causal attention over packed prompts of different lengths
             (gqa_prompt_attn)

A cache is [n_pages][kv heads][page][d]: position p of sequence b is slot
p % page of page table[b][p // page].  Rotation turns the interleaved pairs of
the last r dims of a head by pos * theta^(-2j/r).  An FP8 cache holds E4M3
codes and one fp32 scale for every row, amax / 448.
"""

import math
import random

import numpy as np
import torch

own = False

_ACT = {"bf16": torch.bfloat16, "f16": torch.float16}
_THETA = 1e4


# ---- cases ---------------------------------------------------------------------

def listed():
    return [
        # One decode step of a served batch: a token for each of 32 sequences
        # far into their contexts; launch latency is all there is.
        dict(name="append step", op="append", act="bf16", kv="act", batch=32, longest=1, base=100000, heads=32,
             kv_heads=8, d=128, r=128, page=64, mix=1),
        # Prefill of a packed batch of prompts, rotation on the last 64 dims.
        dict(name="append prompts", op="append", act="bf16", kv="act", batch=12, longest=4096, base=0, heads=32,
             kv_heads=8, d=128, r=64, page=64, mix=2),
        # The same into an FP8 cache with small pages, later chunks of long
        # prompts, narrow heads.
        dict(name="append fp8", op="append", act="f16", kv="fp8", batch=5, longest=8191, base=5000, heads=16,
             kv_heads=4, d=64, r=64, page=16, mix=3),
        # One user's short context: the smallest decode call.
        dict(name="decode single", op="decode", act="bf16", kv="act", batch=1, longest=777, tokens=1, heads=32,
             kv_heads=8, d=128, page=16, window=0, sink=False, mix=4),
        # A served batch of mixed contexts.
        dict(name="decode batch", op="decode", act="bf16", kv="act", batch=32, longest=16384, tokens=1, heads=64,
             kv_heads=8, d=128, page=64, window=0, sink=False, mix=5),
        # Few sequences at 128K: the cache's bytes are everything.
        dict(name="decode 128k", op="decode", act="bf16", kv="act", batch=4, longest=131072, tokens=1, heads=64,
             kv_heads=8, d=128, page=128, window=0, sink=False, mix=0),
        # The same kind of batch on an FP8 cache, with attention sinks.
        dict(name="decode fp8", op="decode", act="bf16", kv="fp8", batch=24, longest=32768, tokens=1, heads=64,
             kv_heads=8, d=128, page=64, window=0, sink=True, mix=6),
        # Four drafted tokens checked at once by a sliding-window layer.
        dict(name="decode draft", op="decode", act="f16", kv="act", batch=16, longest=5000, tokens=4, heads=16,
             kv_heads=8, d=64, page=32, window=1024, sink=True, mix=7),
        # A short question.
        dict(name="prompt short", op="prompt", act="bf16", batch=1, longest=177, prefix=0, heads=32, kv_heads=8, d=128,
             window=0, sink=False, mix=0),
        # A packed batch of prompts.
        dict(name="prompt packed", op="prompt", act="bf16", batch=8, longest=4096, prefix=0, heads=32, kv_heads=8,
             d=128, window=0, sink=False, mix=8),
        # One long prompt, one GPU's heads of a layer that eight share.
        dict(name="prompt 16k", op="prompt", act="bf16", batch=1, longest=16384, prefix=0, heads=8, kv_heads=1, d=128,
             window=0, sink=False, mix=0),
        # Later chunks of prompts in a sliding-window layer with sinks, narrow heads.
        dict(name="prompt window", op="prompt", act="f16", batch=6, longest=2500, prefix=1500, heads=16, kv_heads=4,
             d=64, window=1024, sink=True, mix=9),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "prompt"])
    d = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 8])
    act = rng.choice(["bf16", "bf16", "f16"])
    mix = rng.randrange(1, 1 << 20)
    if op == "append":
        batch = _log(rng, 1, 64)
        longest = 1 if rng.random() < 0.4 else _log(rng, 2, min(8192, 40000 // batch))
        return dict(op=op, act=act, kv=rng.choice(["act", "act", "fp8"]), batch=batch, longest=longest,
                    base=rng.choice([0, _log(rng, 1, 200000)]), heads=heads, kv_heads=kv_heads, d=d,
                    r=rng.choice([d // 2, d]), page=rng.choice([16, 32, 64, 128]), mix=mix)
    if op == "decode":
        longest = _log(rng, 1, 131072)
        batch = _log(rng, 1, max(1, min(64, (4 * 131072 * 8 * 128) // (longest * kv_heads * d))))
        return dict(op=op, act=act, kv=rng.choice(["act", "act", "fp8"]), batch=batch, longest=longest,
                    tokens=rng.choice([1, 1, 1, 2, 4]), heads=heads, kv_heads=kv_heads, d=d,
                    page=rng.choice([16, 32, 64, 128]), window=rng.choice([0, 0, _log(rng, 16, 8192)]),
                    sink=rng.random() < 0.4, mix=mix)
    longest = _log(rng, 1, 8192)
    batch = _log(rng, 1, max(1, min(32, (8 * 16384 * 16384) // (2 * longest * longest * heads))))
    return dict(op=op, act=act, batch=batch, longest=longest, prefix=rng.choice([0, 0, _log(rng, 1, 2 * longest)]),
                heads=heads, kv_heads=kv_heads, d=d, window=rng.choice([0, 0, _log(rng, 16, 4096)]),
                sink=rng.random() < 0.4, mix=mix)


def _lengths(case):
    """One sequence has the longest length, the others spread below it over
    their logarithm; mix 0: all are that long."""
    n, top = case["batch"], case["longest"]
    if case["mix"] == 0 or top == 1:
        return [top] * n
    rng = random.Random(case["mix"])
    return [top] + [_log(rng, max(1, top // 16), top) for _ in range(n - 1)]


def _prefixes(case):
    """Keys that stand before each prompt's queries (earlier chunks)."""
    rng = random.Random(case["mix"] + 1)
    return [rng.randrange(case["prefix"] + 1) if case["prefix"] else 0 for _ in range(case["batch"])]


def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


# ---- inputs --------------------------------------------------------------------

def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _quantise(x):
    """Rows of x as E4M3 codes and fp32 scales."""
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return (x / scale[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def _cache(gen, case, n_pages, act):
    """A pool of pages with what earlier tokens left in it."""
    shape = (n_pages, case["kv_heads"], case["page"], case["d"])
    out = {}
    for name in ("k", "v"):
        if case["kv"] == "act":
            out[name + "_cache"] = torch.randn(shape, generator=gen, device="cuda", dtype=act)
            out[name + "_scale"] = None
        else:
            out[name + "_cache"] = torch.empty(shape, device="cuda", dtype=torch.float8_e4m3fn)
            out[name + "_scale"] = torch.empty(shape[:3], device="cuda")
            for at in range(0, n_pages, 4096):
                x = torch.randn((min(4096, n_pages - at),) + shape[1:], generator=gen, device="cuda")
                out[name + "_cache"][at:at + 4096], out[name + "_scale"][at:at + 4096] = _quantise(x)
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    act = _ACT[case["act"]]
    lens = _lengths(case)
    n_heads, n_kv, d = case["heads"], case["kv_heads"], case["d"]
    s = {"op": case["op"], "act": act, "groups": n_heads // n_kv, "scale": d ** -0.5}

    def rows(n, heads, gain=1.0):
        return torch.randn((n, heads, d), generator=gen, device="cuda").mul_(gain).to(act)

    if case["op"] == "append":
        page, base = case["page"], case["base"]
        rng = random.Random(case["mix"] + 2)
        pos0 = [base + rng.randrange(base // 4 + 1) for _ in lens]
        n = sum(lens)
        s.update(q=rows(n, n_heads), k=rows(n, n_kv), v=rows(n, n_kv), r=case["r"], page=page,
                 cu=_ints(_starts(lens)), pos0=_ints(pos0))
        # the pool holds the pages that these tokens reach, in any order
        width = max((p + t - 1) // page + 1 for p, t in zip(pos0, lens))
        table = np.full((len(lens), width), -1, dtype=np.int32)
        reached = [(b, c) for b, (p, t) in enumerate(zip(pos0, lens)) for c in range(p // page, (p + t - 1) // page + 1)]
        for i, at in enumerate(np.random.RandomState(seed & 0x7fffffff).permutation(len(reached))):
            table[reached[i]] = at
        s.update(_cache(gen, case, len(reached), act), table=torch.from_numpy(table).cuda())
        s.update(q_out=torch.empty_like(s["q"]), k_out=torch.empty_like(s["k"]))
    elif case["op"] == "decode":
        page, t = case["page"], case["tokens"]
        lens = [max(n, t) for n in lens]
        used = [-(-n // page) for n in lens]
        table = np.full((len(lens), max(used)), -1, dtype=np.int32)
        order, at = np.random.RandomState(seed & 0x7fffffff).permutation(sum(used)), 0
        for b, u in enumerate(used):
            table[b, :u] = order[at:at + u]
            at += u
        s.update(_cache(gen, case, sum(used), act), table=torch.from_numpy(table).cuda(), lens=_ints(lens),
                 n_max=max(lens), tokens=t, page=page, window=case["window"], q=rows(len(lens) * t, n_heads, 1.5))
        s["sink"] = torch.randn(n_heads, generator=gen, device="cuda") if case["sink"] else None
        s["out"] = torch.empty_like(s["q"])
    else:
        keys = [n + p for n, p in zip(lens, _prefixes(case))]
        s.update(q=rows(sum(lens), n_heads, 1.5), k=rows(sum(keys), n_kv), v=rows(sum(keys), n_kv),
                 cu_q=_ints(_starts(lens)), cu_k=_ints(_starts(keys)), most_q=max(lens), most_k=max(keys),
                 window=case["window"])
        s["sink"] = torch.randn(n_heads, generator=gen, device="cuda") if case["sink"] else None
        s["out"] = torch.empty_like(s["q"])
    if own:
        import long_context_sparse_gated_b200 as lib
        s["lib"] = lib
        s["params"] = lib.make_gqa_params(
            B=len(lens), n_heads=n_heads, n_kv_heads=n_kv, d=d, r=case.get("r", 0), page=case.get("page", 16),
            window=case.get("window", 0), softmax_scale=s["scale"], rope_theta=_THETA,
            act_fmt=lib.ACT_BF16 if case["act"] == "bf16" else lib.ACT_F16,
            kv_fmt=lib.KV_FP8 if case.get("kv") == "fp8" else lib.KV_ACT)
        if case["op"] != "prompt":
            s["cache"] = lib.make_gqa_cache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        if case["op"] == "decode":
            size = lib.gqa_decode_attn_workspace_bytes(s["params"], s["tokens"], s["n_max"])
            s["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    return s


# ---- the operators in plain form -------------------------------------------------

def _rotated(x, pos, r):
    """The last r dims' pairs turned by pos * theta^(-2j/r), in 32 bits; the
    angles in 64."""
    x = x.float()
    d = x.shape[-1]
    freq = _THETA ** (-2.0 * torch.arange(r // 2, device=x.device, dtype=torch.float64) / r)
    angle = pos.double()[:, None] * freq
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    pairs = x[..., d - r:].unflatten(-1, (r // 2, 2))
    a, b = pairs[..., 0], pairs[..., 1]
    return torch.cat([x[..., :d - r], torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)], -1)


def _append(s):
    n = s["q"].shape[0]
    i = torch.arange(n, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"], i, right=True) - 1
    pos = s["pos0"][b] + i - s["cu"][b]
    page = s["table"][b, (pos // s["page"]).long()].long()
    slot = (pos % s["page"]).long()
    k, v = _rotated(s["k"], pos, s["r"]), s["v"].float()
    s["q_out"].copy_(_rotated(s["q"], pos, s["r"]))
    s["k_out"].copy_(k)
    if s["k_scale"] is None:
        s["k_cache"][page, :, slot] = k.to(s["act"])
        s["v_cache"][page, :, slot] = v.to(s["act"])
    else:
        for name, x in (("k", k), ("v", v)):
            code, scale = _quantise(x)
            s[name + "_cache"].view(torch.uint8)[page, :, slot] = code.view(torch.uint8)
            s[name + "_scale"][page, :, slot] = scale


def _weighted(scores, v, sink):
    """softmax(scores, sink) @ v over the last axis; rows that see nothing give 0.
    Overwrites `scores`; sink [heads] counts in the denominator alone, with
    scores [batch, kv heads, groups, queries, keys]."""
    m = scores.amax(-1, keepdim=True)
    if sink is not None:
        sink = sink.view(scores.shape[1], scores.shape[2])[None, :, :, None, None]
        m = torch.maximum(m, sink)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = scores.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    if sink is not None:
        total = total + (sink - m).exp()
    return (p.flatten(2, 3) @ v).unflatten(2, p.shape[2:4]) / torch.where(total == 0, torch.ones_like(total), total)


def _seen(q_pos, k_pos, window):
    seen = k_pos <= q_pos
    return seen & (k_pos > q_pos - window) if window else seen


def _decode(s):
    n_b, t, page, groups = s["lens"].shape[0], s["tokens"], s["page"], s["groups"]
    pages = s["table"].long().clamp_min(0)

    def gathered(name):  # [batch, kv heads, keys, d]
        x = s[name + "_cache"][pages].float()
        if s[name + "_scale"] is not None:
            x *= s[name + "_scale"][pages][..., None]
        return x.transpose(1, 2).flatten(2, 3)

    q = s["q"].float().view(n_b, t, -1, groups, s["q"].shape[-1]).permute(0, 2, 3, 1, 4)
    scores = (q.flatten(2, 3) @ gathered("k").transpose(-1, -2)).mul_(s["scale"]).unflatten(2, (groups, t))
    k_pos = torch.arange(scores.shape[-1], device="cuda")
    q_pos = s["lens"][:, None] - t + torch.arange(t, device="cuda")
    seen = _seen(q_pos[:, :, None], k_pos, s["window"])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    out = _weighted(scores, gathered("v"), s["sink"])
    s["out"].copy_(out.permute(0, 3, 1, 2, 4).reshape(s["out"].shape))


def _prompt(s):
    groups, cu_q, cu_k = s["groups"], s["cu_q"].long(), s["cu_k"].long()
    n_q, n_k = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    iq, ik = torch.arange(s["most_q"], device="cuda"), torch.arange(s["most_k"], device="cuda")
    at_q = (cu_q[:-1, None] + iq).clamp_max(s["q"].shape[0] - 1)
    at_k = (cu_k[:-1, None] + ik).clamp_max(s["k"].shape[0] - 1)
    q = s["q"][at_q].float().unflatten(2, (-1, groups)).permute(0, 2, 3, 1, 4)
    k, v = (s[x][at_k].float().transpose(1, 2) for x in ("k", "v"))
    scores = (q.flatten(2, 3) @ k.transpose(-1, -2)).mul_(s["scale"]).unflatten(2, (groups, -1))
    q_pos = (n_k - n_q)[:, None] + iq
    seen = _seen(q_pos[:, :, None], ik, s["window"]) & (ik < n_k[:, None])[:, None]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    out = _weighted(scores, v, s["sink"]).permute(0, 3, 1, 2, 4).flatten(2, 3)
    inside = iq < n_q[:, None]
    s["out"][at_q[inside]] = out[inside].to(s["act"])


# ---- one pass ------------------------------------------------------------------

def run(state):
    s, op = state, state["op"]
    if op == "append":
        if own:
            s["lib"].gqa_cache_append(s["params"], s["q"], s["k"], s["v"], s["cu"], s["pos0"], s["cache"], s["table"],
                                      q_out=s["q_out"], k_out=s["k_out"])
        else:
            _append(s)
        return {x: s[x] for x in ("q_out", "k_out", "k_cache", "v_cache", "k_scale", "v_scale")}
    if op == "decode":
        if own:
            s["lib"].gqa_decode_attn(s["params"], s["q"], s["cache"], s["table"], s["lens"], s["tokens"], s["n_max"],
                                     s["out"], s["ws"], sink=s["sink"])
        else:
            _decode(s)
        return s["out"]
    if own:
        s["lib"].gqa_prompt_attn(s["params"], s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["out"], sink=s["sink"])
    else:
        _prompt(s)
    return s["out"]


def _visible(n_q, n_k, window):
    """How many (query, key) pairs a prompt's mask leaves."""
    pos = np.arange(n_k - n_q, n_k, dtype=np.int64)
    pos = pos[pos >= 0]
    return int(np.minimum(pos + 1, window).sum() if window else (pos + 1).sum())


def work(case):
    lens, n_heads, n_kv, d = _lengths(case), case["heads"], case["kv_heads"], case["d"]
    if case["op"] == "append":
        n = sum(lens)
        stored = 2 * n_kv * (d + 4 if case["kv"] == "fp8" else 2 * d)
        # q in and out, k in and out, v in, cache rows out; a turn is 6 operations a pair
        return {"bytes": n * (4 * n_heads * d + 4 * n_kv * d + 2 * n_kv * d + stored),
                "flops": n * (n_heads + n_kv) * case["r"] * 3}
    if case["op"] == "decode":
        t, window = case["tokens"], case["window"]
        lens = [max(n, t) for n in lens]
        keys = sum(min(n, window + t - 1) if window else n for n in lens)
        pairs = sum(_visible(t, n, window) for n in lens)
        row = d + 4 if case["kv"] == "fp8" else 2 * d
        return {"bytes": 2 * keys * n_kv * row + 4 * len(lens) * t * n_heads * d, "flops": 4 * pairs * n_heads * d}
    keys = [n + p for n, p in zip(lens, _prefixes(case))]
    pairs = sum(_visible(n, m, case["window"]) for n, m in zip(lens, keys))
    read = [min(m, n + case["window"] - 1) if case["window"] else m for n, m in zip(lens, keys)]
    return {"bytes": 4 * sum(lens) * n_heads * d + 4 * sum(read) * n_kv * d, "flops": 4 * pairs * n_heads * d}


# ---- the definition, in 64 bits ------------------------------------------------

def _turn64(x, pos, r):
    y = x.double().clone()
    d = x.shape[-1]
    j = torch.arange(r // 2, dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.ones_like(j).expand(len(pos), -1), pos.double()[:, None] * torch.exp(-2 * j / r * math.log(_THETA)))
    z = torch.view_as_complex(y[..., d - r:].reshape(*y.shape[:-1], r // 2, 2)) * turn[:, None]
    y[..., d - r:] = torch.view_as_real(z).flatten(-2)
    return y


def _attend64(q, k, v, q_pos, k_pos, window, sink, scale):
    """One head group: q [g, n, d], k and v [m, d], sink [g] or None."""
    z = torch.einsum("gnd,md->gnm", q, k) * scale
    hidden = k_pos[None, :] > q_pos[:, None]
    if window:
        hidden |= k_pos[None, :] <= q_pos[:, None] - window
    z[hidden.expand_as(z)] = -math.inf
    top = z.amax(-1) if sink is None else torch.maximum(z.amax(-1), sink[:, None])
    top[top == -math.inf] = 0
    z = torch.exp(z - top[..., None])
    below = z.sum(-1)
    if sink is not None:
        below = below + torch.exp(sink[:, None] - top)
    below[below == 0] = 1
    return torch.einsum("gnm,md->gnd", z, v) / below[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    lens = _lengths(case)
    groups, n_kv, d = s["groups"], case["kv_heads"], case["d"]
    sink = s["sink"].double() if s.get("sink") is not None else None
    if case["op"] == "append":
        pos = torch.cat([torch.arange(p, p + n, device="cuda") for p, n in zip(s["pos0"].tolist(), lens)])
        seq = torch.cat([torch.full((n,), b, device="cuda") for b, n in enumerate(lens)])
        k, v = _turn64(s["k"], pos, case["r"]), s["v"].double()
        out = {"q_out": _turn64(s["q"], pos, case["r"]), "k_out": k, "k_scale": None, "v_scale": None}
        at, slot = s["table"].long()[seq, pos // case["page"]], pos % case["page"]
        for name, x in (("k", k), ("v", v)):
            whole = s[name + "_cache"].double()
            if s[name + "_scale"] is not None:
                scale = x.abs().amax(-1) / 448
                scale[scale == 0] = 1
                x = x / scale[..., None]
                scales = s[name + "_scale"].double()
                scales[at, :, slot] = scale
                out[name + "_scale"] = scales
            whole[at, :, slot] = x
            out[name + "_cache"] = whole
        return out
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    if case["op"] == "decode":
        t, page = case["tokens"], case["page"]
        for b, n in enumerate(s["lens"].tolist()):
            pages = s["table"][b, :-(-n // page)].long()
            for h in range(n_kv):
                k, v = (s[x + "_cache"][pages, h].double() for x in ("k", "v"))
                if s["k_scale"] is not None:
                    k, v = k * s["k_scale"][pages, h][..., None].double(), v * s["v_scale"][pages, h][..., None].double()
                mine = slice(h * groups, (h + 1) * groups)
                q = s["q"][b * t:(b + 1) * t, mine].double().transpose(0, 1)
                o = _attend64(q, k.reshape(-1, d)[:n], v.reshape(-1, d)[:n], torch.arange(n - t, n, device="cuda"),
                              torch.arange(n, device="cuda"), case["window"], None if sink is None else sink[mine], s["scale"])
                out[b * t:(b + 1) * t, mine] = o.transpose(0, 1)
        return out
    keys = [n + p for n, p in zip(lens, _prefixes(case))]
    at_q = at_k = 0
    for n, m in zip(lens, keys):
        for h in range(n_kv):
            for g in range(h * groups, (h + 1) * groups):
                o = _attend64(s["q"][at_q:at_q + n, g].double()[None], s["k"][at_k:at_k + m, h].double(),
                              s["v"][at_k:at_k + m, h].double(), torch.arange(m - n, m, device="cuda"),
                              torch.arange(m, device="cuda"), case["window"], None if sink is None else sink[g:g + 1], s["scale"])
                out[at_q:at_q + n, g] = o[0]
        at_q, at_k = at_q + n, at_k + m
    return out
