"""Measured cases of the decode-layer operators: the paged cache's plan, the rotary store into it, attention over it,
the fused norms between blocks, and the routing to experts.

``run`` computes one pass in plain torch operations, or through the library's calls where ``own`` is true.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # One decode step's bookkeeping for a small batch: one new token for each of 8 requests.
        {"name": "plan-decode-8", "op": "plan", "n_req": 8, "tokens": 8, "max_ctx": 4096, "page": 16},
        # A step that mixes prompts and decodes over a thousand requests: most add one token, some a long chunk.
        {"name": "plan-mixed-1000", "op": "plan", "n_req": 1000, "tokens": 131071, "max_ctx": 32768, "page": 16},
        # Decode of 16 sequences: the fp32 rows of the q/k/v projections are rotated and stored.
        {"name": "rope-decode-16", "op": "rope", "tokens": 16, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "axes": 1,
         "interleaved": False, "dtype": "f32", "page": 16},
        # A prompt with images in it: positions of three axes (time, height, width), an odd token count.
        {"name": "rope-prompt-8191", "op": "rope", "tokens": 8191, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "axes": 3, "interleaved": False, "dtype": "f32", "page": 64},
        # Interactive decode of one sequence: latency, all of the GPU on eight kv heads.
        {"name": "attn-decode-1", "op": "attn", "n_req": 1, "new": 1, "ctx": 2047, "hq": 32, "hkv": 8, "d": 128,
         "page": 16, "window": 0},
        # A decode batch of ragged contexts up to about 8k: the cache is the traffic.
        {"name": "attn-decode-64", "op": "attn", "n_req": 64, "new": 64, "ctx": 64 * 4099, "hq": 32, "hkv": 8,
         "d": 128, "page": 16, "window": 0},
        # Chunks of new tokens of uneven length over cached context, a local window, heads of 64 in groups of 5.
        {"name": "attn-chunk-window", "op": "attn", "n_req": 12, "new": 2999, "ctx": 30011, "hq": 20, "hkv": 4,
         "d": 64, "page": 32, "window": 1000},
        # The second half of a long prompt in one chunk: compute.
        {"name": "attn-prompt-8192", "op": "attn", "n_req": 1, "new": 8192, "ctx": 4096, "hq": 32, "hkv": 8,
         "d": 128, "page": 64, "window": 0},
        # Between two projections of one decoded token: fp32 projection output onto the fp32 stream.
        {"name": "norm-decode-1", "op": "norm", "tokens": 1, "dim": 4096, "y": "f32", "stream": "f32", "gate": "row",
         "post": True},
        # The same for a prompt on a bf16 stream, with a gate of its own for each token.
        {"name": "norm-prompt-8192", "op": "norm", "tokens": 8192, "dim": 4096, "y": "bf16", "stream": "bf16",
         "gate": "token", "post": True},
        # The route of one decoded token: 256 experts in 8 groups, sigmoid scores with a balance bias.
        {"name": "route-decode-1", "op": "route", "tokens": 1, "experts": 256, "topk": 8, "groups": 8,
         "topk_group": 4, "score": "sigmoid", "bias": True},
        # The routes of a long prompt: softmax over 256 experts, no groups.
        {"name": "route-prompt-16384", "op": "route", "tokens": 16384, "experts": 256, "topk": 8, "groups": 1,
         "topk_group": 1, "score": "softmax", "bias": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "attn", "attn", "norm", "route"])
    if op == "plan":
        n = _log(rng, 1, 1000)
        return {"op": op, "n_req": n, "tokens": n + _log(rng, 1, 130000), "max_ctx": _log(rng, 16, 32768),
                "page": rng.choice([16, 32, 64, 128])}
    if op == "rope":
        d = rng.choice([64, 96, 128])
        hkv = rng.choice([1, 2, 4, 8])
        return {"op": op, "tokens": _log(rng, 1, 8191), "hq": hkv * rng.choice([1, 2, 3, 4]), "hkv": hkv, "d": d,
                "rot": rng.choice([d, d // 2]), "axes": rng.choice([1, 3]), "interleaved": rng.random() < 0.5,
                "dtype": rng.choice(["f32", "bf16"]), "page": rng.choice([16, 32, 64, 128])}
    if op == "attn":
        d, hkv = rng.choice([64, 96, 128]), rng.choice([1, 2, 4, 8])
        case = {"op": op, "hkv": hkv, "hq": hkv * rng.choice([1, 2, 3, 4, 5, 8]), "d": d,
                "page": rng.choice([16, 32, 64, 128]), "window": rng.choice([0, 0, _log(rng, 100, 4000)])}
        if rng.random() < 0.4:  # decode: one new token each
            n = _log(rng, 1, 64)
            case.update(n_req=n, new=n, ctx=n * _log(rng, 1, 4099))
        else:  # chunks
            n = _log(rng, 1, 16)
            case.update(n_req=n, new=n * _log(rng, 8, max(9, 8192 // (n * n))), ctx=n * _log(rng, 1, 4096 // n))
        while True:
            ctx, new = _lengths(case, 0)
            padded = case["n_req"] * case["hq"] * max(new) * (max(new) + max(ctx))
            if padded <= 32 * 8192 * 12288 and work(case)["flops"] <= 1e12:
                return case
            case["hq"] = case["hkv"] if case["hq"] > case["hkv"] else case["hq"]
            case["new"] = max(case["n_req"], case["new"] // 2)
    if op == "norm":
        return {"op": op, "tokens": _log(rng, 1, 8192), "dim": rng.choice([1000, 1024, 2048, 2880, 4096]),
                "y": rng.choice(["f32", "bf16"]), "stream": rng.choice(["f32", "bf16"]),
                "gate": rng.choice(["none", "row", "token"]), "post": rng.random() < 0.7}
    groups = rng.choice([1, 1, 4, 8])
    return {"op": op, "tokens": _log(rng, 1, 16384), "experts": rng.choice([64, 128, 160, 256]),
            "topk": rng.choice([2, 4, 6, 8]), "groups": groups, "topk_group": max(1, groups // 2),
            "score": rng.choice(["sigmoid", "softmax"]), "bias": rng.random() < 0.5}


def _split(rng, n, total, low):
    """n whole numbers of at least `low` that add up to `total`, uneven."""
    w = [rng.random() + 0.05 for _ in range(n)]
    s, free = sum(w), total - low * n
    parts = [low + int(free * x / s) for x in w]
    parts[0] += total - sum(parts)
    return parts


def _lengths(case, seed):
    """Cached and new tokens of each request: the same lengths for every seed, in another order."""
    rng = random.Random(case["n_req"] * 7919 + case["new"])
    n = case["n_req"]
    pairs = list(zip(_split(rng, n, case["ctx"], 0), _split(rng, n, case["new"], 1)))
    random.Random(seed).shuffle(pairs)
    return [c for c, _ in pairs], [q for _, q in pairs]


def work(case):
    op = case["op"]
    if op == "plan":
        pages = case["tokens"] // case["page"]
        return {"bytes": 16 * case["n_req"] + 8 * pages + 12 * case["tokens"], "flops": 0}
    if op == "rope":
        size = 4 if case["dtype"] == "f32" else 2
        values = case["tokens"] * (case["hq"] + 2 * case["hkv"]) * case["d"]
        return {"bytes": values * (size + 2) + case["tokens"] * 4 * (case["axes"] + 1), "flops": 4 * values}
    if op == "attn":
        ctx, new = _lengths(case, 0)
        w = case["window"] or 1 << 60
        keys = pairs = 0
        for c, n in zip(ctx, new):
            keys += min(c + n, w - 1 + n)
            # positions p = c..c+n-1 see min(p + 1, w) keys
            full = max(0, min(n, w - c))
            pairs += full * c + full * (full + 1) // 2 + (n - full) * (w if full < n else 0)
        rows = case["new"] * case["hq"]
        return {"bytes": rows * (4 * case["d"] + 4) + 4 * keys * case["hkv"] * case["d"],
                "flops": 4 * case["d"] * case["hq"] * pairs}
    if op == "norm":
        size = {"f32": 4, "bf16": 2}
        rows = case["tokens"] * case["dim"]
        gate = {"none": 0, "row": case["dim"], "token": rows}[case["gate"]]
        return {"bytes": rows * (size[case["y"]] + 2 * size[case["stream"]] + 2) + gate * size[case["y"]]
                + 4 * case["dim"] * (1 + case["post"]), "flops": 10 * rows}
    return {"bytes": case["tokens"] * (4 * case["experts"] + 8 * case["topk"]),
            "flops": 6 * case["tokens"] * case["experts"]}


# ---- inputs ------------------------------------------------------------------

def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _type(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = random.Random(seed)

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)

    s = dict(case)
    op = case["op"]
    if op == "plan":
        n, page = case["n_req"], case["page"]
        ctx = [rng.randrange(case["max_ctx"]) if rng.random() < 0.9 else 0 for _ in range(n)]
        if case["tokens"] == n:
            new = [1] * n
        else:  # a tenth of the requests bring a chunk, the others decode one token or are idle
            new = [0 if rng.random() < 0.05 else 1 for _ in range(n)]
            chunk = [r for r in range(n) if r % 10 == 0]
            for r, extra in zip(chunk, _split(rng, len(chunk), case["tokens"] - sum(new), 0)):
                new[r] += extra
        chunks = -(-n // 10)  # the longest is at most 21 / (20 + chunks) of the tokens (see _split)
        ld = (case["max_ctx"] + case["tokens"] * 21 // (20 + chunks) + chunks) // page + 3
        used = sum(-(-c // page) for c in ctx)
        pool = used + case["tokens"] // page + n + 100
        perm = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
        have = torch.tensor([-(-c // page) for c in ctx], device=DEV)
        first = torch.cumsum(have, 0) - have
        col = torch.arange(ld, device=DEV)
        table = torch.where(col < have[:, None], perm[(first[:, None] + col).clamp(max=pool - 1)],
                            torch.full((), -1, dtype=torch.int32, device=DEV))
        s.update(ctx=_i32(ctx), new=_i32(new), table=table.contiguous(), free=perm[used:].contiguous(),
                 head=_i32([rng.randrange(50)]))
    elif op == "rope":
        t, hq, hkv, d, page = case["tokens"], case["hq"], case["hkv"], case["d"], case["page"]
        dtype = _type(case["dtype"])
        n_pages = -(-t // page) + 7
        s["q"] = normal(t, hq, d, dtype=dtype)
        s["kv"] = normal(t, 2, hkv, d, dtype=dtype)  # one projection writes k and v side by side
        s["k_cache"] = normal(n_pages, hkv, page, d, dtype=torch.bfloat16)
        s["v_cache"] = normal(n_pages, hkv, page, d, dtype=torch.bfloat16)
        s["slots"] = torch.randperm(n_pages * page, generator=g, device=DEV)[:t].to(torch.int32)
        start = rng.randrange(20000)
        pos = torch.arange(start, start + t, device=DEV, dtype=torch.int32)
        if case["axes"] == 3:  # frames of 24 x 16 patches
            pos = torch.stack([pos // 384, pos % 384 // 16, pos % 16])
        s["pos"] = pos.reshape(case["axes"], t).contiguous()
        half = case["rot"] // 2
        s["inv_freq"] = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float32) / half)
        s["sections"] = (half,) if case["axes"] == 1 else (half // 4, (half - half // 4) // 2,
                                                           half - half // 4 - (half - half // 4) // 2)
        axis = [a for a, c in enumerate(s["sections"]) for _ in range(c)]
        s["axis"] = torch.tensor(axis, device=DEV)
    elif op == "attn":
        ctx, new = _lengths(case, seed)
        page, hkv, d = case["page"], case["hkv"], case["d"]
        seq = [c + q for c, q in zip(ctx, new)]
        pages = [-(-x // page) for x in seq]
        n_pages, ld = sum(pages) + 5, max(pages) + 2
        perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
        count = torch.tensor(pages, device=DEV)
        first = torch.cumsum(count, 0) - count
        col = torch.arange(ld, device=DEV)
        s["table"] = torch.where(col < count[:, None], perm[(first[:, None] + col).clamp(max=n_pages - 1)],
                                 torch.zeros((), dtype=torch.int32, device=DEV)).contiguous()
        s["q"] = normal(case["new"], case["hq"], d, dtype=torch.bfloat16, std=1.5)
        s["k_cache"] = normal(n_pages, hkv, page, d, dtype=torch.bfloat16)
        s["v_cache"] = normal(n_pages, hkv, page, d, dtype=torch.bfloat16)
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        s["cu_q"], s["seq_lens"] = _i32(cu), _i32(seq)
        s["max_new"], s["max_seq"], s["scale"] = max(new), max(seq), 1.0 / math.sqrt(d)
        s["lens"] = list(zip(cu, new, seq))
    elif op == "norm":
        t, dim = case["tokens"], case["dim"]
        y = _type(case["y"])
        s["y_rows"] = normal(t, dim, dtype=y, std=3.0)
        s["residual"] = normal(t, dim, dtype=_type(case["stream"]), std=2.0)
        s["gates"] = {"none": lambda: None, "row": lambda: normal(dim, dtype=y, std=0.5),
                      "token": lambda: normal(t, dim, dtype=y, std=0.5)}[case["gate"]]()
        s["pre_w"] = 1.0 + normal(dim, std=0.1)
        s["post_w"] = 1.0 + normal(dim, std=0.1) if case["post"] else None
        s["eps"], s["alpha"] = 1e-6, 0.22
    else:
        s["logits"] = normal(case["tokens"], case["experts"], std=1.5)
        s["b"] = normal(case["experts"], std=0.1) if case["bias"] else None
        s["factor"] = 2.5 if case["score"] == "sigmoid" else 1.0
    return s


# ---- one pass ----------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _plain_plan(s):
    page, tokens = s["page"], s["tokens"]
    ctx, new, table, free = s["ctx"].long(), s["new"].long(), s["table"], s["free"]
    seq = ctx + new
    have, total = (ctx + page - 1) // page, (seq + page - 1) // page
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(new, 0)])
    need = total - have
    before = torch.cumsum(need, 0) - need
    col = torch.arange(table.shape[1], device=DEV)
    fresh = (col >= have[:, None]) & (col < total[:, None])
    at = s["head"].long() + before[:, None] + col - have[:, None]
    table.copy_(torch.where(fresh, free[at.clamp(0, free.numel() - 1)], table))
    t = torch.arange(tokens, device=DEV)
    req = torch.searchsorted(cu, t, right=True) - 1
    pos = ctx[req] + t - cu[req]
    slot = table[req, pos // page].long() * page + pos % page
    i32 = torch.int32
    return {"block_table": table, "cu_q": cu.to(i32), "seq_lens": seq.to(i32), "positions": pos.to(i32),
            "token_req": req.to(i32), "slots": slot.to(i32), "free_head": (s["head"] + need.sum()).to(i32)}


def _own_plan(s):
    import mmvq_q2_gb300 as lib
    p = lib.kv_page_plan(s["ctx"], s["new"], s["page"], s["free"], s["table"], s["tokens"], free_head=s["head"])
    return {"block_table": s["table"], "cu_q": p.cu_q, "seq_lens": p.seq_lens, "positions": p.positions,
            "token_req": p.token_req, "slots": p.slot_map, "free_head": p.free_head}


def _rotate(x, cos, sin, interleaved):
    half = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    rest = x[..., 2 * half:]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, rest], dim=-1)


def _plain_rope(s):
    angle = s["pos"].float()[s["axis"]].t() * s["inv_freq"]
    cos, sin = torch.cos(angle), torch.sin(angle)
    k, v = s["kv"][:, 0].float(), s["kv"][:, 1]
    q = _rotate(s["q"].float(), cos, sin, s["interleaved"]).bfloat16()
    page, off = s["slots"].long() // s["page"], s["slots"].long() % s["page"]
    s["k_cache"][page, :, off] = _rotate(k, cos, sin, s["interleaved"]).bfloat16()
    s["v_cache"][page, :, off] = v.bfloat16()
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_rope(s):
    import mmvq_q2_gb300 as lib
    q = lib.kv_rope_store(s["q"], s["kv"][:, 0], s["kv"][:, 1], s["pos"], s["inv_freq"], s["slots"], s["k_cache"],
                          s["v_cache"], sections=s["sections"], interleaved=s["interleaved"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attn(s):
    q, page, hkv, d = s["q"], s["page"], s["hkv"], s["d"]
    tokens, hq = q.shape[:2]
    cu, seq = s["cu_q"].long(), s["seq_lens"].long()
    n, rows = seq.numel(), s["max_new"]
    new = cu[1:] - cu[:-1]
    i, j = torch.arange(rows, device=DEV), torch.arange(s["max_seq"], device=DEV)
    block = s["table"].long()[:, j // page]
    there = (j < seq[:, None])[:, None, :, None]
    off = (j % page).expand(n, -1)
    k = s["k_cache"][block, :, off].float().transpose(1, 2)
    v = s["v_cache"][block, :, off].float().transpose(1, 2).masked_fill(~there, 0.0)
    at = (cu[:-1, None] + i).clamp(max=tokens - 1)
    x = q[at].float().view(n, rows, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    score = torch.matmul(x.reshape(n, hkv, -1, d), k.transpose(2, 3)).mul_(s["scale"])
    score = score.view(n, hkv, hq // hkv, rows, -1)
    p = (seq - new)[:, None] + i
    seen = (j <= p[..., None]) & (j > p[..., None] - (s["window"] or 1 << 30))
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    o = torch.matmul(score.view(n, hkv, -1, score.shape[-1]), v).view(n, hkv, hq // hkv, rows, d) / total
    lse = (top + torch.log(total))[..., 0]
    t = torch.arange(tokens, device=DEV)
    r = torch.searchsorted(cu, t, right=True) - 1
    w = t - cu[r]
    return {"out": o[r, :, :, w].reshape(tokens, hq, d).bfloat16(), "lse": lse[r, :, :, w].reshape(tokens, hq)}


def _own_attn(s):
    import mmvq_q2_gb300 as lib
    out, lse = lib.kv_attention_bf16(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu_q"], s["seq_lens"],
                                     scale=s["scale"], window=s["window"], want_lse=True)
    return {"out": out, "lse": lse}


def _plain_norm(s):
    u = s["y_rows"].float()
    if s["post_w"] is not None:
        u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + s["eps"]) * s["post_w"]
    if s["gates"] is not None:
        u = u * s["gates"].float()
    h = s["residual"].float() + s["alpha"] * u
    n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + s["eps"]) * s["pre_w"]
    return {"stream": h.to(s["residual"].dtype), "normed": n.bfloat16()}


def _own_norm(s):
    import mmvq_q2_gb300 as lib
    h, n = lib.norm_gate_residual(s["residual"], s["pre_w"], s["eps"], y=s["y_rows"], post_w=s["post_w"],
                                  gate=s["gates"], alpha=s["alpha"])
    return {"stream": h, "normed": n}


def _plain_route(s):
    x = s["logits"]
    if s["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        # the sum in 64 bits, so that no choice depends on the order of its terms
        e = torch.exp(x - x.amax(-1, keepdim=True))
        score = e / e.double().sum(-1, keepdim=True).float()
    c = score if s["b"] is None else score + s["b"]
    if s["groups"] > 1:
        parts = torch.sort(c.view(c.shape[0], s["groups"], -1), dim=-1, descending=True, stable=True)[0]
        rank = torch.sort(parts[..., 0] + parts[..., 1], dim=-1, descending=True, stable=True)[1]
        kept = torch.zeros(rank.shape, dtype=torch.bool, device=DEV).scatter_(1, rank[:, :s["topk_group"]], True)
        c = c.masked_fill(~kept.repeat_interleave(s["experts"] // s["groups"], dim=1), -math.inf)
    ids = torch.sort(c, dim=-1, descending=True, stable=True)[1][:, :s["topk"]]
    w = score.gather(1, ids)
    return {"ids": ids.to(torch.int32), "weights": w / (w.sum(-1, keepdim=True) + 1e-20) * s["factor"]}


def _own_route(s):
    import mmvq_q2_gb300 as lib
    ids, w = lib.moe_route_topk(s["logits"], s["topk"], bias=s["b"], score=s["score"], n_group=s["groups"],
                                topk_group=s["topk_group"], renorm=True, scale=s["factor"])
    return {"ids": ids, "weights": w}


_plain = {"plan": _plain_plan, "rope": _plain_rope, "attn": _plain_attn, "norm": _plain_norm, "route": _plain_route}
_own = {"plan": _own_plan, "rope": _own_rope, "attn": _own_attn, "norm": _own_norm, "route": _own_route}


# ---- 64 bits -----------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": lambda s: None, "rope": _exact_rope, "attn": _exact_attn, "norm": _exact_norm,
            "route": _exact_route}[case["op"]](s)


def _exact_rope(s):
    t, half = s["pos"].shape[1], s["rot"] // 2

    def turn(x):
        # pairs as complex numbers times e^(i angle)
        x = x.double().cpu()
        ang = torch.stack([s["pos"][a].double().cpu() for a in s["axis"].tolist()], 1) * s["inv_freq"].double().cpu()
        w = torch.polar(torch.ones_like(ang), ang)[:, None]
        first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if s["interleaved"] else \
            (slice(0, half), slice(half, 2 * half))
        z = torch.complex(x[..., first], x[..., second]) * w
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
        return x

    k_cache, v_cache = s["k_cache"].double().cpu(), s["v_cache"].double().cpu()
    page, off = (s["slots"].cpu().long() // s["page"]), (s["slots"].cpu().long() % s["page"])
    k_cache[page, :, off] = turn(s["kv"][:, 0])
    v_cache[page, :, off] = s["kv"][:, 1].double().cpu()
    return {"q": turn(s["q"]), "k_cache": k_cache, "v_cache": v_cache}


def _exact_attn(s):
    q, d, page = s["q"], s["d"], s["page"]
    group = s["hq"] // s["hkv"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=DEV)
    for r, (at, new, seq) in enumerate(s["lens"]):
        blocks = s["table"][r, : -(-seq // page)].long()
        for h in range(s["hkv"]):
            k = s["k_cache"][blocks, h].reshape(-1, d)[:seq].double()
            v = s["v_cache"][blocks, h].reshape(-1, d)[:seq].double()
            for i in range(0, new, 1024):
                rows = torch.arange(i, min(new, i + 1024), device=DEV)
                back = (seq - new + rows)[:, None] - torch.arange(seq, device=DEV)
                hide = (back < 0) | ((back >= s["window"]) if s["window"] else False)
                for head in range(h * group, (h + 1) * group):
                    z = (q[at + rows, head].double() @ k.t()) * s["scale"]
                    z = torch.where(hide, -math.inf, z)
                    lse[at + rows, head] = torch.logsumexp(z, -1)
                    out[at + rows, head] = torch.softmax(z, -1) @ v
    return {"out": out, "lse": lse}


def _exact_norm(s):
    def norm(x, w):
        return x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt() * w.double()

    u = s["y_rows"].double()
    if s["post_w"] is not None:
        u = norm(u, s["post_w"])
    if s["gates"] is not None:
        u = s["gates"].double() * u
    h = u * s["alpha"] + s["residual"].double()
    return {"stream": h, "normed": norm(h, s["pre_w"])}


def _exact_route(s):
    x = s["logits"].double()
    score = torch.sigmoid(x) if s["score"] == "sigmoid" else torch.softmax(x, -1)
    c = score if s["b"] is None else score + s["b"].double()
    if s["groups"] > 1:
        group = torch.arange(s["experts"], device=DEV) // (s["experts"] // s["groups"])
        best = torch.stack([c[:, group == i].topk(2, -1)[0].sum(-1) for i in range(s["groups"])], 1)
        floor = best.topk(s["topk_group"], -1)[0][:, -1:]
        c = torch.where((best >= floor)[:, group], c, -math.inf)
    ids = c.topk(s["topk"], -1)[1]
    w = torch.gather(score, 1, ids)
    return {"ids": None, "weights": w / w.sum(-1, keepdim=True) * s["factor"]}
