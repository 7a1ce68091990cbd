"""Measured cases of the products with 8-bit floating-point weights: rows and blocks into e4m3 with a scale for each
block of 128, the same fused behind SwiGLU, the matrix product of such operands, and a whole mixture-of-experts layer
for a few tokens.

``run`` computes one pass in plain torch operations, or through the library's calls where ``own`` is true.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BLOCK = 128
TOP = 448.0  # the largest e4m3 value


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # Activations of a small decode batch before a projection: latency.
        {"name": "quantize-decode-8", "op": "quantize", "rows": 8, "k": 4096, "dtype": "bf16", "block_rows": 1},
        # The same for a prompt, an odd number of tokens.
        {"name": "quantize-prompt-8191", "op": "quantize", "rows": 8191, "k": 4096, "dtype": "bf16", "block_rows": 1},
        # A weight matrix at load time, a scale for each 128 x 128 values.
        {"name": "quantize-weights-20480", "op": "quantize", "rows": 20480, "k": 2048, "dtype": "f32",
         "block_rows": 128},
        # Between the two products of a dense feed-forward block, one decoded token for each of 8 sequences.
        {"name": "swiglu-decode-8", "op": "swiglu", "rows": 8, "n": 2048, "dtype": "f32"},
        # The same for a prompt on bf16 products.
        {"name": "swiglu-prompt-8191", "op": "swiglu", "rows": 8191, "n": 2048, "dtype": "bf16"},
        # An output projection for one decoded token.
        {"name": "gemm-decode-1", "op": "gemm", "m": 1, "n": 4096, "k": 4096, "out": "f32"},
        # A decode batch against a large matrix: the weights are the traffic.
        {"name": "gemm-decode-16", "op": "gemm", "m": 16, "n": 16384, "k": 16384, "out": "f32"},
        # A chunk of a prompt, no size a multiple of a tile's, the last block of each row short.
        {"name": "gemm-chunk-203", "op": "gemm", "m": 203, "n": 5000, "k": 4112, "out": "bf16"},
        # A long prompt: compute.
        {"name": "gemm-prompt-8191", "op": "gemm", "m": 8191, "n": 8192, "k": 4096, "out": "bf16"},
        # The routed experts of one decoded token.
        {"name": "moe-decode-1", "op": "moe", "m": 1, "pad": 0, "experts": 256, "topk": 8, "dim": 4096, "inter": 2048,
         "out": "bf16"},
        # Of a decode batch, most experts with one token.
        {"name": "moe-decode-8", "op": "moe", "m": 8, "pad": 0, "experts": 256, "topk": 8, "dim": 4096, "inter": 2048,
         "out": "bf16"},
        # Of a captured step for 32 tokens that 29 fill, experts with one to five tokens.
        {"name": "moe-decode-32", "op": "moe", "m": 32, "pad": 3, "experts": 256, "topk": 8, "dim": 4096,
         "inter": 2048, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "swiglu", "gemm", "gemm", "gemm", "moe", "moe"])
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 8191), "k": 16 * _log(rng, 4, 256), "dtype": rng.choice(["f32", "bf16"]),
                "block_rows": rng.choice([1, 1, 128])}
    if op == "swiglu":
        return {"op": op, "rows": _log(rng, 1, 8191), "n": 16 * _log(rng, 4, 128), "dtype": rng.choice(["f32", "bf16"])}
    if op == "gemm":
        case = {"op": op, "m": _log(rng, 1, 8191), "n": _log(rng, 64, 16384), "k": 16 * _log(rng, 8, 1024),
                "out": rng.choice(["f32", "bf16"])}
        if rng.random() < 0.5:  # whole blocks, as most models have
            case["n"], case["k"] = -(-case["n"] // BLOCK) * BLOCK, -(-case["k"] // BLOCK) * BLOCK
        while case["m"] * case["n"] * case["k"] > 8191 * 8192 * 4096:
            case["m"] = -(-case["m"] // 2)
        return case
    experts = rng.choice([8, 16, 64, 128, 256])
    case = {"op": op, "m": _log(rng, 1, 32), "pad": 0, "experts": experts, "topk": rng.choice([1, 2, 4, 6, 8]),
            "dim": rng.choice([1024, 2048, 2880, 4096]), "inter": rng.choice([512, 768, 1408, 1520, 2048]),
            "out": "bf16"}
    if rng.random() < 0.3:
        case["pad"] = rng.randrange(case["m"])
    return case


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    op = case["op"]
    if op == "quantize":
        rows, k = case["rows"], case["k"]
        scales = -(-rows // case["block_rows"]) * _blocks(k)
        return {"bytes": rows * k * ((4 if case["dtype"] == "f32" else 2) + 1) + 4 * scales, "flops": 3 * rows * k}
    if op == "swiglu":
        rows, n = case["rows"], case["n"]
        return {"bytes": rows * n * (2 * (4 if case["dtype"] == "f32" else 2) + 1) + 4 * rows * _blocks(n),
                "flops": 10 * rows * n}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * k + 4 * (m + _blocks(n)) * _blocks(k) + m * n * (4 if case["out"] == "f32" else 2),
                "flops": 2 * m * n * k}
    m, e, d, i = case["m"] - case["pad"], case["experts"], case["dim"], case["inter"]
    used = e * (1.0 - (1.0 - case["topk"] / e) ** m)  # experts with a token, on average
    size = 3 * d * i + 4 * 3 * _blocks(d) * _blocks(i)
    return {"bytes": used * size + m * (2 * d + 8 * case["topk"]) + case["m"] * 2 * d,
            "flops": 6 * m * case["topk"] * d * i}


# ---- inputs ------------------------------------------------------------------

def _type(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0):
        return torch.randn(shape, generator=g, device=DEV).mul_(std).to(dtype)

    def weights(*shape):
        """e4m3 values that fill the type's range, as a block's quantiser leaves them, and the blocks' scales."""
        w = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
        flat = w.view(-1)
        for at in range(0, flat.numel(), 1 << 28):
            n = min(1 << 28, flat.numel() - at)
            flat[at:at + n] = normal(n, std=100.0).clamp_(-TOP, TOP).to(torch.float8_e4m3fn)
        scales = torch.exp(normal(*shape[:-2], _blocks(shape[-2]), _blocks(shape[-1]), std=0.2))
        return w, scales / (100.0 * math.sqrt(shape[-1]))

    s = dict(case)
    op = case["op"]
    if op == "quantize":
        # tokens, or rows of a matrix, of different size
        s["x"] = (normal(case["rows"], case["k"]) * torch.exp(normal(case["rows"], 1))).to(_type(case["dtype"]))
    elif op == "swiglu":
        s["gate_up"] = normal(case["rows"], 2 * case["n"], std=1.5, dtype=_type(case["dtype"]))
    elif op == "gemm":
        s["x"] = normal(case["m"], case["k"], std=100.0).clamp_(-TOP, TOP).to(torch.float8_e4m3fn)
        s["x_scales"] = torch.exp(normal(case["m"], _blocks(case["k"]), std=0.5)) / 100.0
        s["w"], s["w_scales"] = weights(case["n"], case["k"])
    else:
        m, e, d, i = case["m"], case["experts"], case["dim"], case["inter"]
        s["x"] = normal(m, d, dtype=torch.bfloat16)
        logits = normal(m, e)
        top, ids = torch.sort(logits, dim=-1, descending=True)
        s["ids"] = ids[:, :case["topk"]].to(torch.int32).contiguous()
        s["route_w"] = torch.softmax(top[:, :case["topk"]], -1).contiguous()
        if case["pad"]:
            s["ids"][m - case["pad"]:] = -1
        s["gate_up"], s["gate_up_scales"] = weights(e, 2, i, d)
        s["down"], s["down_scales"] = weights(e, d, i)
    return s


# ---- one pass ----------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _spread(scales, rows, cols):
    """The scale of each value from those of the 128 x 128 blocks."""
    return scales.repeat_interleave(BLOCK, -2)[..., :rows, :].repeat_interleave(BLOCK, -1)[..., :cols]


def _encode(x, block_rows):
    """fp32 rows -> e4m3 values and scales."""
    rows, k = x.shape
    more, wide = -rows % block_rows, -k % BLOCK
    whole = torch.nn.functional.pad(x, (0, wide, 0, more)) if more or wide else x
    blocks = whole.view((rows + more) // block_rows, block_rows, (k + wide) // BLOCK, BLOCK)
    top = blocks.abs().amax((1, 3)).clamp(min=TOP * 2.0 ** -120)
    values = (blocks * (TOP / top)[:, None, :, None]).to(torch.float8_e4m3fn)
    values = values.view(rows + more, k + wide)[:rows, :k].contiguous()
    return {"values": values, "scales": top / TOP}


def _plain_quantize(s):
    return _encode(s["x"].float(), s["block_rows"])


def _own_quantize(s):
    import mmvq_q2_gb300 as lib
    values, scales = lib.fp8_quantize(s["x"], block_rows=s["block_rows"])
    return {"values": values, "scales": scales}


def _plain_swiglu(s):
    gate, up = s["gate_up"].float().chunk(2, -1)
    return _encode(gate / (1.0 + torch.exp(-gate)) * up, 1)


def _own_swiglu(s):
    import mmvq_q2_gb300 as lib
    values, scales = lib.swiglu_fp8_rows(s["gate_up"])
    return {"values": values, "scales": scales}


def _plain_gemm(s):
    x = s["x"].float() * s["x_scales"].repeat_interleave(BLOCK, -1)[:, :s["k"]]
    w = s["w"].float() * _spread(s["w_scales"], s["n"], s["k"])
    return {"y": torch.matmul(x, w.t()).to(_type(s["out"]))}


def _own_gemm(s):
    import mmvq_q2_gb300 as lib
    return {"y": lib.fp8_gemm(s["x"], s["x_scales"], s["w"], s["w_scales"], out_dtype=_type(s["out"]))}


def _plain_moe(s):
    m, k, d, i = s["m"], s["topk"], s["dim"], s["inter"]
    there = s["ids"] >= 0
    ids = s["ids"].clamp(min=0).long().view(-1)

    def of(weights, scales, rows, cols):
        picked = weights.view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()
        return picked.mul_(_spread(scales[ids], rows, cols))

    x = s["x"].float().repeat_interleave(k, 0)
    both = torch.matmul(of(s["gate_up"], s["gate_up_scales"], i, d), x[:, None, :, None])[..., 0]
    gate, up = both[:, 0], both[:, 1]
    h = gate / (1.0 + torch.exp(-gate)) * up
    y = torch.matmul(of(s["down"], s["down_scales"], d, i), h[..., None]).view(m, k, d)
    return {"y": (y * torch.where(there, s["route_w"], 0.0)[..., None]).sum(1).to(_type(s["out"]))}


def _own_moe(s):
    import mmvq_q2_gb300 as lib
    return {"y": lib.fp8_moe(s["x"], s["ids"], s["route_w"], s["gate_up"], s["gate_up_scales"], s["down"],
                             s["down_scales"], out_dtype=_type(s["out"]))}


_plain = {"quantize": _plain_quantize, "swiglu": _plain_swiglu, "gemm": _plain_gemm, "moe": _plain_moe}
_own = {"quantize": _own_quantize, "swiglu": _own_swiglu, "gemm": _own_gemm, "moe": _own_moe}


# ---- 64 bits -----------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"quantize": _exact_quantize, "swiglu": _exact_swiglu, "gemm": _exact_gemm,
            "moe": _exact_moe}[case["op"]](s)


def _to_e4m3(v):
    """The nearest e4m3 value, ties to even: steps of an eighth of a value's power of two, 2^-9 at the least."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(v / step) * step


def _exact_encode(x, block_rows):
    values = torch.empty_like(x)
    scales = torch.empty((-(-x.shape[0] // block_rows), _blocks(x.shape[1])), dtype=torch.float64, device=DEV)
    for c in range(scales.shape[1]):
        part = x[:, c * BLOCK:(c + 1) * BLOCK]
        high = part.abs().max(1)[0]
        if block_rows > 1:
            high = torch.stack([h.max() for h in high.split(block_rows)])
        scales[:, c] = torch.clamp(high, min=TOP * 2.0 ** -120) / TOP
        row_scale = scales[:, c].repeat_interleave(block_rows)[:x.shape[0]]
        values[:, c * BLOCK:(c + 1) * BLOCK] = _to_e4m3(part / row_scale[:, None])
    return {"values": values, "scales": scales}


def _exact_quantize(s):
    return _exact_encode(s["x"].double(), s["block_rows"])


def _exact_swiglu(s):
    n = s["n"]
    z = s["gate_up"].double()
    return _exact_encode(torch.sigmoid(z[:, :n]) * z[:, :n] * z[:, n:], 1)


def _block_product(x, w, w_scales):
    """x [t, k] (64 bits, scaled) times the block-scaled w^T, one column of blocks after another."""
    y = torch.zeros((x.shape[0], w.shape[0]), dtype=torch.float64, device=DEV)
    for c in range(w_scales.shape[1]):
        at = slice(c * BLOCK, (c + 1) * BLOCK)
        row_scale = w_scales[:, c].double().repeat_interleave(BLOCK)[:w.shape[0]]
        y += (x[:, at] @ w[:, at].double().t()) * row_scale
    return y


def _exact_gemm(s):
    x = s["x"].double()
    for c in range(s["x_scales"].shape[1]):
        x[:, c * BLOCK:(c + 1) * BLOCK] *= s["x_scales"][:, c:c + 1].double()
    return {"y": _block_product(x, s["w"], s["w_scales"])}


def _exact_moe(s):
    y = torch.zeros((s["m"], s["dim"]), dtype=torch.float64, device=DEV)
    ids = s["ids"].cpu()
    for e in sorted(set(ids.view(-1).tolist()) - {-1}):
        token, choice = (t.to(DEV) for t in (ids == e).nonzero(as_tuple=True))
        x = s["x"][token].double()
        gate, up = (_block_product(x, s["gate_up"][e, j], s["gate_up_scales"][e, j]) for j in (0, 1))
        part = _block_product(torch.nn.functional.silu(gate) * up, s["down"][e], s["down_scales"][e])
        y.index_add_(0, token, part * s["route_w"][token, choice][:, None].double())
    return {"y": y}
