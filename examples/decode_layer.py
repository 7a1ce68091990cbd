"""One transformer layer on Q2_K weights, prompt and decode, with nothing between its calls.

    python examples/decode_layer.py

Every step is a call of the library: the page plan, norms with gate and residual, Q2_K projections, rotary store,
paged attention, routing, routed experts.  A decode step is captured once as a CUDA graph and replayed; lengths, page
table and positions change on the device alone.  The weights are synthetic.  ``main`` prints how far each stage is
from the same stage in plain torch (see ``check``), and the time of a replayed step.
"""
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import mmvq_q2_gb300 as lib  # noqa: E402
import synth  # noqa: E402

EPS = 1e-6


def bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


class Layer:
    """Weights, cache and the calls of one layer."""

    def __init__(self, dim=4096, hq=32, hkv=8, d=128, experts=32, groups=4, topk=8, inter=2048, requests=4,
                 max_len=4096, page=16, seed=0):
        self.dim, self.hq, self.hkv, self.d = dim, hq, hkv, d
        self.experts, self.groups, self.topk, self.inter, self.page = experts, groups, topk, inter, page

        def q2k(name, n, k):
            return torch.from_numpy(synth.q2k_matrix(seed, name, n, k)).cuda()

        def weight(name):
            return 1.0 + 0.1 * torch.from_numpy(synth.rng(seed, name).standard_normal(dim, dtype=np.float32)).cuda()

        self.wq, self.wk, self.wv = q2k("wq", hq * d, dim), q2k("wk", hkv * d, dim), q2k("wv", hkv * d, dim)
        self.wo = q2k("wo", dim, hq * d)
        self.mats = [[q2k(f"{kind}{e}", *shape) for e in range(experts)] for kind, shape in
                     (("gate", (inter, dim)), ("up", (inter, dim)), ("down", (dim, inter)))]
        self.expert_ptrs = torch.stack([lib.pointer_table(m) for m in self.mats])
        self.router = bf16(synth.f32_to_bf16_bits(
            synth.rng(seed, "router").standard_normal((experts, dim), dtype=np.float32) * 0.02))
        self.bias = torch.from_numpy(synth.rng(seed, "bias").standard_normal(experts, dtype=np.float32) * 0.05).cuda()
        self.norms = [weight(f"norm{i}") for i in range(4)]  # before and after attention, before and after the experts
        self.gate = weight("gate")
        self.alpha, self.scale = 0.25, d ** -0.5 / 16
        half = d // 2
        self.inv_freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float32) / half)
        per_request = -(-max_len // page)
        n_pages = requests * per_request
        self.k_cache = torch.empty((n_pages, hkv, page, d), dtype=torch.bfloat16, device="cuda")
        self.v_cache = torch.empty_like(self.k_cache)
        self.table = torch.full((requests, per_request), -1, dtype=torch.int32, device="cuda")
        order = synth.rng(seed, "pages").permutation(n_pages).astype(np.int32)
        self.free = torch.from_numpy(order).cuda()
        self.head = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ctx = torch.zeros(requests, dtype=torch.int32, device="cuda")

    def project(self, w, n, n_q8, k):
        """Q2_K rows against the normed tokens: quantised for up to 8 of them, on the tensor cores for more."""
        return lib.q2k_mmq_bf16(w, n) if n.shape[0] > 8 else lib.q2k_mmvq_q8_1(w, n_q8, k)

    def step(self, stream, new_lens):
        """fp32 ``stream [T, dim]`` of the new tokens, request by request, updated in place; what the stages gave."""
        T = stream.shape[0]
        plan = lib.kv_page_plan(self.ctx, new_lens, self.page, self.free, self.table, T, free_head=self.head)
        _, n1, n1_q8 = lib.norm_gate_residual(stream, self.norms[0], EPS, residual_out=stream, want_q8=True)
        q = self.project(self.wq, n1, n1_q8, self.dim).view(T, self.hq, self.d)
        if T > 8:
            k, v = lib.q2k_mmq_bf16(self.wk, n1), lib.q2k_mmq_bf16(self.wv, n1)
        else:
            k, v = lib.q2k_mmvq_pair(self.wk, self.wv, n1_q8, self.dim)
        k, v = k.view(T, self.hkv, self.d), v.view(T, self.hkv, self.d)
        q_rot = lib.kv_rope_store(q, k, v, plan.positions, self.inv_freq, plan.slot_map, self.k_cache, self.v_cache)
        o, _ = lib.kv_attention_bf16(q_rot, self.k_cache, self.v_cache, self.table, plan.cu_q, plan.seq_lens,
                                     scale=self.scale)
        o = o.view(T, -1)
        y = self.project(self.wo, o, None if T > 8 else lib.q8_1_quantize_rows(o), self.hq * self.d)
        before = stream.clone()
        _, n2 = lib.norm_gate_residual(stream, self.norms[2], EPS, y=y, post_w=self.norms[1], gate=self.gate,
                                       alpha=self.alpha, residual_out=stream)
        logits = lib.dense_gemm_bf16(n2, self.router)
        ids, w, ptrs = lib.moe_route_topk(logits, self.topk, bias=self.bias, score="sigmoid", n_group=self.groups,
                                          topk_group=self.groups // 2, scale=2.5, expert_ptrs=self.expert_ptrs)
        moe = torch.empty((T, self.dim), dtype=torch.float32, device="cuda")
        ws = torch.empty(lib.q2k_moe_m1_workspace_bytes(self.topk, self.dim, self.inter), dtype=torch.uint8,
                         device="cuda")
        for t in range(T):
            lib.q2k_moe_m1(ptrs[t], self.topk, self.dim, self.inter, n2[t], w[t], y=moe[t], workspace=ws)
        middle = stream.clone()
        _, out = lib.norm_gate_residual(stream, self.norms[0], EPS, y=moe, post_w=self.norms[3], alpha=self.alpha,
                                        residual_out=stream)
        # the next step's lengths and free pages
        self.ctx.copy_(plan.seq_lens)
        self.head.copy_(plan.free_head)
        return dict(plan=plan, n1=n1, q=q, k=k, v=v, o=o, y=y, before=before, middle=middle, n2=n2, logits=logits,
                    ids=ids, w=w, moe=moe, stream=stream, out=out)


def rms(x, w):
    x = x.double()
    return x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()


def check(layer, s, history):
    """How far each stage is from plain 64-bit torch on the stage's own inputs, relative to the result's norm.
    ``history``: per request the rotated K and V of all its tokens so far; this step's are appended."""
    def off(got, want):
        return ((got.double() - want).norm() / want.norm()).item()

    def dense(w, k):
        return lib.q2k_dequant_rows(w, k).double()

    d, far = layer.d, {}
    n1 = s["n1"].double()
    far["projections"] = max(off(s[name].reshape(n1.shape[0], -1), n1 @ dense(w, layer.dim).t())
                             for name, w in (("q", layer.wq), ("k", layer.wk), ("v", layer.wv)))
    angle = (s["plan"].positions[:, None].float() * layer.inv_freq).double()[:, None]

    def rotated(x):
        a, b = x.double().chunk(2, -1)
        return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1).bfloat16()

    q, k, v = rotated(s["q"]).double(), rotated(s["k"]), s["v"].bfloat16()
    o, cu = torch.empty_like(q), s["plan"].cu_q.tolist()
    for r, (a, b) in enumerate(zip(cu, cu[1:])):
        if a == b:
            continue
        history[r] = [torch.cat([h, x[a:b]]) for h, x in zip(history[r], (k, v))]
        keys, values = (h.double().repeat_interleave(layer.hq // layer.hkv, 1) for h in history[r])
        score = torch.einsum("thd,jhd->htj", q[a:b], keys) * layer.scale
        j, n = torch.arange(len(keys), device="cuda"), b - a
        score.masked_fill_(j > (len(keys) - n + torch.arange(n, device="cuda"))[:, None], -torch.inf)
        o[a:b] = torch.einsum("htj,jhd->thd", score.softmax(-1), values)
    far["attention"] = off(s["o"].view_as(o), o)
    far["out projection"] = off(s["y"], s["o"].double() @ dense(layer.wo, layer.hq * d).t())
    middle = s["before"].double() + layer.alpha * rms(s["y"], layer.norms[1]) * layer.gate.double()
    far["norms"] = max(off(s["middle"], middle), off(s["n2"], rms(middle, layer.norms[2])))
    score = torch.sigmoid(s["logits"].double())
    best = (score + layer.bias.double()).view(-1, layer.groups, layer.experts // layer.groups)
    kept = best.topk(2, -1)[0].sum(-1).topk(layer.groups // 2, -1)[1]
    mask = torch.zeros(best.shape[:2], dtype=torch.bool, device="cuda").scatter_(1, kept, True)
    ids = best.masked_fill(~mask[..., None], -torch.inf).flatten(1).topk(layer.topk, -1)[1]
    w = score.gather(1, ids)
    far["route"] = 0.0 if torch.equal(ids, s["ids"].long()) else 1.0
    far["route weights"] = off(s["w"], w / w.sum(-1, keepdim=True) * 2.5)
    moe = torch.zeros_like(s["moe"], dtype=torch.float64)
    for t, row in enumerate(s["ids"].tolist()):
        x = s["n2"][t].double()
        for e, weight in zip(row, s["w"][t].tolist()):
            g, u = (dense(layer.mats[i][e], layer.dim) @ x for i in (0, 1))
            moe[t] += weight * (dense(layer.mats[2][e], layer.inter) @ (torch.nn.functional.silu(g) * u))
    far["experts"] = off(s["moe"], moe)
    far["stream"] = off(s["stream"], s["middle"].double() + layer.alpha * rms(s["moe"], layer.norms[3]))
    return far


def main():
    requests = 4
    layer = Layer(requests=requests)
    history = [[torch.empty((0, layer.hkv, layer.d), dtype=torch.bfloat16, device="cuda")] * 2
               for _ in range(requests)]

    def report(what, far):
        print(what + ":", ", ".join(f"{name} {v:.1e}" for name, v in far.items()))

    prompts = torch.tensor([37, 5, 0, 100], dtype=torch.int32, device="cuda")  # one request joins later
    stream = torch.randn(int(prompts.sum()), layer.dim, device="cuda")
    report("prompts", check(layer, layer.step(stream, prompts), history))

    one = torch.ones(requests, dtype=torch.int32, device="cuda")
    stream = torch.randn(requests, layer.dim, device="cuda")
    report("decode", check(layer, layer.step(stream, one), history))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = layer.step(stream, one)
    for i in range(3):
        stream.copy_(torch.randn(requests, layer.dim, device="cuda"))
        graph.replay()
        report(f"replay {i}", check(layer, s, history))
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(200):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"a replayed step of {requests} tokens: {begin.elapsed_time(end) / 200 * 1e3:.1f} us")
    assert lib.q2k_device_error() == 0


if __name__ == "__main__":
    main()
