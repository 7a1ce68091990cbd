"""The decode-layer calls against plain 64-bit computations of the same
formulas: kv_page_plan, kv_rope_store, kv_attention_bf16,
norm_gate_residual, moe_route_topk, and one layer that runs them together
with the projections.

Tolerances come from the roundings the calls state:
  * bf16 results: half a unit in the last of 8 bits, at most 2^-8 of the
    value, plus the fp32 arithmetic before it;
  * attention: the probabilities enter the second product as bf16, off by at
    most 2^-8 of each, so at most 2^-8 * sum_j p_j |v_j|; fp32 scores add less
    than 2^-12 of the same sum at these sizes;
  * whole numbers are equal.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
HALF_ULP = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def lib():
    from mmvq_q2_gb300 import build
    build.build()
    import mmvq_q2_gb300 as q
    q.lib()
    q.q2k_device_error(clear=True)
    yield q
    torch.cuda.synchronize()
    assert q.q2k_device_error(clear=True) == 0


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def within(got, want, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    over = ((got - want).abs() - tol).max().item() if got.numel() else 0.0
    assert over <= 0, f"{what}: {over:.3e} beyond the tolerance"


# ---- kv_page_plan ----------------------------------------------------------------

def plan_by_hand(ctx, new, page, free, head, table, max_tokens):
    """The plan in plain Python; returns table, cu, seq, positions, requests, slots, head, error bits."""
    table = [list(row) for row in table]
    ld, err, taken = len(table[0]), 0, 0
    cu, seq, pos, req, slots = [0], [], [], [], []
    if head < 0:
        head, err = 0, err | 4
    for r, (c, w) in enumerate(zip(ctx, new)):
        if c < 0 or w < 0:
            err |= 4
        c, w = max(c, 0), max(w, 0)
        seq.append(c + w)
        if w and c + w > ld * page:
            err |= 2
        for col in range(min(-(-c // page), ld), min(-(-(c + w) // page), ld)):
            at = head + taken
            taken += 1
            if at >= len(free):
                err |= 1
            table[r][col] = free[at] if at < len(free) else -1
        for i in range(w):
            p = c + i
            col = p // page
            entry = table[r][col] if col < ld else -1
            pos.append(p)
            req.append(r)
            slots.append(entry * page + p % page if entry >= 0 else -1)
        cu.append(cu[-1] + w)
    if cu[-1] > max_tokens:
        err |= 8
    cu = [min(c, max_tokens) for c in cu]
    pad = [-1] * max(0, max_tokens - len(pos))
    cut = lambda v: (v + pad)[:max_tokens]  # noqa: E731
    return table, cu, seq, cut(pos), cut(req), cut(slots), max(head, min(head + taken, len(free))), err


PLANS = {
    "one": ([0], [1], 16, 4, 8, 0, 1),
    "page-edges": ([0, 15, 16, 17, 31, 32, 0, 5], [16, 1, 1, 15, 2, 0, 17, 0], 16, 6, 64, 3, 60),
    "idle": ([40, 0, 7], [0, 0, 0], 16, 4, 8, 0, 5),
    "no-tokens-wanted": ([40, 0], [0, 0], 32, 4, 8, 0, 0),
    "pool-runs-out": ([10, 0, 20], [40, 40, 40], 16, 8, 5, 1, 120),
    "row-too-short": ([10, 60, 100], [40, 20, 3], 16, 4, 40, 0, 63),
    "negative": ([-5, 20], [3, -2], 16, 4, 10, -1, 10),
    "too-many-tokens": ([3, 3, 3], [10, 10, 10], 16, 4, 20, 0, 17),
    "page-1024": ([1000, 1024, 5000], [100, 1, 2000], 1024, 9, 20, 0, 2200),
}


@pytest.mark.parametrize("name", PLANS)
def test_page_plan_by_hand(lib, name):
    ctx, new, page, ld, n_free, head, max_tokens = PLANS[name]
    used = 1000
    table = [[used + 10 * r + c if c < -(-max(x, 0) // page) else -7 for c in range(ld)] for r, x in enumerate(ctx)]
    free = [500 - 3 * i for i in range(n_free)]
    want = plan_by_hand(ctx, new, page, free, head, table, max_tokens)
    dt, err = i32(table), i32([0])
    p = lib.kv_page_plan(i32(ctx), i32(new), page, i32(free), dt, max_tokens, free_head=i32([head]), err_flag=err)
    got = (dt.tolist(), p.cu_q.tolist(), p.seq_lens.tolist(), p.positions.tolist(), p.token_req.tolist(),
           p.slot_map.tolist(), p.free_head.item(), err.item())
    assert got == tuple(want)


@pytest.mark.parametrize("n_req", [1, 511, 512, 513, 2500, 16384])
def test_page_plan_many_requests_and_a_strided_table(lib, n_req):
    page, ld = 16, 6
    cpu = torch.Generator().manual_seed(n_req)
    ctx = torch.randint(0, 40, (n_req,), generator=cpu).tolist()
    new = torch.randint(0, 30, (n_req,), generator=cpu).tolist()
    table = [[100000 + r * ld + c for c in range(ld)] for r in range(n_req)]
    free = list(range(3 * n_req + 5))
    total = sum(new) + 3
    want = plan_by_hand(ctx, new, page, free, 0, table, total)
    wide = torch.full((n_req, ld + 3), -9, dtype=torch.int32, device=DEV)
    wide[:, :ld] = i32(table)
    p = lib.kv_page_plan(i32(ctx), i32(new), page, i32(free), wide[:, :ld], total)
    # the row may use its whole stride: these requests stay within ld columns
    assert wide[:, :ld].tolist() == want[0] and (wide[:, ld:] == -9).all()
    assert p.cu_q.tolist() == want[1] and p.seq_lens.tolist() == want[2] and p.positions.tolist() == want[3]
    assert p.token_req.tolist() == want[4] and p.slot_map.tolist() == want[5] and p.free_head.item() == want[6]


# ---- kv_rope_store ---------------------------------------------------------------

def turned(x, pos, sections, inv_freq, interleaved):
    """x [T, H, D] rotated in 64 bits; the angle is one fp32 product, as the call states."""
    axis = torch.tensor([a for a, c in enumerate(sections) for _ in range(c)], device=DEV, dtype=torch.long)
    ang = (pos[axis].float().t() * inv_freq).double()
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    half = inv_freq.numel()
    i = torch.arange(half, device=DEV)
    i1, i2 = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    out = x.double().clone()
    a, b = out[..., i1].clone(), out[..., i2].clone()
    out[..., i1], out[..., i2] = a * c - b * s, b * c + a * s
    return out


ROPES = [
    # T, Hq, Hkv, D, rot, sections, interleaved, dtype, page
    (1, 4, 2, 128, 128, (64,), False, torch.float32, 16),
    (1, 1, 1, 64, 64, (32,), True, torch.bfloat16, 16),
    (37, 5, 1, 128, 64, (8, 12, 12), False, torch.bfloat16, 32),
    (37, 4, 4, 96, 96, (16, 16, 16), True, torch.float32, 64),
    (5, 3, 3, 96, 48, (24,), False, torch.float32, 16),
    (129, 32, 8, 128, 128, (16, 24, 24), False, torch.float32, 16),
    (9, 130, 2, 128, 128, (64, 0), True, torch.bfloat16, 16),
    (6, 2, 2, 100, 100, (50,), False, torch.float32, 16),
    (6, 2, 1, 72, 26, (3, 10, 0), True, torch.bfloat16, 16),
    (4, 2, 2, 16, 0, (0,), False, torch.float32, 16),
    (3, 2, 1, 512, 512, (256,), False, torch.float32, 1024),
    (3, 1, 1, 1, 0, (0,), False, torch.float32, 16),
    # many tokens, a token to a block
    (2501, 12, 4, 128, 128, (16, 24, 24), False, torch.float32, 64),
    (2434, 12, 4, 128, 64, (32,), True, torch.bfloat16, 16),
    (9999, 4, 2, 96, 96, (48,), False, torch.bfloat16, 16),
]


@pytest.mark.parametrize("case", ROPES, ids=lambda c: "-".join(map(str, c[:5])))
def test_rope_store(lib, case):
    T, Hq, Hkv, D, rot, sections, interleaved, dtype, page = case
    g = gen(T * D + rot)
    q, k, v = normal(g, T, Hq, D, dtype=dtype), normal(g, T, Hkv, D, dtype=dtype), normal(g, T, Hkv, D, dtype=dtype)
    n_pages = T // page + 3
    kc, vc = (normal(g, n_pages, Hkv, page, D, dtype=torch.bfloat16) for _ in range(2))
    kc0, vc0 = kc.clone(), vc.clone()
    slots = torch.randperm(n_pages * page, generator=g, device=DEV)[:T].to(torch.int32)
    if T > 4:
        slots[2] = -1  # padding: not stored
    pos = torch.randint(0, 150000, (len(sections), T), generator=g, device=DEV, dtype=torch.int32)
    inv = 10000.0 ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float32) / max(1, rot // 2))
    out = lib.kv_rope_store(q, k, v, pos, inv, slots, kc, vc, sections=sections, interleaved=interleaved)
    # sincosf is good to 2 units of 2^-24, the two products and the sum to 3 more: 2^-21 of |a| + |b|, each
    # at most the head's largest value
    want = turned(q, pos, sections, inv, interleaved)
    within(out, want, HALF_ULP * want.abs() + 2.0 ** -20 * q.double().abs().amax(-1, keepdim=True), "q")
    live = (slots >= 0).nonzero()[:, 0]
    at = slots[live].long()
    want_k = turned(k, pos, sections, inv, interleaved)[live]
    within(kc[at // page, :, at % page], want_k,
           HALF_ULP * want_k.abs() + 2.0 ** -20 * k[live].double().abs().amax(-1, keepdim=True), "k")
    assert torch.equal(vc[at // page, :, at % page], v[live].bfloat16())
    # nothing else of the cache changed
    kc[at // page, :, at % page] = kc0[at // page, :, at % page]
    vc[at // page, :, at % page] = vc0[at // page, :, at % page]
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)


def test_rope_store_strides_unaligned_views_and_bad_slots(lib):
    T, Hq, Hkv, D, page = 21, 6, 2, 64, 16
    g = gen(5)
    inv = 500000.0 ** (-torch.arange(32, device=DEV, dtype=torch.float32) / 32)
    pos = torch.arange(90, 90 + T, device=DEV, dtype=torch.int32)
    slots = torch.arange(T, device=DEV, dtype=torch.int32)
    both = normal(g, 4, 2, Hkv, page, D, dtype=torch.bfloat16)  # K and V pages alternate
    results = []
    for shift in (0, 1):  # one projection's row holds q, k and v; shifted by a value it is off 16 bytes
        flat = normal(gen(6), T * ((Hq + 2 * Hkv) * D + 8) + 8)
        if shift:
            flat = torch.cat([flat[:1], flat[:-1]])
        rows = flat[shift:shift + T * ((Hq + 2 * Hkv) * D + 8)].view(T, -1)
        q = rows[:, :Hq * D].unflatten(1, (Hq, D))
        k = rows[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        v = rows[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].unflatten(1, (Hkv, D))
        c = both.clone()
        q_out = torch.zeros(T, Hq * D + 24, device=DEV, dtype=torch.bfloat16)
        err = i32([0])
        lib.kv_rope_store(q, k, v, pos, inv, slots, c[:, 0], c[:, 1],
                          q_out=q_out[:, :Hq * D].unflatten(1, (Hq, D)), err_flag=err)
        assert err.item() == 0 and (q_out[:, Hq * D:] == 0).all()
        results.append((q_out, c, turned(q, pos[None], (32,), inv, False)))
    # value by value and 16 at a time give the same bits
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
    want = results[0][2]
    within(results[0][0][:, :Hq * D].unflatten(1, (Hq, D)), want, HALF_ULP * want.abs() + 1e-5, "strided q")
    # store only, and a slot past the cache: flagged, not stored
    c, err = both.clone(), i32([0])
    bad = slots.clone()
    bad[3] = 4 * page
    k = normal(g, T, Hkv, D)
    assert lib.kv_rope_store(None, k, k, pos, inv, bad, c[:, 0], c[:, 1], err_flag=err) is None
    assert err.item() == 1
    assert torch.equal(c[0, :, :, 3], both[0, :, :, 3]) and not torch.equal(c[0, :, :, 4], both[0, :, :, 4])
    # no tokens
    out = lib.kv_rope_store(q[:0], k[:0], k[:0], pos[:0], inv, slots[:0], c[:, 0], c[:, 1])
    assert out.shape == (0, Hq, D)


# ---- kv_attention_bf16 -----------------------------------------------------------

class Cache:
    """A paged cache of given requests: pages in random order, what no request owns holds `fill`."""

    def __init__(self, g, seq, hkv, d, page, fill=float("nan"), alternate=False, spare=3, std=1.0):
        counts = [-(-max(s, 0) // page) for s in seq]
        self.n_pages = sum(counts) + spare
        perm = torch.randperm(self.n_pages, generator=g, device=DEV).tolist()
        ld = max(counts + [0]) + 2
        rows, at = [], 0
        for c in counts:
            rows.append(perm[at:at + c] + [-1] * (ld - c))
            at += c
        self.table = i32(rows) if rows else torch.zeros((0, ld), dtype=torch.int32, device=DEV)
        shape = (self.n_pages, 2, hkv, page, d) if alternate else (2, self.n_pages, hkv, page, d)
        buf = torch.full(shape, fill, dtype=torch.bfloat16, device=DEV)
        self.k, self.v = (buf[:, 0], buf[:, 1]) if alternate else (buf[0], buf[1])
        self.keys, self.values = [], []
        for r, s in enumerate(seq):
            k, v = (normal(g, max(s, 0), hkv, d, dtype=torch.bfloat16, std=std) for _ in range(2))
            self.keys.append(k)
            self.values.append(v)
            if s > 0:
                j = torch.arange(s, device=DEV)
                pages = self.table[r].long()[j // page]
                self.k[pages, :, j % page] = k
                self.v[pages, :, j % page] = v


def attention_64(q, keys, values, cu, seq, scale, window):
    """out, lse and sum_j p_j |v_j| in 64 bits, request by request."""
    T, Hq, D = q.shape
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=DEV)
    size = torch.zeros_like(out)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=DEV)
    for r, s in enumerate(seq):
        a, b = cu[r], cu[r + 1]
        if a == b or s <= 0:
            continue
        group = Hq // keys[r].shape[1]
        k = keys[r].double().repeat_interleave(group, 1)
        v = values[r].double().repeat_interleave(group, 1)
        p = s - (b - a) + torch.arange(b - a, device=DEV)
        j = torch.arange(s, device=DEV)
        seen = j <= p[:, None]
        if window:
            seen &= j > p[:, None] - window
        score = torch.einsum("thd,jhd->htj", q[a:b].double(), k) * scale
        score = score.masked_fill(~seen, -math.inf)
        z = torch.logsumexp(score, -1)
        w = torch.exp(score - z.masked_fill(z == -math.inf, 0.0)[..., None])
        out[a:b] = torch.einsum("htj,jhd->thd", w, v)
        size[a:b] = torch.einsum("htj,jhd->thd", w, v.abs())
        lse[a:b] = z.t()
    return out, lse, size


def check_attention(got, lse, want):
    out, z, size = want
    within(got, out, HALF_ULP * out.abs() + (HALF_ULP + 2.0 ** -12) * size + 1e-30, "out")
    empty = z == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    assert (got[empty] == 0).all()
    within(lse.masked_fill(empty, 0.0), z.masked_fill(empty, 0.0), 2.0 ** -15 + 2.0 ** -19 * z.masked_fill(empty, 0.0).abs(),
           "lse")


ATTENTIONS = [
    # context lengths, new tokens, Hq, Hkv, D, page, window
    ([0], [1], 1, 1, 128, 16, 0),
    ([5], [1], 4, 4, 64, 16, 0),
    ([126], [1], 8, 2, 128, 16, 0),
    ([127], [1], 8, 2, 128, 128, 0),
    ([128], [1], 8, 2, 128, 32, 0),
    ([1000, 0, 63, 129, 4000], [1, 1, 1, 1, 1], 32, 8, 128, 16, 0),
    ([300, 20, 700], [1, 1, 1], 16, 1, 128, 64, 0),
    ([300, 20, 700], [1, 1, 1], 128, 1, 64, 64, 0),
    ([0], [128], 1, 1, 128, 16, 0),
    ([0], [129], 1, 1, 64, 16, 0),
    ([3], [257], 2, 1, 128, 256, 0),
    ([100], [511], 3, 1, 128, 16, 0),
    ([0, 0, 0], [17, 200, 33], 6, 2, 128, 32, 0),
    ([700, 0, 3, 90, 11], [1, 0, 300, 2, 64], 8, 2, 128, 16, 0),
    ([700, 40, 3], [60, 5, 300], 20, 4, 64, 32, 0),
    ([50], [90], 7, 1, 96, 16, 0),
    ([50], [90], 10, 2, 80, 16, 0),
    ([50], [90], 4, 2, 16, 16, 0),
    ([50], [90], 4, 2, 48, 1024, 0),
    ([260], [90], 4, 2, 112, 16, 0),
    ([333, 0], [40, 90], 8, 2, 128, 16, 1),
    ([333, 0], [40, 90], 8, 2, 128, 16, 7),
    ([333, 0], [40, 300], 8, 2, 128, 16, 128),
    ([3333, 0, 90], [1, 1, 1], 8, 2, 128, 16, 200),
    ([1000, 5], [300, 700], 4, 4, 64, 32, 129),
    ([12000], [1], 4, 1, 128, 16, 0),
    ([20001, 7], [3, 3], 8, 2, 128, 64, 0),
    ([2000], [1100], 4, 1, 128, 16, 0),
]


@pytest.mark.parametrize("case", ATTENTIONS, ids=lambda c: f"ctx{c[0][0]}-new{c[1][0]}-h{c[2]}.{c[3]}-d{c[4]}-p{c[5]}-w{c[6]}")
def test_attention(lib, case):
    ctx, new, Hq, Hkv, D, page, window = case
    g = gen(sum(ctx) + sum(new) + D)
    seq = [c + n for c, n in zip(ctx, new)]
    c = Cache(g, seq, Hkv, D, page)  # unused rows hold NaN
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = normal(g, cu[-1], Hq, D, dtype=torch.bfloat16, std=1.5)
    out, lse = lib.kv_attention_bf16(q, c.k, c.v, c.table, i32(cu), i32(seq), window=window, want_lse=True)
    check_attention(out, lse, attention_64(q, c.keys, c.values, cu, seq, D ** -0.5, window))
    # the same call again gives the same bits
    again, lse2 = lib.kv_attention_bf16(q, c.k, c.v, c.table, i32(cu), i32(seq), window=window, want_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("n_req, new, ctx, heads, window", [
    (32, [1], [0, 700, 90], (8, 2), 0),          # as many as one warp takes
    (33, [1], [0, 700, 90], (8, 2), 0),
    (33, [1, 0, 40], [900, 3, 0], (2, 1), 0),
    (64, [0, 1, 150, 1], [5, 1300, 0, 260], (4, 1), 0),
    (385, [1, 2], [0, 127, 300], (4, 2), 0),     # more than a block has threads
    (385, [0, 33, 1, 5], [0, 127, 130], (4, 2), 50),
    (1000, [1, 0, 0, 3], [20, 1, 0], (1, 1), 0),
])
def test_attention_of_many_requests(lib, n_req, new, ctx, heads, window):
    """Every way the work is counted and divided: few and many requests, with few and many key tiles."""
    g = gen(31)
    news = [new[i % len(new)] for i in range(n_req)]
    seq = [news[i] + ctx[i % len(ctx)] for i in range(n_req)]
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    c = Cache(g, seq, heads[1], 64, 16)
    q = normal(g, cu[-1], heads[0], 64, dtype=torch.bfloat16)
    out, lse = lib.kv_attention_bf16(q, c.k, c.v, c.table, i32(cu), i32(seq), window=window, want_lse=True)
    check_attention(out, lse, attention_64(q, c.keys, c.values, cu, seq, 64 ** -0.5, window))
    assert lib.q2k_device_error(clear=True) == 0


@pytest.mark.parametrize("ctx, new, heads, d, window", [
    ([511], [1], (4, 1), 128, 0),                     # four key tiles
    ([512], [1], (4, 1), 128, 0),                     # five
    ([300, 0, 0, 129, 7], [1, 0, 1, 3, 2], (8, 2), 64, 0),
    ([300, 450], [2, 2], (128, 2), 96, 0),            # a token fills half a row tile
    ([400, 90], [16, 5], (16, 2), 128, 100),          # a window that leaves out whole tiles
    ([40 * i for i in range(16)], [1] * 16, (16, 8), 128, 0),
    ([60 * i for i in range(16)], [1] * 16, (32, 8), 64, 0),  # as long as a CTA's share and four tiles
    ([500] * 19, [1] * 19, (8, 8), 64, 0),            # 152 items
    ([500] * 20, [1] * 20, (8, 8), 64, 0),            # more
])
def test_attention_of_few_key_tiles(lib, ctx, new, heads, d, window):
    """Items that are not split, next to such as are."""
    g = gen(32)
    seq = [c + n for c, n in zip(ctx, new)]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    c = Cache(g, seq, heads[1], d, 16)
    q = normal(g, cu[-1], heads[0], d, dtype=torch.bfloat16)
    out, lse = lib.kv_attention_bf16(q, c.k, c.v, c.table, i32(cu), i32(seq), window=window, want_lse=True)
    check_attention(out, lse, attention_64(q, c.keys, c.values, cu, seq, d ** -0.5, window))
    assert lib.q2k_device_error(clear=True) == 0


def test_attention_without_cached_rows(lib):
    """Requests whose cache is shorter than their new tokens: the first rows see nothing."""
    g = gen(1)
    seq, new = [5, 0, 1, 200], [9, 4, 3, 300]
    c = Cache(g, seq, 2, 128, 16)
    cu = [0, 9, 13, 16, 316]
    q = normal(g, 316, 4, 128, dtype=torch.bfloat16)
    out, lse = lib.kv_attention_bf16(q, c.k, c.v, c.table, i32(cu), i32(seq), want_lse=True)
    check_attention(out, lse, attention_64(q, c.keys, c.values, cu, seq, 128 ** -0.5, 0))


@pytest.mark.parametrize("window", [0, 150])
def test_attention_large_scores_and_probabilities_near_one(lib, window):
    """Scores in the hundreds, rising along the keys, so the running maximum moves on every tile."""
    g = gen(2)
    seq, new = [900, 700], [1, 260]
    c = Cache(g, seq, 1, 128, 16)
    for r in range(2):
        lift = torch.linspace(-1, 1, seq[r], device=DEV)[:, None, None]
        c.keys[r] = (0.1 * c.keys[r].float() + 4 * lift).bfloat16()
        j = torch.arange(seq[r], device=DEV)
        c.k[c.table[r].long()[j // 16], :, j % 16] = c.keys[r]
    cu = [0, 1, 261]
    q = (normal(g, 261, 2, 128) * 0.1 + torch.tensor([4.0, -4.0], device=DEV)[:, None]).bfloat16()
    out, lse = lib.kv_attention_bf16(q, c.k, c.v, c.table, i32(cu), i32(seq), window=window, want_lse=True)
    want, z, size = attention_64(q, c.keys, c.values, cu, seq, 128 ** -0.5, window)
    # scores up to 181: their fp32 rounding (128 terms of up to 16, 2^-24 each) reaches e^(2^-12) - 1
    within(out, want, HALF_ULP * want.abs() + (HALF_ULP + 2.0 ** -10) * size, "out")
    within(lse, z, 2.0 ** -12 + 2.0 ** -19 * z.abs(), "lse")


def test_attention_strides_alternating_pages_padding_rows(lib):
    g = gen(3)
    seq, new, Hq, Hkv, D = [77, 300], [7, 100], 6, 2, 64
    c = Cache(g, seq, Hkv, D, 16, alternate=True)
    cu = [0, 7, 107]
    wide = normal(g, 120, Hq * D + 40, dtype=torch.bfloat16)
    q = wide[:, 8:8 + Hq * D].unflatten(1, (Hq, D))
    out_wide = torch.full((120, Hq * D + 6), 3.0, dtype=torch.bfloat16, device=DEV)
    out = out_wide[:, 3:3 + Hq * D].unflatten(1, (Hq, D))
    table = torch.full((2, c.table.shape[1] + 5), -1, dtype=torch.int32, device=DEV)
    table[:, :c.table.shape[1]] = c.table
    lse = torch.full((120, Hq), 5.0, device=DEV)
    lib.kv_attention_bf16(q, c.k, c.v, table[:, :c.table.shape[1]], i32(cu), i32(seq), out=out, lse=lse, scale=0.3)
    check_attention(out[:107], lse[:107], attention_64(q[:107], c.keys, c.values, cu, seq, 0.3, 0))
    # tokens past the last request, and what lies around the rows, stay
    assert (out[107:] == 3.0).all() and (lse[107:] == 5.0).all()
    assert (out_wide[:, :3] == 3.0).all() and (out_wide[:, 3 + Hq * D:] == 3.0).all()
    # no tokens, no requests
    o, z = lib.kv_attention_bf16(q[:0], c.k, c.v, table, i32([0, 0, 0]), i32(seq), want_lse=True)
    assert o.shape == (0, Hq, D) and z.shape == (0, Hq)
    lib.kv_attention_bf16(q, c.k, c.v, table[:0], i32([0]), i32([]), out=out)
    assert (out[107:] == 3.0).all()


def test_attention_reads_bad_table_entries_as_zeros_and_says_so(lib):
    g = gen(4)
    c = Cache(g, [64], 1, 64, 16, fill=0.0)
    q = normal(g, 1, 2, 64, dtype=torch.bfloat16)
    table = c.table.clone()
    table[0, 1] = c.n_pages
    table[0, 2] = -5
    c.keys[0][16:48] = 0
    c.values[0][16:48] = 0
    torch.cuda.synchronize()
    assert lib.q2k_device_error(clear=True) == 0
    out, lse = lib.kv_attention_bf16(q, c.k, c.v, table, i32([0, 1]), i32([64]), want_lse=True)
    check_attention(out, lse, attention_64(q, c.keys, c.values, [0, 1], [64], 0.125, 0))
    torch.cuda.synchronize()
    assert lib.q2k_device_error(clear=True) == 2
    # a length past the table's row reads no entry of another row
    lib.kv_attention_bf16(q, c.k, c.v, c.table[:, :2], i32([0, 1]), i32([1 << 14]))
    torch.cuda.synchronize()
    assert lib.q2k_device_error(clear=True) == 2


def test_attention_in_a_cache_past_32_bit_offsets(lib):
    """Pages at byte (and element) offsets beyond 2^32."""
    g = gen(7)
    Hkv, D, page, seq = 8, 128, 64, [500, 130]
    n_pages = (5 << 30) // (Hkv * page * D)  # 5 Gi values each
    small = Cache(g, seq, Hkv, D, page, spare=0)
    high = torch.tensor([n_pages - 1 - 3 * i for i in range(small.n_pages)], device=DEV)
    k = torch.empty((n_pages, Hkv, page, D), dtype=torch.bfloat16, device=DEV)
    v = torch.empty((n_pages, Hkv, page, D), dtype=torch.bfloat16, device=DEV)
    k[high], v[high] = small.k, small.v
    table = torch.where(small.table >= 0, high[small.table.clamp(min=0).long()].to(torch.int32), -1)
    q = normal(g, 3, 16, D, dtype=torch.bfloat16)
    cu = [0, 1, 3]
    out, lse = lib.kv_attention_bf16(q, k, v, table.contiguous(), i32(cu), i32(seq), want_lse=True)
    check_attention(out, lse, attention_64(q, small.keys, small.values, cu, seq, D ** -0.5, 0))
    new = normal(g, 1, Hkv, D, dtype=torch.bfloat16)
    lib.kv_rope_store(None, new, new, i32([0]), torch.ones(64, device=DEV), i32([(n_pages - 1) * page + 5]), k, v)
    assert torch.equal(k[n_pages - 1, :, 5], new[0]) and torch.equal(v[n_pages - 1, :, 5], new[0])


def test_attention_on_another_stream_and_in_a_graph(lib):
    g = gen(8)
    seq, new = [700, 90], [1, 1]
    c = Cache(g, seq, 2, 128, 16)
    q = normal(g, 2, 8, 128, dtype=torch.bfloat16)
    cu, lens = i32([0, 1, 2]), i32(seq)
    want, _ = lib.kv_attention_bf16(q, c.k, c.v, c.table, cu, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(q)
    ws = torch.empty(lib.kv_attention_workspace_bytes(2, 8, 2, 128), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    lib.kv_attention_bf16(q, c.k, c.v, c.table, cu, lens, out=out, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(graph):
        lib.kv_attention_bf16(q, c.k, c.v, c.table, cu, lens, out=out, workspace=ws)
    # new lengths in place: the same graph serves the next step
    lens.copy_(i32([640, 33]))
    graph.replay()
    torch.cuda.synchronize()
    want = attention_64(q, [k[:s] for k, s in zip(c.keys, (640, 33))], [v[:s] for v, s in zip(c.values, (640, 33))],
                        [0, 1, 2], [640, 33], 128 ** -0.5, 0)
    within(out, want[0], HALF_ULP * want[0].abs() + (HALF_ULP + 2.0 ** -12) * want[2], "replayed")


def test_what_a_call_allocates_belongs_to_the_stream_it_runs_on(lib, monkeypatch):
    """A workspace that goes back at the call's end must not serve another stream while the kernels run."""
    side, streams, empty = torch.cuda.Stream(), [], torch.empty
    g = gen(21)
    c = Cache(g, [40], 2, 64, 16)
    q, x, k = normal(g, 1, 4, 64, dtype=torch.bfloat16), normal(g, 2, 256), normal(g, 1, 2, 64)
    args = i32([0, 1]), i32([40])
    free, table, head = i32(list(range(8))), torch.full((1, 8), -1, dtype=torch.int32, device=DEV), i32([0])
    logits, one, freq = normal(g, 2, 16), torch.ones(256, device=DEV), torch.ones(32, device=DEV)
    pos, slot, ctx, new = i32([3]), i32([-1]), i32([3]), i32([1])
    torch.cuda.synchronize()

    def noted(*a, **kw):
        streams.append(torch.cuda.current_stream())
        return empty(*a, **kw)

    monkeypatch.setattr(torch, "empty", noted)
    lib.kv_page_plan(ctx, new, 16, free, table, 1, free_head=head, stream=side)
    lib.kv_rope_store(q, k.to(torch.bfloat16), k.to(torch.bfloat16), pos, freq, slot, c.k, c.v, stream=side)
    lib.kv_attention_bf16(q, c.k, c.v, c.table, *args, want_lse=True, stream=side)
    lib.norm_gate_residual(x, one, 1e-6, want_q8=True, stream=side)
    lib.moe_route_topk(logits, 2, stream=side)
    monkeypatch.undo()
    side.synchronize()
    assert len(streams) == 10 and all(s == side for s in streams), streams


# ---- norm_gate_residual ----------------------------------------------------------

def norm_64(residual, y, post_w, gate, alpha, pre_w, eps):
    h = residual.double()
    size = h.abs()
    if y is not None:
        u = y.double()
        if post_w is not None:
            u = u / (u.square().mean(-1, keepdim=True) + eps).sqrt() * post_w.double()
        if gate is not None:
            u = u * gate.double()
        size = size + (alpha * u).abs()
        h = h + alpha * u
    inv = 1.0 / (h.square().mean(-1, keepdim=True) + eps).sqrt()
    return h, h * inv * pre_w.double(), size, size * inv * pre_w.double().abs()


NORMS = [
    # T, dim, y type, stream type, post, gate, alpha
    (1, 4096, "f32", "f32", True, "row", 1.0),
    (3, 4096, "bf16", "bf16", True, "token", 0.22),
    (2, 64, "bf16", "f32", False, "none", -0.5),
    (5, 8, "f32", "bf16", True, "token", 1.0),
    (4, 1, "f32", "f32", True, "row", 1.0),
    (7, 1001, "bf16", "bf16", True, "token", 0.5),
    (3, 2880, "f32", "bf16", False, "row", 2.0),
    (2, 8192, "f32", "f32", True, "token", 1.0),
    (2, 8200, "bf16", "bf16", True, "row", 1.0),
    (2, 16384, "bf16", "f32", True, "row", 1.0),
    (2, 32768, "f32", "f32", True, "token", 1.0),
    (300, 1024, "bf16", "bf16", True, "row", 0.1),
    (2, 4096, None, "bf16", False, "none", 1.0),
    (2, 77, None, "f32", False, "none", 1.0),
    # more rows than blocks
    (700, 2880, "bf16", "bf16", True, "token", 0.3),
    (1300, 4096, "bf16", "bf16", True, "row", 1.0),
    (900, 4096, None, "bf16", False, "none", 1.0),
    (1500, 2048, "f32", "f32", False, "token", 1.0),
    (5000, 160, "f32", "bf16", True, "row", 1.0),
    (400, 8192, "bf16", "f32", True, "row", 1.0),
]
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("case", NORMS, ids=lambda c: "-".join(map(str, c)))
def test_norm_gate_residual(lib, case):
    T, dim, yt, st, post, gate_kind, alpha = case
    g = gen(T * dim)
    res = normal(g, T, dim, std=2.0, dtype=TYPES[st])
    y = None if yt is None else normal(g, T, dim, std=3.0, dtype=TYPES[yt])
    gate = None if gate_kind == "none" else normal(g, *((dim,) if gate_kind == "row" else (T, dim)), dtype=TYPES[yt])
    pre, post_w = 1 + normal(g, dim, std=0.1), 1 + normal(g, dim, std=0.1) if post else None
    h64, n64, hs, ns = norm_64(res, y, post_w, gate, alpha, pre, 1e-6)
    want_q8 = dim % 32 == 0
    got = lib.norm_gate_residual(res, pre, 1e-6, y=y, post_w=post_w, gate=gate, alpha=alpha, want_q8=want_q8)
    # fp32 sums of a row in blocks of at most dim / 256 terms: 2^-18 of the terms' size covers them at 32768
    within(got[0], h64, 2.0 ** -20 * hs + (HALF_ULP * h64.abs() if st == "bf16" else 0), "stream")
    within(got[1], n64, 2.0 ** -18 * ns + HALF_ULP * n64.abs(), "normed")
    if want_q8:
        assert torch.equal(got[2], lib.q8_1_quantize_rows(got[1]))
    # in place gives the same bits
    inplace = res.clone()
    lib.norm_gate_residual(inplace, pre, 1e-6, y=y, post_w=post_w, gate=gate, alpha=alpha, residual_out=inplace)
    assert torch.equal(inplace, got[0])


def test_norm_strides_zero_rows_and_huge_values(lib):
    g = gen(11)
    T, dim = 5, 256
    wide_y, wide_r = normal(g, T, dim + 4), normal(g, T, dim + 12, dtype=torch.bfloat16)
    gate_w = normal(g, T, dim + 8)
    pre = 1 + normal(g, dim, std=0.1)
    out = torch.full((T, dim + 3), 9.0, dtype=torch.bfloat16, device=DEV)
    for off in (0, 1):  # on and off 16-byte boundaries
        y, r, gate = wide_y[:, off:off + dim], wide_r[:, off:off + dim], gate_w[:, off:off + dim]
        h, n = lib.norm_gate_residual(r, pre, 1e-5, y=y, post_w=pre, gate=gate, alpha=0.7, out=out[:, :dim])
        h64, n64, hs, ns = norm_64(r, y, pre, gate, 0.7, pre, 1e-5)
        within(h, h64, 2.0 ** -20 * hs + HALF_ULP * h64.abs(), "stream")
        within(n, n64, 2.0 ** -18 * ns + HALF_ULP * n64.abs(), "normed")
        assert (out[:, dim:] == 9.0).all()
    # a row of zeros: eps keeps the norm finite
    z = torch.zeros(2, dim, device=DEV)
    h, n = lib.norm_gate_residual(z, pre, 1e-6, y=z, post_w=pre)
    assert (h == 0).all() and (n == 0).all()
    # no tokens
    h, n = lib.norm_gate_residual(z[:0], pre, 1e-6)
    assert h.shape == (0, dim) and n.shape == (0, dim)
    # one row's NaN stays its own
    r = normal(g, 3, dim)
    r[1, 7] = float("nan")
    _, n = lib.norm_gate_residual(r, pre, 1e-6)
    assert torch.isfinite(n[0]).all() and torch.isfinite(n[2]).all() and torch.isnan(n[1]).all()


# ---- moe_route_topk --------------------------------------------------------------

def route_64(x, topk, bias, score, n_group, topk_group, renorm, scale):
    """ids and weights by sorting 64-bit scores; ties to the lowest index.  Also the smallest gap that decides."""
    x = x.double().cpu()
    x = torch.where(torch.isnan(x), -math.inf, x).clamp(max=3.4028234663852886e38)
    if score == "sigmoid":
        s = 1 / (1 + torch.exp(-x))
    else:
        top = x.amax(-1, keepdim=True).clamp(min=-3.4028234663852886e38)
        e = torch.exp(x - top)
        s = e / e.sum(-1, keepdim=True).clamp(min=1e-300)
    c = s if bias is None else s + bias.double().cpu()
    m, E = c.shape
    ids = torch.zeros(m, topk, dtype=torch.int32)
    w = torch.zeros(m, topk, dtype=torch.float64)
    gap = math.inf

    def smallest(v):
        v = v[:topk + 1] if len(v) > topk else v
        d = [a - b for a, b in zip(v, v[1:]) if a != b]
        return min(d, default=math.inf)

    for t in range(m):
        allowed = list(range(E))
        row = c[t].tolist()
        if n_group > 1:
            size = E // n_group
            best = [sum(sorted(row[i * size:(i + 1) * size], reverse=True)[:2]) for i in range(n_group)]
            order = sorted(range(n_group), key=lambda i: (-best[i], i))
            near = [best[i] for i in order[:topk_group + 1]]
            gap = min([gap] + [a - b for a, b in zip(near, near[1:]) if a != b])
            keep = set(order[:topk_group])
            allowed = [e for e in allowed if e // size in keep]
        order = sorted(allowed, key=lambda e: (-row[e], e))
        gap = min(gap, smallest([row[e] for e in order]))
        ids[t] = torch.tensor(order[:topk], dtype=torch.int32)
        w[t] = s[t, order[:topk]]
        if renorm:
            w[t] /= w[t].sum() + 1e-20
    return ids, w * scale, gap


ROUTES = [
    # m, E, topk, score, bias, groups, topk_group, renorm, scale, dtype
    (1, 256, 8, "sigmoid", True, 8, 4, True, 2.5, torch.float32),
    (33, 256, 8, "softmax", False, 1, 1, True, 1.0, torch.float32),
    (5, 8, 2, "softmax", False, 1, 1, False, 1.0, torch.float32),
    (7, 64, 6, "softmax", True, 8, 3, False, 16.0, torch.float32),
    (7, 160, 6, "softmax", False, 8, 3, True, 1.0, torch.float32),
    (9, 100, 5, "sigmoid", True, 4, 2, True, 1.0, torch.float32),
    (3, 1, 1, "sigmoid", False, 1, 1, True, 1.0, torch.float32),
    (3, 32, 32, "softmax", False, 1, 1, True, 1.0, torch.float32),
    (4, 32, 4, "sigmoid", True, 32, 7, True, 1.0, torch.float32),
    (6, 1024, 32, "softmax", False, 32, 9, True, 1.0, torch.float32),
    (6, 1000, 10, "sigmoid", True, 10, 3, True, 1.0, torch.float32),
    (4, 128, 4, "softmax", False, 1, 1, True, 1.0, torch.bfloat16),
    (130, 512, 8, "sigmoid", False, 1, 1, True, 1.0, torch.float32),
]


@pytest.mark.parametrize("case", ROUTES, ids=lambda c: "-".join(map(str, c[:9])))
def test_route(lib, case):
    m, E, topk, score, with_bias, groups, topk_group, renorm, scale, dtype = case
    # logits a permutation of a fine grid, so that scores differ by far more than fp32 rounds
    g = gen(E + topk)
    rank = torch.stack([torch.randperm(E, generator=g, device=DEV) for _ in range(m)]).float()
    x = ((rank + 0.5) / E * 4 - 2).to(dtype)
    bias = None
    if with_bias:
        bias = normal(g, E, std=0.05)
    ids, w, gap = route_64(x, topk, bias, score, groups, topk_group, renorm, scale)
    got_ids, got_w = lib.moe_route_topk(x, topk, bias=bias, score=score, n_group=groups, topk_group=topk_group,
                                        renorm=renorm, scale=scale)
    if gap > 4e-7:  # scores and biases are below 2: fp32 places every sum within 2.4e-7
        assert torch.equal(got_ids.cpu(), ids)
        within(got_w.cpu(), w, 2.0 ** -20 * w.abs(), "weights")
    else:  # a near tie may fall either way; the scores chosen may not differ by more than that
        assert torch.allclose(got_w.sum(-1).cpu().double(), w.sum(-1), rtol=1e-5)
        assert (got_ids.cpu() == ids).float().mean() > 0.97


def test_route_ties_masked_experts_and_empty_rows(lib):
    E, k = 64, 4
    x = torch.zeros(6, E, device=DEV)
    x[1, 10:20] = 1.0                      # ties: lowest indexes
    x[2] = -math.inf
    x[2, 40], x[2, 7] = 0.5, 0.25          # two experts left of 64
    x[3] = -math.inf                       # none left
    x[4] = float("nan")
    x[4, 5] = 1.0
    x[5, 9] = math.inf
    ids, w = lib.moe_route_topk(x, k)
    ids, w = ids.tolist(), w.tolist()
    assert ids[0] == [0, 1, 2, 3] and w[0] == [0.25] * 4
    assert ids[1] == [10, 11, 12, 13]
    assert ids[2] == [40, 7, 0, 1] and w[2][2:] == [0, 0] and abs(w[2][0] - 1 / (1 + math.exp(-0.25))) < 1e-6
    assert ids[3] == [0, 1, 2, 3] and w[3] == [0, 0, 0, 0]
    assert ids[4] == [5, 0, 1, 2] and w[4] == [1, 0, 0, 0]
    assert ids[5] == [9, 0, 1, 2] and w[5] == [1, 0, 0, 0]
    ids, w = lib.moe_route_topk(x[3:4], k, score="sigmoid", bias=torch.arange(E, device=DEV, dtype=torch.float32))
    assert ids.tolist() == [[63, 62, 61, 60]] and w.tolist() == [[0, 0, 0, 0]]
    # a group of one expert scores by it alone; whole groups of -inf bias go last
    bias = torch.zeros(E, device=DEV)
    bias[:32] = -math.inf
    ids, _ = lib.moe_route_topk(x[:1], k, bias=bias, score="sigmoid", n_group=2, topk_group=1)
    assert ids.tolist() == [[32, 33, 34, 35]]


def test_route_strided_logits_and_pointer_tables(lib):
    E, k, m = 96, 3, 5
    g = gen(21)
    wide = normal(g, m, E + 7)
    base = torch.arange(3 * E, dtype=torch.int64, device=DEV).view(3, E) * 1000
    ids, w, ptrs = lib.moe_route_topk(wide[:, 3:3 + E], k, expert_ptrs=base)
    dense = lib.moe_route_topk(wide[:, 3:3 + E].contiguous(), k)
    assert torch.equal(ids, dense[0]) and torch.equal(w, dense[1])
    want = torch.cat([base[i][ids.long()] for i in range(3)], dim=1)
    assert torch.equal(ptrs, want)
    ids, w = lib.moe_route_topk(wide[:0, :E], k)
    assert ids.shape == (0, k)


# ---- together --------------------------------------------------------------------

def test_one_layer_prompt_decode_and_replay():
    """The example's layer at small sizes: prompts of uneven length, decode, and a captured decode step whose
    lengths, pages and positions move on the device alone."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_layer.py")
    spec = importlib.util.spec_from_file_location("decode_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    layer = example.Layer(dim=1024, hq=8, hkv=2, d=128, experts=16, groups=4, topk=4, inter=512, requests=3,
                          max_len=128)
    history = [[torch.empty((0, 2, 128), dtype=torch.bfloat16, device=DEV)] * 2 for _ in range(3)]
    # the library's bars: q8_1 activations 1e-2, bf16 matmuls 2e-3 of the result; the experts quantise twice
    bars = {"projections": 1e-2, "attention": 5e-3, "out projection": 1e-2, "norms": 4e-3, "route": 0.0,
            "route weights": 1e-6, "experts": 2e-2, "stream": 1e-6}

    def held(s):
        far = example.check(layer, s, history)
        assert all(far[name] <= bars[name] for name in bars), far

    g = gen(31)
    held(layer.step(normal(g, 24, 1024), i32([17, 0, 7])))   # more than 8 tokens: the matmul's projections
    held(layer.step(normal(g, 5, 1024), i32([1, 3, 1])))
    stream, one = normal(g, 3, 1024), i32([1, 1, 1])
    held(layer.step(stream, one))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = layer.step(stream, one)
    for _ in range(10):  # across page boundaries
        stream.copy_(normal(g, 3, 1024))
        graph.replay()
        torch.cuda.synchronize()
        held(s)
    assert layer.ctx.tolist() == [17 + 1 + 11, 3 + 11, 8 + 11]
