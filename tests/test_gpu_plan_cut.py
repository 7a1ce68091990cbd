"""kv_page_plan with more new tokens than max_tokens: the plan of the tokens
that are kept, whole in itself, so that the rest can go in the next step."""
import pytest
import torch

from test_gpu_layer_ops import (DEV, Cache, attention_64, check_attention, gen, i32, lib, normal,  # noqa: F401
                                plan_by_hand)

pytestmark = pytest.mark.gpu


def kept_of(new, max_tokens):
    kept, left = [], max_tokens
    for n in new:
        kept.append(min(max(n, 0), left))
        left -= kept[-1]
    return kept


CUTS = {
    # cached, new, page, table columns, free pages, head, max_tokens
    "inside-a-request": ([3, 3, 3], [10, 10, 10], 16, 4, 20, 0, 17),
    "between-requests": ([3, 3, 3], [10, 10, 10], 16, 4, 20, 2, 20),
    "nothing-kept": ([30, 16], [5, 90], 16, 8, 20, 1, 0),
    "idle-and-new": ([0, 40, 0, 7], [0, 1, 50, 60], 32, 4, 9, 0, 33),
    # what was cut would have outgrown its row, or the pool
    "row-long-enough": ([10, 60], [20, 900], 16, 6, 30, 0, 40),
    "pool-large-enough": ([10, 0], [20, 900], 16, 60, 6, 1, 60),
    "row-too-short-all-the-same": ([10, 60], [20, 900], 16, 4, 30, 0, 40),
    "negative": ([-5, 20, 6], [3, -2, 300], 16, 20, 10, -1, 10),
}


@pytest.mark.parametrize("name", CUTS)
def test_a_cut_plan_is_the_plan_of_what_is_kept(lib, name):  # noqa: F811
    ctx, new, page, ld, n_free, head, max_tokens = CUTS[name]
    table = [[1000 + 10 * r + c if c < -(-max(x, 0) // page) else -7 for c in range(ld)] for r, x in enumerate(ctx)]
    free = [500 - 3 * i for i in range(n_free)]
    want = plan_by_hand(ctx, kept_of(new, max_tokens), page, free, head, table, max_tokens)
    want = want[:-1] + (want[-1] | 8 | (4 if min(new) < 0 else 0),)
    dt, err = i32(table), i32([0])
    p = lib.kv_page_plan(i32(ctx), i32(new), page, i32(free), dt, max_tokens, free_head=i32([head]), err_flag=err)
    got = (dt.tolist(), p.cu_q.tolist(), p.seq_lens.tolist(), p.positions.tolist(), p.token_req.tolist(),
           p.slot_map.tolist(), p.free_head.item(), err.item())
    assert got == want


@pytest.mark.parametrize("n_req, max_tokens", [(513, 3000), (2500, 5000), (2500, 1), (16384, 200000)])
def test_a_cut_plan_of_many_requests(lib, n_req, max_tokens):  # noqa: F811
    page, ld = 16, 6
    cpu = torch.Generator().manual_seed(n_req + max_tokens)
    ctx = torch.randint(0, 40, (n_req,), generator=cpu).tolist()
    new = torch.randint(0, 30, (n_req,), generator=cpu).tolist()
    assert sum(new) > max_tokens
    table = [[100000 + r * ld + c for c in range(ld)] for r in range(n_req)]
    free = list(range(3 * n_req + 5))
    want = plan_by_hand(ctx, kept_of(new, max_tokens), page, free, 0, table, max_tokens)
    dt = i32(table)
    p = lib.kv_page_plan(i32(ctx), i32(new), page, i32(free), dt, max_tokens)
    assert dt.tolist() == want[0] and p.cu_q.tolist() == want[1] and p.seq_lens.tolist() == want[2]
    assert p.positions.tolist() == want[3] and p.token_req.tolist() == want[4] and p.slot_map.tolist() == want[5]
    assert p.free_head.item() == want[6]


def test_steps_of_a_cut_plan_cover_the_prompt(lib):  # noqa: F811
    """A step too large for its arrays, run as the plans say until nothing is left: store and attention agree on the
    positions, no row reads a slot that no token was stored in, and the result is that of the whole."""
    Hq, Hkv, D, page, max_tokens = 4, 2, 64, 16, 60
    ctx, new = [3, 40, 0, 17], [10, 75, 0, 30]
    g = gen(12)
    seq = [c + n for c, n in zip(ctx, new)]
    whole = Cache(g, seq, Hkv, D, page)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = normal(g, cu[-1], Hq, D, dtype=torch.bfloat16)
    want = attention_64(q, whole.keys, whole.values, cu, seq, D ** -0.5, 0)
    kc, vc = (torch.full((24, Hkv, page, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table = torch.full((4, 8), -1, dtype=torch.int32, device=DEV)
    free, still = i32(torch.randperm(24, generator=torch.Generator().manual_seed(5)).tolist()), torch.zeros(D // 2, device=DEV)

    def store(plan, rows):
        """The kept tokens' K and V; angles of zero leave them as they are."""
        k, v = (torch.cat([x[r][a:b] for r, (a, b) in enumerate(rows)]) for x in (whole.keys, whole.values))
        pad = plan.slot_map.numel() - len(k)
        k, v = (torch.cat([x, torch.zeros(pad, Hkv, D, dtype=x.dtype, device=DEV)]) for x in (k, v))
        lib.kv_rope_store(None, k, v, plan.positions, still, plan.slot_map, kc, vc)

    plan = lib.kv_page_plan(i32([0] * 4), i32(ctx), page, free, table, max_tokens)
    store(plan, [(0, c) for c in ctx])
    head, at = plan.free_head, list(ctx)
    got, lse = torch.zeros_like(q), torch.zeros(cu[-1], Hq, device=DEV)
    steps = 0
    while at != seq:
        left = [s - a for s, a in zip(seq, at)]
        kept = kept_of(left, max_tokens)
        err = i32([0])
        plan = lib.kv_page_plan(i32(at), i32(left), page, free, table, max_tokens, free_head=head, err_flag=err)
        assert err.item() == (8 if sum(left) > max_tokens else 0)
        store(plan, [(a, a + n) for a, n in zip(at, kept)])
        rows = torch.cat([torch.arange(cu[r] + a - ctx[r], cu[r] + a - ctx[r] + n) for r, (a, n) in
                          enumerate(zip(at, kept))])
        x = torch.zeros(max_tokens, Hq, D, dtype=torch.bfloat16, device=DEV)
        x[:len(rows)] = q[rows.to(DEV)]
        o, z = lib.kv_attention_bf16(x, kc, vc, table, plan.cu_q, plan.seq_lens, want_lse=True)
        got[rows.to(DEV)], lse[rows.to(DEV)] = o[:len(rows)], z[:len(rows)]
        head, at = plan.free_head, plan.seq_lens.tolist()
        steps += 1
        assert steps < 5, at
    assert steps == 2
    check_attention(got, lse, want)


def test_a_request_that_outgrows_a_strided_table(lib):  # noqa: F811
    """Columns past the row's own belong to someone else, whatever the stride."""
    page, ld, ctx, new = 16, 4, [10, 60, 100], [40, 20, 3]
    table = [[1000 + 10 * r + c if c < -(-x // page) else -7 for c in range(ld)] for r, x in enumerate(ctx)]
    free = [500 - 3 * i for i in range(40)]
    want = plan_by_hand(ctx, new, page, free, 0, table, 63)
    wide, err = torch.full((3, ld + 5), -9, dtype=torch.int32, device=DEV), i32([0])
    wide[:, :ld] = i32(table)
    p = lib.kv_page_plan(i32(ctx), i32(new), page, i32(free), wide[:, :ld], 63, err_flag=err)
    assert wide[:, :ld].tolist() == want[0] and (wide[:, ld:] == -9).all()
    assert p.slot_map.tolist() == want[5] and p.free_head.item() == want[6] and err.item() == want[7] == 2


def test_plan_arrays_side_by_side_and_over_one_another(lib):  # noqa: F811
    """Inputs and outputs in one buffer, back to back, are fine; the lengths updated in place are refused."""
    ctx, new, page, free = [3, 16, 40], [5, 0, 9], 16, list(range(50, 70))
    want = plan_by_hand(ctx, new, page, free, 2, [[7, -7, -7, -7], [8, -7, -7, -7], [1, 2, 3, -7]], 15)
    sizes = (3, 3, 20, 1, 4, 3, 15, 15, 15, 1)  # ctx, new, free, head, cu_q .. free_head
    buf = torch.full((sum(sizes),), -77, dtype=torch.int32, device=DEV)
    a, b, pool, head, *out = buf.split_with_sizes(sizes)
    for x, v in ((a, ctx), (b, new), (pool, free), (head, [2])):
        x.copy_(i32(v))
    table = i32([[7, -7, -7, -7], [8, -7, -7, -7], [1, 2, 3, -7]])
    out = lib.PagePlan._make(out)
    p = lib.kv_page_plan(a, b, page, pool, table, 15, free_head=head, out=out)
    got = (table.tolist(), p.cu_q.tolist(), p.seq_lens.tolist(), p.positions.tolist(), p.token_req.tolist(),
           p.slot_map.tolist(), p.free_head.item())
    assert got == want[:-1] and a.tolist() == ctx and b.tolist() == new
    for wrong in (out._replace(seq_lens=a), out._replace(seq_lens=b), out._replace(free_head=head)):
        with pytest.raises(lib.Q2KError):
            lib.kv_page_plan(a, b, page, pool, table, 15, free_head=head, out=wrong)
