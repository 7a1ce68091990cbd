"""norm_gate_residual with squares near and past fp32's range, and
moe_route_topk where its sums lie close together: every choice that 64 bits
decide by more than fp32's roundings has to be that one."""
import pytest
import torch

from test_gpu_layer_ops import DEV, HALF_ULP, TYPES, gen, lib, norm_64, normal, route_64, within  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 255, 4096, 8200])  # runs of 8 values, value by value
@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("post", [False, True])
def test_norm_of_huge_values(lib, dim, types, post):  # noqa: F811
    """Rows of about 1e16 have squares in range and are as any others; those of 1e21 have not: their rms is infinite
    in fp32, and the normed row is zero, beside rows that are not touched by that."""
    g = gen(dim)
    y_type, s_type = (TYPES[t] for t in types)
    size = torch.tensor([1.0, 1e16, 1e21, 1e16, 1e-3], device=DEV)[:, None]
    res = (normal(g, 5, dim) * size).to(s_type)
    y = (normal(g, 5, dim) * size).to(y_type)
    pre = 1 + normal(g, dim, std=0.1)
    h, n = lib.norm_gate_residual(res, pre, 1e-6, y=y, post_w=pre if post else None, alpha=0.5)
    h64, n64, hs, ns = norm_64(res, y, pre if post else None, None, 0.5, pre, 1e-6)
    if post:  # the normed y of row 2 is zero
        h64[2] = res[2].double()
        hs[2] = h64[2].abs()
    n64[2] = 0
    ns[2] = 0
    within(h, h64, 2.0 ** -20 * hs + (HALF_ULP * h64.abs() if types[1] == "bf16" else 0), "stream")
    within(n, n64, 2.0 ** -18 * ns + HALF_ULP * n64.abs(), "normed")


CLOSE = [
    # m, E, topk, groups, topk_group, renorm
    (6, 1024, 32, 32, 9, True),
    (6, 1024, 32, 32, 9, False),
    (40, 1024, 8, 16, 4, False),
    (12, 1000, 10, 10, 3, False),
    (30, 512, 6, 1, 1, True),
    (30, 1024, 16, 1, 1, False),
]


@pytest.mark.parametrize("case", CLOSE, ids=lambda c: "-".join(map(str, c)))
def test_route_decides_by_small_gaps(lib, case):  # noqa: F811
    """Softmax scores of hundreds of experts are small, and so are the gaps that decide.  A score is good to 2^-22
    (the exponential's 2 units, one division) and a sum of two to 2^-21 of itself, so gaps above 2^-20 of the largest
    sum decide as in 64 bits."""
    m, E, topk, groups, topk_group, renorm = case
    g = gen(E + topk + groups)
    rank = torch.stack([torch.randperm(E, generator=g, device=DEV) for _ in range(m)]).float()
    x = (rank + 0.5) / E * 4 - 2
    ids, w, gap = route_64(x, topk, None, "softmax", groups, topk_group, renorm, 1.0)
    largest = torch.softmax(x.double(), -1).max().item() * (2 if groups > 1 else 1)
    assert gap > 2.0 ** -20 * largest  # of the inputs: no choice is a matter of rounding
    got_ids, got_w = lib.moe_route_topk(x, topk, n_group=groups, topk_group=topk_group, renorm=renorm)
    assert torch.equal(got_ids.cpu(), ids)
    within(got_w.cpu(), w, 2.0 ** -20 * w.abs(), "weights")


@pytest.mark.parametrize("T, dim", [(3, 4096), (700, 2880), (3, 1001), (900, 64)])  # few and many rows, value by value
def test_norm_without_some_of_its_outputs(lib, T, dim):  # noqa: F811
    """The C call takes NULL for outputs that are not wanted; the others have the bits that they have beside them."""
    g = gen(T + dim)
    res, y, post, pre = normal(g, T, dim), normal(g, T, dim), normal(g, dim), normal(g, dim)
    q8 = dim % 32 == 0
    want = lib.norm_gate_residual(res, pre, 1e-6, y=y, post_w=post, alpha=0.5, want_q8=q8)
    stream = torch.cuda.current_stream().cuda_stream
    for keep in ((0,), (1,), (2,), (0, 1), (1, 2), (0, 2)):
        if 2 in keep and not q8:
            continue
        got = [torch.full_like(w, 1) if i in keep else None for i, w in enumerate(want)] + [None] * (not q8)
        h, n, e = (None if t is None else t.data_ptr() for t in got)
        assert lib.lib().norm_gate_residual(y.data_ptr(), 0, dim, post.data_ptr(), None, 0, res.data_ptr(), 0, dim, 0.5,
                                            pre.data_ptr(), 1e-6, T, dim, h, dim, n, dim, e, stream) == 0
        for i in keep:
            assert torch.equal(got[i], want[i]), (keep, i)
