"""fp8_moe where a block of 128 values spans far more than a value's 8 bits:
each bf16 value enters as it is if it is within 2^-30 of the largest of its
block, else off by less than 2^-37 of that.

Tolerances as in test_gpu_fp8.py, with 2^-37 in the place of 2^-20.
"""
import pytest
import torch

from test_gpu_fp8 import BF16, DEV, F32, TINY, U, blocks, codes, gen, lib, normal, scales, spread, within  # noqa: F401

pytestmark = pytest.mark.gpu

PART = 2.0 ** -37


def largest(v):
    """Of each value's block of 128."""
    n = v.shape[1]
    top = torch.nn.functional.pad(v.abs(), (0, -n % 128)).view(v.shape[0], -1, 128).amax(-1)
    return top.repeat_interleave(128, 1)[:, :n]


def want_of(x, ids, route_w, gate_up, gs, down, ds, rounded=2.0 ** -8):
    E, _, inter, dim = gate_up.shape
    want, tol, size = (torch.zeros(x.shape, dtype=torch.float64, device=DEV) for _ in range(3))
    per_up, per_down = (128 + blocks(dim) + 8) * U, (128 + blocks(inter) + 8) * U
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        a = x[t].double()
        off = largest(a) * PART + TINY
        (g, dg), (u, du) = ((a @ w.t(), a.abs() @ w.abs().t() * per_up + off @ w.abs().t())
                            for w in (gate_up[e, i].double() * spread(gs[e, i], inter, dim) for i in (0, 1)))
        s = g * torch.sigmoid(g)
        h = s * u
        dh = 1.1 * dg * u.abs() + s.abs() * du + 1.1 * dg * du
        dh = dh + (h.abs() + dh) * (rounded + 2.0 ** -20) + TINY
        w = down[e].double() * spread(ds[e], dim, inter)
        r = route_w[t, j].double()[:, None]
        want.index_add_(0, t, r * (h @ w.t()))
        dh = dh + largest(h.abs() + dh) * PART
        part = (h.abs() + dh) @ w.abs().t()
        tol.index_add_(0, t, r.abs() * (dh @ w.abs().t() + part * per_down))
        size.index_add_(0, t, r.abs() * part)
    return want, tol + size * (ids.shape[1] + 2) * U + TINY


def inputs(seed, m, E, topk, dim, inter):
    g = gen(seed)
    gate_up, down = codes(g, E, 2, inter, dim), codes(g, E, dim, inter)
    gs, ds = scales(g, E, 2, blocks(inter), blocks(dim)), scales(g, E, blocks(dim), blocks(inter))
    x = normal(g, m, dim, dtype=BF16)
    ids = torch.stack([torch.randperm(E, generator=g, device=DEV)[:topk] for _ in range(m)]).to(torch.int32)
    return [x, ids, torch.rand(m, topk, generator=g, device=DEV) + 0.1, gate_up, gs, down, ds]


SIZES = [(1, 4, 2, 256, 128), (2, 2, 2, 272, 400), (5, 8, 3, 512, 384), (8, 1, 1, 144, 256), (13, 4, 2, 1040, 272), (20, 2, 2, 400, 528),
         (3, 4, 2, 10240, 128), (40, 2, 1, 384, 144)]


@pytest.mark.parametrize("far", [2.0 ** 12, 2.0 ** 18, 2.0 ** 25, 2.0 ** 31])
@pytest.mark.parametrize("m,E,topk,dim,inter", SIZES)
def test_moe_of_a_channel_far_above_the_others_whose_weights_are_zero(lib, m, E, topk, dim, inter, far):  # noqa: F811
    """What is left of y comes from the values far below."""
    args = inputs(m + dim, m, E, topk, dim, inter)
    x, gate_up = args[0], args[3]
    for b in range(0, dim, 128):
        x[:, b + b // 128 % min(128, dim - b)] *= far
        gate_up[:, :, :, b + b // 128 % min(128, dim - b)] = 0
    x[0, : min(dim, 128)] = x[0, : min(dim, 128)] / far  # (one block whose values are all far below the next one's)
    args[4] /= dim ** 0.5
    args[6] /= inter ** 0.5
    want, tol = want_of(*args)
    within(lib.fp8_moe(*args), want, tol)


@pytest.mark.parametrize("far", [2.0 ** 8, 2.0 ** 12, 2.0 ** 15])
@pytest.mark.parametrize("m,E,topk,dim,inter", SIZES)
def test_moe_of_an_h_far_above_the_others_whose_weights_are_zero(lib, m, E, topk, dim, inter, far):  # noqa: F811
    """Rows of gate and up that make one h of a block about far^2 times the others."""
    args = inputs(m + inter, m, E, topk, dim, inter)
    gate_up, gs, down = args[3:6]
    quarter = codes(gen(5), E, 2, inter, dim, std=120.0 / far)  # (codes down to 2^-9)
    gate_up.copy_(torch.where((quarter.float() == 0), torch.full_like(quarter.float(), 2.0 ** -9), quarter.float()))
    at = torch.arange(0, inter, 128, device=DEV) + 7
    gate_up[:, :, at] = codes(gen(6), E, 2, len(at), dim, std=120.0)
    gs.fill_(4.0 / (120.0 * dim ** 0.5))
    down[:, :, at] = 0
    args[6] /= inter ** 0.5
    want, tol = want_of(*args)
    within(lib.fp8_moe(*args), want, tol)


@pytest.mark.parametrize("m,E,topk,dim,inter", SIZES)
def test_moe_of_rows_with_values_of_every_size(lib, m, E, topk, dim, inter):  # noqa: F811
    """Exponents over 40 binades; some tokens plain, some with one such value a row."""
    args = inputs(m * 3 + dim, m, E, topk, dim, inter)
    x, g = args[0], gen(m)
    spans = torch.exp2(torch.floor(torch.rand(m, dim, generator=g, device=DEV) * -40))
    spans[::3] = 1
    spans[1::3] = torch.where(torch.arange(dim, device=DEV) == dim // 2, 2.0 ** -20, 1.0)
    x.copy_(x.float() * spans)
    args[4] /= dim ** 0.5
    args[6] /= inter ** 0.5
    want, tol = want_of(*args)
    y = lib.fp8_moe(*args)
    within(y, want, tol)
    assert torch.equal(y, lib.fp8_moe(*args))


def test_moe_of_a_wide_block_beside_nan(lib):  # noqa: F811
    """A token with a NaN, one with an infinity and one whose values span far, in one pass."""
    args = inputs(9, 3, 1, 1, 256, 128)
    args[0][0, 5], args[0][1, 130] = float("nan"), float("inf")
    args[0][2, ::2] *= 2.0 ** -20
    args[4] /= 16
    args[6] /= 11
    want, tol = want_of(args[0][2:], args[1][2:], args[2][2:], *args[3:])
    y = lib.fp8_moe(*args)
    assert torch.isnan(y[:2]).all()
    within(y[2:], want, tol)


@pytest.mark.parametrize("m,E,topk,dim,inter", [(1, 1, 1, 256, 16), (5, 4, 2, 144, 16), (3, 2, 1, 512, 32), (20, 2, 2, 272, 16), (40, 1, 1, 128, 48),
                                                (6, 8, 4, 1040, 16), (32, 64, 8, 4096, 16)])
def test_moe_keeps_eleven_bits_of_h(lib, m, E, topk, dim, inter):  # noqa: F811
    """Few h, so that what their rounding leaves does not average out."""
    args = inputs(m + 7 * dim, m, E, topk, dim, inter)
    args[4] /= dim ** 0.5
    args[6] /= inter ** 0.5
    want, tol = want_of(*args, rounded=2.0 ** -11)
    within(lib.fp8_moe(*args), want, tol)


@pytest.mark.parametrize("gate_scale,down_scale", [(2.0 ** -118, 2.0 ** -40), (2.0 ** -78, 2.0 ** -120), (2.0 ** -76, 2.0 ** -126)])
@pytest.mark.parametrize("m,E,topk,dim,inter", [(1, 1, 1, 256, 128), (3, 4, 2, 144, 272), (20, 2, 2, 272, 128)])
def test_moe_of_the_largest_tokens_and_h(lib, m, E, topk, dim, inter, gate_scale, down_scale):  # noqa: F811
    """x up to bf16's largest value, h up to 2^120 and beyond: the powers of two beside them stay in range."""
    args = inputs(m + inter, m, E, topk, dim, inter)
    g = gen(m)
    size = 0.5 + 0.5 * torch.rand(m, dim, generator=g, device=DEV)
    args[0].copy_(torch.sign(args[0].float()) * size * 3.38e38)
    args[0][0, 0] = torch.finfo(BF16).max
    args[4].fill_(gate_scale / dim ** 0.5)
    args[6].fill_(down_scale / inter ** 0.5)
    want, tol = want_of(*args, rounded=2.0 ** -11)
    assert torch.isfinite(want).all() and want.abs().max() < 3e38
    within(lib.fp8_moe(*args), want, tol)
