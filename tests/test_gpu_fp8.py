"""The calls with 8-bit floating-point operands against plain 64-bit
computations of the same formulas: fp8_quantize, swiglu_fp8_rows, fp8_gemm,
fp8_moe, and a feed-forward half of a layer that runs them together.

Tolerances come from the roundings the calls state (S = the sum of the
products' absolute values, with their scales):
  * codes and scales of fp8_quantize follow from single fp32 operations, so
    they are equal;
  * a block's 128 products are added in fp32, each addition off by at most
    2^-23 of the sum so far (whatever its rounding), then scaled and added to
    the other blocks: (128 + blocks + 4) * 2^-23 * S;
  * bf16 results: 2^-8 of the value more;
  * fp8_moe: x enters with at most 2^-20 of its block's largest value off, h
    is rounded to bf16 (2^-8); silu has a slope of at most 1.1, and what is
    off in g and u is carried through h and down with it.  fp32 has no normal
    values below 2^-126: x, h and what is made of them may be off by 2^-120
    each where they are near that, whatever their own size.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -23
TINY = 2.0 ** -120


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


def blocks(n):
    return -(-n // 128)


def normal(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def codes(g, *shape, std=60.0):
    return normal(g, *shape, std=std).clamp(-448, 448).to(E4M3)


def scales(g, *shape):
    return torch.exp(normal(g, *shape)) * 0.01


def spread(s, rows, cols):
    return s.double().repeat_interleave(128, -2)[..., :rows, :].repeat_interleave(128, -1)[..., :cols]


def guarded(rows, cols, dtype, extra=0, fill=7.0):
    """[rows, cols] inside a larger buffer of `fill`, rows cols + extra apart; and a check that the rest is untouched."""
    ld = cols + extra
    raw = torch.full((rows * ld + 64,), fill, dtype=F32, device=DEV).to(dtype)
    view = raw[32:32 + rows * ld].view(rows, ld)[:, :cols]

    def untouched():
        mask = torch.ones(raw.shape, dtype=torch.bool, device=DEV)
        mask[32:32 + rows * ld].view(rows, ld)[:, :cols] = False
        assert (raw.float()[mask] == fill).all()

    return view, untouched


def within(got, want, tol, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), what
    over = ((got - want).abs() - tol).max().item() if got.numel() else 0.0
    assert over <= 0, f"{what}: {over:.3e} beyond the tolerance"


# ---- fp8_quantize ------------------------------------------------------------------

def encode_on_host(x, block_rows):
    """The stated fp32 operations one by one, on the CPU."""
    x = x.float().cpu()
    rows, K = x.shape
    q, s = torch.empty((rows, K), dtype=E4M3), torch.empty(-(-rows // block_rows), blocks(K))
    for i in range(s.shape[0]):
        for b in range(s.shape[1]):
            at = (slice(i * block_rows, (i + 1) * block_rows), slice(b * 128, (b + 1) * 128))
            c = x[at].abs().max().clamp(min=448 * 2.0 ** -120)
            s[i, b] = c / 448
            q[at] = (x[at] * (c.reciprocal() * 448)).to(E4M3)
    return q, s


def same_codes(a, b):
    return torch.equal(a.view(torch.uint8).cpu(), b.view(torch.uint8).cpu())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,K,block_rows", [
    (1, 128, 1), (1, 1, 1), (3, 127, 1), (5, 129, 1), (7, 4096, 1), (33, 264, 1), (200, 72, 1), (2, 5000, 1),
    (300, 8, 1), (17, 2048, 1), (1, 1, 128), (127, 128, 128), (129, 130, 128), (257, 384, 128), (128, 1000, 128), (300, 77, 128)])
def test_quantize(lib, dtype, rows, K, block_rows):
    x = normal(gen(rows * K), rows, K, dtype=dtype) * torch.exp(2 * normal(gen(1), rows, 1)).to(dtype)
    q, s = lib.fp8_quantize(x, block_rows=block_rows)
    want_q, want_s = encode_on_host(x, block_rows)
    assert torch.equal(s.cpu(), want_s) and same_codes(q, want_q)
    # and what they stand for is within half a step of x: 2^-4 of it, or 2^-10 of the scale near zero
    up = s.double().repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :K]
    within(q.double() * up, x.double(), (x.double().abs() * 2.0 ** -4).maximum(up * 2.0 ** -10) * (1 + 2.0 ** -20))


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("offset,extra", [(0, 8), (1, 0), (3, 5), (8, 0)])
def test_quantize_strides_and_alignment(lib, offset, extra, block_rows):
    rows, K = 37, 392
    big = normal(gen(3), rows * (K + extra) + offset, dtype=BF16)
    x = big[offset:].view(rows, K + extra)[:, :K]
    out, untouched = guarded(rows, K, torch.uint8, extra=extra)
    q, s = lib.fp8_quantize(x, block_rows=block_rows, values=out.view(E4M3))
    want_q, want_s = encode_on_host(x, block_rows)
    assert torch.equal(s.cpu(), want_s) and same_codes(q.contiguous(), want_q)
    untouched()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_extremes(lib, dtype, block_rows):
    x = torch.zeros((6, 256), dtype=dtype, device=DEV)
    x[1, :128] = 3.0e38
    x[2, 5] = 1e-38
    x[3, 7], x[3, 200] = 1.0, -1e-30
    if block_rows == 128:
        x = x.repeat_interleave(128, 0)
    q, s = lib.fp8_quantize(x, block_rows=block_rows)
    want_q, want_s = encode_on_host(x, block_rows)
    assert torch.equal(s.cpu(), want_s) and same_codes(q, want_q)
    assert torch.isfinite(q.float()).all() and (q[x == 0].float() == 0).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("K", [384, 383])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_of_nan_and_infinity_marks_the_block(lib, bad, K, block_rows):
    x = normal(gen(5), 256, K)
    x[130, 140] = bad
    q, s = lib.fp8_quantize(x, block_rows=block_rows)
    hit = torch.zeros((256, K), dtype=torch.bool, device=DEV)
    hit[slice(128, 256) if block_rows == 128 else 130, 128:256] = True
    assert torch.equal(torch.isnan(q.float()), hit)
    assert torch.isnan(s).sum() == 1 and torch.isnan(s[1 if block_rows == 128 else 130, 1])


# ---- swiglu_fp8_rows ---------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,N,extra", [(1, 128, 0), (1, 1, 0), (9, 200, 0), (33, 2048, 0), (5, 131, 0), (40, 1520, 24), (300, 16, 0)])
def test_swiglu(lib, dtype, rows, N, extra):
    full = normal(gen(N), rows, 2 * N + extra, std=2.0, dtype=dtype)
    x = full[:, :2 * N]
    q, s = lib.swiglu_fp8_rows(x)
    g, u = x.double().chunk(2, -1)
    h = g * torch.sigmoid(g) * u
    up = s.double().repeat_interleave(128, 1)[:, :N]
    # h in fp32: 2^-22 for the power of two, 2^-23 for the reciprocal, 2^-24 for each of five roundings, 11 * 2^-24 in all;
    # the scale follows h's largest, then the division: 12 of the 16 * 2^-24 allowed
    pad = torch.nn.functional.pad(h.abs(), (0, -N % 128)).view(rows, -1, 128).amax(-1)
    within(s, pad / 448, pad / 448 * 2.0 ** -20)
    within(q.double() * up, h, (h.abs() * 2.0 ** -4).maximum(up * 2.0 ** -10) * (1 + 2.0 ** -10))


def test_swiglu_far_ends(lib):
    x = torch.tensor([[-1e30, -200.0, -100.0, 0.0, 100.0, 1e4, -0.0, 5.0] + [1.0, 2.0, 3.0, 4.0, 5.0, 6.0, 7.0, 8.0]], device=DEV)
    q, s = lib.swiglu_fp8_rows(x)
    h = (q.double() * s.double())[0]
    # the largest gets code 448 and reads as 448 times a scale of 6e4 / 448 that is rounded once
    assert torch.isfinite(h).all() and abs(h[5] - 6e4) <= 6e4 * 2.0 ** -24 and (h[[0, 1, 3, 6]] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", [16, 13])
def test_swiglu_of_small_gates_and_large_ups(lib, dtype, N):
    """e^-g near fp32's largest, up large: what is left is far from zero."""
    x = torch.cat([torch.linspace(-88.6, -86.0, N, device=DEV), torch.full((N,), 1e30, device=DEV)]).to(dtype)[None]
    q, s = lib.swiglu_fp8_rows(x)
    g, u = x.double().chunk(2, -1)
    h = g * torch.exp(g) / (1 + torch.exp(g)) * u
    # e^g may be below fp32's normal values, off by 2 units of 2^-149 of at least 2^-129 there: 2^-19
    within(q.double() * s.double(), h, (h.abs() * 2.0 ** -4).maximum(s.double() * 2.0 ** -10) * (1 + 2.0 ** -10))


# ---- fp8_gemm ----------------------------------------------------------------------

def gemm_want(x, xs, w, ws):
    a = x.double() * xs.double().repeat_interleave(128, -1)[:, :x.shape[1]]
    b = w.double() * spread(ws, *w.shape)
    return a @ b.t(), a.abs() @ b.abs().t()


def gemm_tol(want, size, K, dtype):
    return size * ((128 + blocks(K) + 4) * U) + (want.abs() * 2.0 ** -8 if dtype == BF16 else 0.0)


GEMM_SIZES = [
    *[(m, 96, 256) for m in (1, 2, 3, 7, 8, 9, 15, 16, 17, 24, 31, 32, 33, 48, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 300, 513)],
    *[(m, N, 384) for m in (1, 9, 40, 130) for N in (1, 2, 5, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 500, 1000)],
    *[(m, 160, K) for m in (1, 12, 30, 70, 256) for K in (16, 32, 48, 64, 112, 128, 144, 240, 256, 272, 512, 528, 640, 1024, 1040, 2064, 4096, 4112)],
    (8, 64, 131072), (20, 33, 65552), (3, 16, 65536), (1, 4096, 4096), (16, 2048, 16384), (8, 1024, 20480), (203, 5000, 4112), (1500, 1300, 1536), (32, 6000, 1040), (700, 128, 16400),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,N,K", GEMM_SIZES)
def test_gemm(lib, dtype, m, N, K):
    g = gen(m * 7 + N * 3 + K)
    x, xs, w, ws = codes(g, m, K), scales(g, m, blocks(K)), codes(g, N, K), scales(g, blocks(N), blocks(K))
    want, size = gemm_want(x, xs, w, ws)
    out, untouched = guarded(m, N, dtype)
    y = lib.fp8_gemm(x, xs, w, ws, out=out)
    within(y, want, gemm_tol(want, size, K, dtype))
    untouched()
    again = lib.fp8_gemm(x, xs, w, ws, out_dtype=dtype)
    assert torch.equal(again, y)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m", [1, 5, 16, 20, 33, 140])
def test_gemm_strides(lib, dtype, m):
    N, K = 133, 400
    g = gen(m)
    wide = torch.full((m, K + 48), math.nan, device=DEV).to(E4M3)
    x = wide[:, 16:16 + K]
    x.copy_(codes(g, m, K))
    xs = torch.full((m, blocks(K) + 3), math.nan, device=DEV)[:, 1:1 + blocks(K)]
    xs.copy_(scales(g, m, blocks(K)))
    w, ws = codes(g, N, K), scales(g, blocks(N), blocks(K))
    out, untouched = guarded(m, N, dtype, extra=3)
    y = lib.fp8_gemm(x, xs, w, ws, out=out)
    want, size = gemm_want(x, xs, w, ws)
    within(y, want, gemm_tol(want, size, K, dtype))
    untouched()


@pytest.mark.parametrize("m", [1, 16, 40, 200])
def test_gemm_nan_stays_in_its_row_and_column(lib, m):
    N, K = 300, 1168
    g = gen(9)
    x, xs, w, ws = codes(g, m, K), scales(g, m, blocks(K)), codes(g, N, K), scales(g, blocks(N), blocks(K))
    for k in (0, K - 1):
        wb = w.clone()
        wb.view(torch.uint8)[37, k] = 0x7f
        y = lib.fp8_gemm(x, xs, wb, ws)
        hit = torch.zeros_like(y, dtype=torch.bool)
        hit[:, 37] = True
        assert torch.equal(torch.isnan(y), hit)
        xb = x.clone()
        xb.view(torch.uint8)[m - 1, k] = 0xff
        y = lib.fp8_gemm(xb, xs, w, ws)
        hit = torch.zeros_like(y, dtype=torch.bool)
        hit[m - 1] = True
        assert torch.equal(torch.isnan(y), hit)
    xsb = xs.clone()
    xsb[0, -1] = math.inf
    y = lib.fp8_gemm(x, xsb, w, ws)
    assert not torch.isfinite(y[0]).any() and torch.isfinite(y[1:]).all()


@pytest.mark.parametrize("m", [1, 16, 200])
def test_gemm_all_codes_and_extreme_scales(lib, m):
    """Every finite code, the smallest and largest among them, and scales far from 1."""
    K, N = 256, 256
    c = torch.arange(256, dtype=torch.uint8, device=DEV)
    c[127], c[255] = 0, 0
    x = c.view(E4M3).repeat(m, 1)
    w = torch.stack([torch.roll(c, i) for i in range(N)]).view(E4M3)
    xs, ws = torch.full((m, 2), 2.0 ** 40, device=DEV), torch.full((2, 2), 2.0 ** -60, device=DEV)
    xs[:, 1] = 2.0 ** -20
    want, size = gemm_want(x, xs, w, ws)
    within(lib.fp8_gemm(x, xs, w, ws), want, gemm_tol(want, size, K, F32))


def test_gemm_of_no_rows(lib):
    z = torch.zeros((0, 128), device=DEV)
    assert lib.fp8_gemm(z.to(E4M3), z[:, :1], torch.zeros((4, 128), device=DEV).to(E4M3),
                        torch.zeros((1, 1), device=DEV)).shape == (0, 4)


def test_gemm_refuses(lib):
    z = torch.zeros((4, 256), device=DEV).to(E4M3)
    s = torch.zeros((4, 2), device=DEV)
    with pytest.raises(lib.Q2KError, match="shape"):
        lib.fp8_gemm(z[:, :136].contiguous(), s, z[:, :136].contiguous(), s[:1])
    with pytest.raises(lib.Q2KError, match="misaligned"):
        lib.fp8_gemm(z.view(-1)[8:8 + 512].view(2, 256), s[:2], z, s[:1])


# ---- fp8_moe -----------------------------------------------------------------------

def moe_inputs(seed, m, E, topk, dim, inter):
    g = gen(seed)
    gate_up = codes(g, E, 2, inter, dim)
    gs = scales(g, E, 2, blocks(inter), blocks(dim)) / math.sqrt(dim)
    down, ds = codes(g, E, dim, inter), scales(g, E, blocks(dim), blocks(inter)) / math.sqrt(inter)
    x = normal(g, m, dim, dtype=BF16) * torch.exp(normal(g, m, 1)).to(BF16)
    # few values far below the others
    x = torch.where(torch.rand(m, dim, generator=g, device=DEV) < 0.05, x * 2.0 ** -18, x)
    ids = torch.stack([torch.randperm(E, generator=g, device=DEV)[:topk] for _ in range(max(m, 1))])[:m].to(torch.int32)
    route_w = torch.rand(m, topk, generator=g, device=DEV) + 0.1
    return [x, ids, route_w, gate_up, gs, down, ds]


def moe_want(x, ids, route_w, gate_up, gs, down, ds, dtype):
    """The formula in 64 bits, and how far the call may be off."""
    E, _, inter, dim = gate_up.shape
    m = x.shape[0]
    want, tol, size = (torch.zeros((m, dim), dtype=torch.float64, device=DEV) for _ in range(3))
    per_up, per_down = (128 + blocks(dim) + 8) * U, (128 + blocks(inter) + 8) * U
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        a = x[t].double()
        top = torch.nn.functional.pad(a.abs(), (0, -dim % 128)).view(len(t), -1, 128).amax(-1)
        off = top.repeat_interleave(128, 1)[:, :dim] * 2.0 ** -20 + TINY
        (g, dg), (u, du) = ((a @ w.t(), a.abs() @ w.abs().t() * per_up + off @ w.abs().t())
                            for w in (gate_up[e, i].double() * spread(gs[e, i], inter, dim) for i in (0, 1)))
        s = g * torch.sigmoid(g)
        h = s * u
        dh = 1.1 * dg * u.abs() + s.abs() * du + 1.1 * dg * du
        dh = dh + (h.abs() + dh) * (2.0 ** -8 + 2.0 ** -20) + TINY
        w = down[e].double() * spread(ds[e], dim, inter)
        r = route_w[t, j].double()[:, None]
        want.index_add_(0, t, r * (h @ w.t()))
        # h in bf16 enters as it is, but for what is far below its block's largest
        top = torch.nn.functional.pad(h.abs() + dh, (0, -inter % 128)).view(len(t), -1, 128).amax(-1)
        dh = dh + top.repeat_interleave(128, 1)[:, :inter] * 2.0 ** -20
        part = (h.abs() + dh) @ w.abs().t()
        tol.index_add_(0, t, r.abs() * (dh @ w.abs().t() + part * per_down))
        size.index_add_(0, t, r.abs() * part)
    tol = tol + size * (ids.shape[1] + 2) * U + TINY
    return want, tol + ((want.abs() + tol) * 2.0 ** -8 if dtype == BF16 else 0.0)


def moe_check(lib, args, dtype, what=""):
    out, untouched = guarded(args[0].shape[0], args[0].shape[1], dtype)
    y = lib.fp8_moe(*args, out=out)
    want, tol = moe_want(*args, dtype)
    within(y, want, tol, what)
    untouched()
    return y


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,E,topk,dim,inter", [
    (1, 8, 2, 256, 128), (1, 1, 1, 16, 16), (1, 4, 4, 128, 256), (2, 8, 2, 272, 144), (3, 16, 3, 144, 272),
    (4, 8, 8, 512, 384), (5, 8, 2, 1040, 528), (8, 32, 4, 640, 768), (9, 4, 2, 384, 256), (16, 64, 6, 1024, 512),
    (17, 3, 2, 400, 208), (33, 8, 2, 256, 640), (64, 16, 4, 128, 128), (128, 8, 8, 256, 256), (40, 1, 1, 528, 272),
    (128, 1, 1, 256, 256), (32, 64, 32, 128, 128), (7, 1024, 8, 64, 32), (1, 4, 2, 4096, 2048), (6, 16, 4, 2880, 1520),
    (2, 2, 1, 16384, 128), (2, 2, 1, 128, 16384), (20, 2, 1, 16384, 32), (20, 2, 1, 32, 16384), (3, 4, 2, 32, 48),
    (128, 2, 1, 16384, 64), (3, 4, 2, 9744, 160), (32, 8, 8, 256, 256), (33, 8, 8, 256, 128), (43, 16, 6, 144, 272)])
def test_moe(lib, dtype, m, E, topk, dim, inter):
    args = moe_inputs(m * 31 + E, m, E, topk, dim, inter)
    y = moe_check(lib, args, dtype)
    assert torch.equal(lib.fp8_moe(*args, out_dtype=dtype), y)


def test_moe_ids_that_count_nothing(lib):
    args = moe_inputs(3, 9, 8, 3, 272, 256)
    ids = args[1]
    ids[0], ids[4, 1], ids[5, 0], ids[8] = -1, -1, 8, -1
    ids[6, 2] = 2 ** 31 - 1
    args[2][0] = math.nan  # nothing reads it
    y = moe_check(lib, [args[0], ids, torch.where((ids < 0) | (ids >= 8), 0.0, args[2]), *args[3:]], F32)
    z = lib.fp8_moe(*args)
    assert torch.equal(z, y) and (y[[0, 8]] == 0).all()
    ids.fill_(-1)
    for dtype in (F32, BF16):
        out, untouched = guarded(9, 272, dtype)
        assert (lib.fp8_moe(*args, out=out) == 0).all()
        untouched()


def test_moe_the_same_expert_twice(lib):
    args = moe_inputs(4, 5, 4, 3, 256, 144)
    args[1][:, 1] = args[1][:, 0]
    args[1][2] = 3
    moe_check(lib, args, F32)


def test_moe_one_expert_for_all(lib):
    """More tokens on one expert than one pass takes, the other experts idle."""
    for m in (15, 16, 17, 32, 33, 100):
        args = moe_inputs(m, m, 6, 2, 272, 400)
        args[1][:, 0], args[1][:, 1] = 5, torch.arange(m, device=DEV) % 2
        moe_check(lib, args, F32, m)


def test_moe_strides(lib):
    args = moe_inputs(8, 6, 8, 2, 272, 144)
    raw = torch.full((6 * 293 + 1,), math.nan, dtype=BF16, device=DEV)
    x = raw[1:].view(6, 293)[:, 3:275]  # rows on odd addresses
    x.copy_(args[0])
    out, untouched = guarded(6, 272, BF16, extra=5)
    y = lib.fp8_moe(x, *args[1:], out=out)
    assert torch.equal(y, lib.fp8_moe(*args, out_dtype=BF16))
    untouched()


def test_moe_nan_and_infinity_stay_with_their_token(lib):
    args = moe_inputs(2, 5, 2, 2, 256, 256)
    good = lib.fp8_moe(*args)
    args[0][1, 200] = math.nan
    args[0][3, 0] = -math.inf
    y = lib.fp8_moe(*args)
    assert torch.isnan(y[[1, 3]]).all() and torch.equal(y[[0, 2, 4]], good[[0, 2, 4]])


def test_moe_extreme_inputs(lib):
    """Rows of zeros, of the smallest and of large values."""
    args = moe_inputs(6, 5, 4, 2, 256, 128)
    args[0][0] = 0
    args[0][1] = 1e-38
    args[0][2] *= 2.0 ** 60
    args[0][3, 128:] = 0
    args[4].mul_(2.0 ** -30)
    moe_check(lib, args, F32)


def test_moe_of_no_tokens(lib):
    args = moe_inputs(6, 0, 4, 2, 256, 128)
    assert lib.fp8_moe(*args).shape == (0, 256)


def test_moe_uses_any_workspace(lib):
    """What the workspace holds before a call does not matter."""
    args = moe_inputs(12, 12, 16, 4, 256, 384)
    need = lib.fp8_moe_workspace_bytes(12, 4, 256, 384)
    ys = [lib.fp8_moe(*args, workspace=torch.full((need,), fill, dtype=torch.uint8, device=DEV)) for fill in (0, 255, 127)]
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


# ---- streams and graphs ------------------------------------------------------------

def ffn(lib, x, w1, s1, w2, s2, logits, experts):
    """A dense block on 8-bit weights beside the routed experts."""
    q, qs = lib.fp8_quantize(x)
    h, hs = lib.swiglu_fp8_rows(lib.fp8_gemm(q, qs, w1, s1, out_dtype=BF16))
    dense = lib.fp8_gemm(h, hs, w2, s2)
    ids, route_w = lib.moe_route_topk(logits, 3)
    return dense, ids, route_w, lib.fp8_moe(x, ids, route_w, *experts)


@pytest.mark.parametrize("m", [1, 6, 40])
def test_feed_forward_together_and_captured(lib, m):
    dim, inter, E = 512, 384, 16
    g = gen(m)
    raw1, raw2 = normal(g, 2 * inter, dim, std=0.05), normal(g, dim, inter, std=0.05)
    (w1, s1), (w2, s2) = lib.fp8_quantize(raw1, block_rows=128), lib.fp8_quantize(raw2, block_rows=128)
    experts = moe_inputs(m, m, E, 3, dim, inter)[3:]
    x, logits = normal(g, m, dim, dtype=BF16), normal(g, m, E)
    dense, ids, route_w, routed = ffn(lib, x, w1, s1, w2, s2, logits, experts)
    # against 64 bits from the weights as they were: three roundings to e4m3 (each rms about 2^-5.3 of the value) on
    # random signs, so their sum over a row is about as far off, relative to its norm
    g64, u64 = (x.double() @ raw1.double().t()).chunk(2, -1)
    want = (g64 * torch.sigmoid(g64) * u64) @ raw2.double().t()
    assert (dense.double() - want).norm() <= 0.1 * want.norm()
    want, tol = moe_want(x, ids, route_w, *experts, F32)
    within(routed, want, tol)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    xs, ls = x.clone(), logits.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        ffn(lib, xs, w1, s1, w2, s2, ls, experts)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            out = ffn(lib, xs, w1, s1, w2, s2, ls, experts)
    for i in range(3):
        xs.copy_(normal(g, m, dim, dtype=BF16) if i else x)
        ls.copy_(normal(g, m, E) if i else logits)
        graph.replay()
        torch.cuda.synchronize()
        want = ffn(lib, xs, w1, s1, w2, s2, ls, experts)
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert torch.equal(want[1], out[1])


def test_calls_on_streams_of_their_own(lib):
    """Two calls at once, each with a workspace of its own."""
    sets = [moe_inputs(i, 8, 16, 4, 512, 384) for i in range(2)]
    want = [lib.fp8_moe(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [lib.fp8_moe(*s, stream=st) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,N,extra", [(40, 133, 3), (40, 130, 6), (200, 257, 7), (300, 1001, 7), (300, 1002, 2), (130, 1000, 8), (513, 127, 1)])
def test_gemm_leaves_what_follows_a_row(lib, dtype, m, N, extra):
    """Rows of y that end inside 16 bytes, with aligned row starts."""
    g = gen(N)
    K = 256
    x, xs, w, ws = codes(g, m, K), scales(g, m, 2), codes(g, N, K), scales(g, blocks(N), 2)
    out, untouched = guarded(m, N, dtype, extra=extra)
    y = lib.fp8_gemm(x, xs, w, ws, out=out)
    want, size = gemm_want(x, xs, w, ws)
    within(y, want, gemm_tol(want, size, K, dtype))
    untouched()


def test_two_captured_steps_with_workspaces_of_their_own(lib):
    """Replayed one after another and at once."""
    sets = [moe_inputs(20 + i, 6, 8, 3, 512, 384) for i in range(2)]
    want = [lib.fp8_moe(*s) for s in sets]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in sets]
    for s, st in zip(sets, streams):
        work = torch.empty(lib.fp8_moe_workspace_bytes(6, 3, 512, 384), dtype=torch.uint8, device=DEV)
        st.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            outs.append(lib.fp8_moe(*s, workspace=work))
        graphs.append((graph, work))
    torch.cuda.synchronize()
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for (graph, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_ids_written_by_the_launch_before(lib):
    """The second launch reads ids and weights before it waits for the first: what came before has to be complete."""
    args = moe_inputs(31, 4, 16, 2, 256, 256)
    good = lib.fp8_moe(*args)
    ids, w = args[1].clone(), args[2].clone()
    for _ in range(50):
        ids.fill_(-1)
        w.fill_(0)
        ids.copy_(args[1])
        w.copy_(args[2])
        assert torch.equal(lib.fp8_moe(args[0], ids, w, *args[3:]), good)


def test_repeated_calls_give_the_same_bits(lib):
    args = moe_inputs(77, 19, 12, 4, 640, 528)
    x, xs, w, ws = codes(gen(1), 77, 1168), scales(gen(2), 77, 10), codes(gen(3), 900, 1168), scales(gen(4), 8, 10)
    moe, gemm = lib.fp8_moe(*args), lib.fp8_gemm(x, xs, w, ws)
    few = lib.fp8_gemm(x[:9], xs[:9], w, ws)
    for _ in range(20):
        assert torch.equal(lib.fp8_moe(*args), moe) and torch.equal(lib.fp8_gemm(x, xs, w, ws), gemm)
        assert torch.equal(lib.fp8_gemm(x[:9], xs[:9], w, ws), few)


def test_small_products_on_two_streams_at_once(lib):
    """Products of few tiles, whose clusters could share SMs: none waits for another's tensor memory."""
    g, sides = gen(43), (torch.cuda.Stream(), torch.cuda.Stream())
    inputs = []
    for m, N in ((1, 144), (16, 272), (24, 512), (48, 256)):
        x, w = codes(g, m, 1024), codes(g, N, 1024)
        inputs.append((x, scales(g, m, 8), w, scales(g, blocks(N), 8)))
    alone = [lib.fp8_gemm(*i) for i in inputs]
    torch.cuda.synchronize()
    got = []
    for turn in range(50):
        for side in sides:
            got += [(n, lib.fp8_gemm(*inputs[n], stream=side)) for n in range(len(inputs))]
    torch.cuda.synchronize()
    assert all(torch.equal(alone[n], y) for n, y in got)
