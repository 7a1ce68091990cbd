"""swiglu_fp8_rows over the whole range of finite gates and ups.

A row has one value of h throughout, so that its scale is |h| / 448: h to
within its roundings, not to within those of an e4m3 code.  2^-20 of h: the
power of two 2^-22, the reciprocal 2^-23, two roundings of 2^-24 up to the
reciprocal and two of the products, the scale's division 2^-24: 11 of
16 * 2^-24; where e^-g is above 2^126 the sigmoid has two bits fewer, 4 * 2^-24
more.
"""
import pytest
import torch

from test_gpu_fp8 import BF16, DEV, F32, gen, lib  # noqa: F401

pytestmark = pytest.mark.gpu


def rows_of(gates, ups, N, dtype):
    """[n, 2 N]: a gate and an up a row, N times each, as they are in `dtype`."""
    g, u = (torch.as_tensor(t, dtype=torch.float64).to(device=DEV).to(dtype)[:, None].expand(-1, N) for t in (gates, ups))
    return torch.cat([g, u], 1).contiguous()


def check(lib, x, N):  # noqa: F811
    g, u = x[:, 0].double(), x[:, N].double()
    h = torch.where(g >= 0, g / (1 + torch.exp(-g)), g * torch.exp(g) / (1 + torch.exp(g))) * u
    assert (h.abs() < 2.0 ** 128).all() and (h.abs() > 2.0 ** -110).all()
    q, s = lib.swiglu_fp8_rows(x)
    off = ((s.double() * 448 - h.abs()[:, None]).abs() / h.abs()[:, None]).amax(1)
    bad = ~(off <= 2.0 ** -20)
    assert not bad.any(), [(a.item(), b.item(), o.item()) for a, b, o in zip(g[bad], u[bad], off[bad])][:8]
    assert (q.double() == 448 * torch.sign(h)[:, None]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", [16, 13, 300])
def test_swiglu_of_the_largest_gates(lib, dtype, N):  # noqa: F811
    """-g log2(e) is past fp32's range from 2.36e38 on; h is g u."""
    gates, ups = (2.3e38, 2.37e38, 2.5e38, 3.0e38, 3.38e38), (1.0, -1.0, 0.5, -1e-3, 1e-30, 1e-45 if dtype == F32 else 1e-40)
    x = rows_of([g for g in gates for _ in ups], [u for _ in gates for u in ups], N, dtype)
    check(lib, x, N)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", [16, 13, 300])
def test_swiglu_of_the_smallest_gates_and_large_ups(lib, dtype, N):  # noqa: F811
    """Gates near and below fp32's smallest normal value; h is g u / 2."""
    gates = (1e-37, 1.17549e-38, -2.35e-38, 4.7e-38, -3e-39, 1.2345e-40, 1e-40, -1e-41 if dtype == F32 else -2e-40)
    ups = (1e38, -3.3e38, 1.7e37, 1e30)
    x = rows_of([g for g in gates for _ in ups], [u for _ in gates for u in ups], N, dtype)
    check(lib, x, N)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", [16, 13])
def test_swiglu_of_gates_and_ups_of_every_size(lib, dtype, N):  # noqa: F811
    """Exponents of g and h spread over all that fp32 has, down to where e^-g leaves it."""
    n, seed = 20000, gen(N)

    def uniform(lo, hi):
        return torch.rand(n, generator=seed, device=DEV, dtype=torch.float64) * (hi - lo) + lo

    sign = torch.where(uniform(0, 1) < 0.5, -1.0, 1.0)
    g = torch.exp2(uniform(-149, 128)).clamp(max=3.38e38) * torch.where(uniform(0, 1) < 0.5, -1.0, 1.0)
    g = torch.where(g < -1, uniform(-88.6, 0), g).to(dtype).double()
    sigmoid = torch.where(g >= 0, 1 / (1 + torch.exp(-g)), torch.exp(g) / (1 + torch.exp(g)))
    u = (torch.exp2(uniform(-100, 120)) / (g * sigmoid).abs() * sign).to(dtype).double()
    fits = (u.abs() < 3.38e38) & (u.abs() > 2.0 ** -126) & ((g * sigmoid * u).abs() > 2.0 ** -105)
    fits &= (u * sigmoid).abs() > 2.0 ** -126  # (that product is rounded where fp32 has all its bits)
    assert fits.sum() > n // 3
    check(lib, rows_of(g[fits], u[fits], N, dtype), N)
