"""swiglu_fp8_rows over the whole range of finite gates and ups.

A row has one value of h throughout, so that its scale is |h| / 448: h to
within its roundings, not to within those of an e4m3 code.  2^-20 of h: the
power of two 2^-22, the reciprocal 2^-23, four more roundings of 2^-24 (the
correction, its product, the sum, and the two products of h are at most five;
the correction's own is in 1 + 2^-17), the scale's division 2^-24: 12 of
16 * 2^-24; where e^-g is above 2^126 the sigmoid has two bits fewer, 4 * 2^-24
more.
"""
import pytest
import torch

from test_gpu_fp8 import BF16, DEV, F32, gen, lib  # noqa: F401


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
