"""Layer norm where its accuracy could get lost: points without spread, values far
from one, sums over many channels.

Tolerances.  u = 2^-24 is half a float32 step; a storage rounding is off by at
most finfo(t).eps / 2 of the value (and by half the smallest subnormal).
"""

import pytest

from fno_testlib import torch_dtype
from fourier_neural_spectral_fno_b200 import capi

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}

# channel counts whose reciprocal rounds badly, in shapes for the pipelines (from a
# million values on, or four), odd grids, small grids, rows of whole pieces and
# others, and the kernels for any channel count
CONSTANT = [(1, 41, 102400), (2, 61, 34400), (1, 63, 66600), (3, 7, 200008), (1, 14, 300000),
            (4, 28, 37504), (1, 97, 10816), (1, 125, 8392), (2, 112, 4688),
            (2, 7, 257), (2, 41, 1023), (1, 63, 4099), (3, 97, 259), (1, 125, 777), (2, 30, 301),
            (2, 61, 64), (1, 125, 132), (3, 60, 35),
            (9, 56, 1), (5, 63, 1), (4, 448, 1), (3, 776, 1), (6, 1000, 1), (5, 1001, 1),
            (2, 896, 1), (3, 3584, 1), (1, 1100, 5), (2, 4096, 1), (3, 4095, 1), (2, 8191, 1),
            (2, 8192, 1), (3, 6137, 1)]
# more channels than the first sum of float16 values is exact for
LONG = [(2, 8200, 1), (3, 12001, 1), (2, 16384, 1)]


@pytest.mark.parametrize("shape", CONSTANT, ids=str)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_layer_norm_constant_points_of_any_size(shape, dtype):
    """Points of C equal 16-bit values v give mean = v, y = beta and dgamma = 0.

    Every partial sum k v has at most 11 + 13 significant bits: exact.  The first
    mean is off by the reciprocal's and the product's rounding, d = v - m0 with |d| <=
    2.1 u |v|, and is a few steps of v, so that its sums k d are exact; their mean e is
    off by 2.1 u |d|.  So mean = m0 + e lies within 5 u^2 |v| of v before its rounding,
    which gives v; |xh| <= 5 u^2 |v| eps^-1/2; and the variance, mean(d^2) - e^2, is
    off from 0 by at most 8 u d^2.  In the backward x - mean = 0."""
    import torch
    outer, C, inner = shape
    g = torch.Generator(device="cuda").manual_seed(41)
    dt = torch_dtype(dtype)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    # sizes from 2^-4 to 2^15.9, each with all its bits
    v = torch.exp2(20 * torch.rand((outer, 1, inner), generator=g, device="cuda") - 4.1)
    v = (v * rnd(outer, 1, inner).sign()).to(dt)
    for k, known in enumerate((1000.0, 250.0, 33856.0, 3.0)):
        if k < outer * inner:
            v.view(-1)[k] = known
    x = v.expand(outer, C, inner).contiguous()
    gamma, beta = (1 + 0.2 * rnd(C)).to(dt), (0.2 * rnd(C)).to(dt)
    d = capi.layer_norm_desc(outer, C, inner, dtype, EPS)
    y = torch.empty_like(x)
    mean, rstd = (torch.empty((outer, inner), device="cuda") for _ in range(2))
    capi.fno_layer_norm_fwd(d, x, gamma, beta, y, mean, rstd)
    v6 = v.double()[:, 0]
    assert torch.equal(mean.double(), v6)
    r0 = EPS ** -0.5
    assert bool(((rstd.double() - r0).abs()
                 <= r0 * (8 * U + 8 * U * (2.1 * U * v6) ** 2 / EPS)).all())
    be = beta.double()[:, None]
    off = 5 * U * U * v6.abs()[:, None] * r0 * gamma.double().abs()[:, None]
    tol = off + HALF[dtype] * off + 4 * U * be.abs() + TINY[dtype]
    assert bool(((y.double() - be).abs() <= tol).all())
    dy = (0.3 * rnd(outer, C, inner)).to(dt)
    dx = torch.empty_like(x)
    dg, db = torch.ones(C, device="cuda"), torch.empty(C, device="cuda")
    capi.fno_layer_norm_bwd(d, x, gamma, mean, rstd, dy, dx, dg, db)
    assert not bool(dg.any())


@pytest.mark.parametrize("shape", CONSTANT + LONG, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_layer_norm_points_of_one_step(shape, dtype):
    """C equal values but for one channel, which is a step of the type (in float32
    2^-10 of the value) away: y within (2 C + 16) u (1 + |xh|) |gamma| + 4 u |y|, as for
    any other point, since the deviations are corrected by their own mean.  (The first
    mean is off by at most 2.1 u |v|, the sum of up to 2^13 values of 11 bits being exact,
    or by the 20 additions that a value takes part in; the spread is at least 2^-11 |v| /
    C^1/2: the square of their quotient, which enters the variance with a relative error
    of C u, stays below one.)"""
    import torch
    outer, C, inner = shape
    g = torch.Generator(device="cuda").manual_seed(43)
    dt = torch_dtype(dtype)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    v = torch.exp2(10 * torch.rand((outer, 1, inner), generator=g, device="cuda"))
    v = (v * rnd(outer, 1, inner).sign()).to(dt)
    x = v.expand(outer, C, inner).contiguous()
    step = 2.0 ** -9 if dtype == "f32" else torch.finfo(dt).eps
    x[:, C // 3] = (x[:, C // 3].double() * (1 + step)).to(dt)
    gamma, beta = (1 + 0.2 * rnd(C)).to(dt), (0.2 * rnd(C)).to(dt)
    d = capi.layer_norm_desc(outer, C, inner, dtype, EPS)
    y = torch.empty_like(x)
    capi.fno_layer_norm_fwd(d, x, gamma, beta, y)
    x6, ga = x.double(), gamma.double()[:, None]
    rm = x6.mean(1, keepdim=True)
    xh = (x6 - rm) / ((x6 - rm).square().mean(1, keepdim=True) + EPS).sqrt()
    ry = xh * ga + beta.double()[:, None]
    tol = (2 * C + 16) * U * (1 + xh.abs()) * ga.abs() + 4 * U * ry.abs()
    tol = tol + HALF[dtype] * (ry.abs() + tol) + TINY[dtype]
    assert bool(((y.double() - ry).abs() <= tol).all())


@pytest.mark.parametrize("shape", [(3, 20, 70008), (2, 64, 33000), (1, 97, 40008), (33, 128, 256),
                                   (2, 20, 1023), (2, 65, 257), (3, 32, 64), (2, 200, 16),
                                   (9, 56, 1), (4, 1001, 1), (2, 300, 40), (1, 33000, 1)], ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("spread,size,eps", [(2.0 ** 50, 2.0 ** -35, 1e-5), (2.0 ** -60, 2.0 ** 12, 1e-37)],
                         ids=["wide", "narrow"])
def test_layer_norm_backward_far_from_one(shape, dtype, spread, size, eps):
    """x of spread 2^50 with dy of 2^-35, and of spread 2^-60 with dy of 2^12: dx, 2^-85
    and 2^72, lies well inside the type's range, as do xh, g and the means of g and g xh;
    so dx is off by rstd (C + 16) u (|g| + mean|g| + |xh| mean|g xh|) and its rounding to
    storage, as everywhere else."""
    import torch
    outer, C, inner = shape
    g = torch.Generator(device="cuda").manual_seed(53)
    dt = torch_dtype(dtype)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, dy = (spread * rnd(*shape)).to(dt), (size * rnd(*shape)).to(dt)
    gamma = (1 + 0.2 * rnd(C)).to(dt)
    d = capi.layer_norm_desc(outer, C, inner, dtype, eps)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = (torch.empty((outer, inner), device="cuda") for _ in range(2))
    dg, db = (torch.empty(C, device="cuda") for _ in range(2))
    capi.fno_layer_norm_fwd(d, x, gamma, None, y, mean, rstd)
    capi.fno_layer_norm_bwd(d, x, gamma, mean, rstd, dy, dx, dg, db)
    r = rstd.double()[:, None]
    xh = (x.double() - mean.double()[:, None]) * r
    gg = dy.double() * gamma.double()[:, None]
    ref = r * (gg - gg.mean(1, keepdim=True) - xh * (gg * xh).mean(1, keepdim=True))
    tol = r * (C + 16) * U * (gg.abs() + gg.abs().mean(1, keepdim=True)
                              + xh.abs() * (gg * xh).abs().mean(1, keepdim=True))
    tol = tol + HALF[dtype] * (ref.abs() + tol) + TINY[dtype]
    assert bool(((dx.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("shape", [(1, 1100, 5), (1, 4099, 6), (2, 33000, 3), (2, 33000, 1),
                                   (1, 100003, 3), (1, 100003, 1), (1, 1 << 20, 2),
                                   (2, 1 << 20, 1)], ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layer_norm_sums_over_many_channels(shape, dtype):
    """Values of one sign and nearly one size, whose roundings add up in a long chain.

    A thread's sum over the channels is compensated: off by 2 u and C u^2 <= u / 16 of its
    terms' sizes, whose own products are rounded once; where threads share a row, five
    steps of a warp's and eight of a CTA's sum follow.  That is n = 20 roundings at most,
    whatever C is, and the tolerances are those with C terms, with n in the place of C:
    y (2 n + 16) u (1 + |xh|) |gamma| + 4 u |y|; dx rstd (n + 16) u (|g| + mean|g| + |xh|
    mean|g xh|); each with its rounding to storage."""
    import torch
    outer, C, inner = shape
    n = 20
    g = torch.Generator(device="cuda").manual_seed(59)
    dt = torch_dtype(dtype)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = (1.1 + 0.02 * rnd(*shape)).to(dt)
    dy = (0.1 + 0.001 * rnd(*shape)).to(dt)
    gamma, beta = (1 + 0.02 * rnd(C)).to(dt), (0.2 * rnd(C)).to(dt)
    d = capi.layer_norm_desc(outer, C, inner, dtype, EPS)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = (torch.empty((outer, inner), device="cuda") for _ in range(2))
    capi.fno_layer_norm_fwd(d, x, gamma, beta, y, mean, rstd)
    x6, ga = x.double(), gamma.double()[:, None]
    rm = x6.mean(1, keepdim=True)
    xh = (x6 - rm) / ((x6 - rm).square().mean(1, keepdim=True) + EPS).sqrt()
    ry = xh * ga + beta.double()[:, None]
    tol = (2 * n + 16) * U * (1 + xh.abs()) * ga.abs() + 4 * U * ry.abs()
    assert bool(((y.double() - ry).abs()
                 <= tol + HALF[dtype] * (ry.abs() + tol) + TINY[dtype]).all())
    assert bool(((mean.double() - rm[:, 0]).abs() <= (n + 4) * U * x6.abs().mean(1)).all())
    capi.fno_layer_norm_bwd(d, x, gamma, mean, rstd, dy, dx)
    r = rstd.double()[:, None]
    xh = (x6 - mean.double()[:, None]) * r
    gg = dy.double() * ga
    ref = r * (gg - gg.mean(1, keepdim=True) - xh * (gg * xh).mean(1, keepdim=True))
    tol = r * (n + 16) * U * (gg.abs() + gg.abs().mean(1, keepdim=True)
                              + xh.abs() * (gg * xh).abs().mean(1, keepdim=True))
    assert bool(((dx.double() - ref).abs()
                 <= tol + HALF[dtype] * (ref.abs() + tol) + TINY[dtype]).all())


@pytest.mark.parametrize("channels", [63, 128, 768, 1000, 2047, 4095, 4096, 6137, 8184, 8192, 12001])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_layer_norm_rows_on_both_sides_of_a_power_of_two(channels, dtype):
    """Rows of 1024 with one channel a step above and one a half step below, whose sum
    needs the finest bits: y within the tolerance above."""
    import torch
    rows = 40
    g = torch.Generator(device="cuda").manual_seed(67)
    dt = torch_dtype(dtype)
    eps = torch.finfo(dt).eps
    x = torch.full((rows, channels), 1024.0, device="cuda", dtype=dt)
    up = torch.randint(0, channels // 2, (rows, 1), generator=g, device="cuda")
    down = torch.randint(channels // 2, channels, (rows, 1), generator=g, device="cuda")
    x.scatter_(1, up, 1024 * (1 + eps)).scatter_(1, down, 1024 * (1 - eps / 2))
    d = capi.layer_norm_desc(rows, channels, 1, dtype, EPS)
    y = torch.empty_like(x)
    capi.fno_layer_norm_fwd(d, x, None, None, y)
    x6 = x.double()
    rm = x6.mean(1, keepdim=True)
    ry = (x6 - rm) / ((x6 - rm).square().mean(1, keepdim=True) + EPS).sqrt()
    tol = (2 * channels + 16) * U * (1 + ry.abs()) + 4 * U * ry.abs()
    tol = tol + HALF[dtype] * (ry.abs() + tol) + TINY[dtype]
    assert bool(((y.double() - ry).abs() <= tol).all())
