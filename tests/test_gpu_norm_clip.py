"""Layer norm, the gradient norm, clipping and the clipped Adam step on the GPU
against the float64 oracle.

Tolerances.  u = 2^-24 is half a float32 step; a storage rounding is off by at
most finfo(t).eps / 2 of the value (and by half the smallest subnormal).

Forward: a sum of C terms in any order is off by at most C u times the sum of
their sizes.  Each xh therefore carries at most (2 C + 16) u (1 + |xh|) from the
mean, the variance and the last operations, and y that times |gamma|, plus
4 u |y| and the rounding to storage.
Backward: the two means over the channels are off by (C + 8) u of the mean of
their terms' sizes; xh, taken from the given statistics, by 4 u |xh|; so dx by
rstd (C + 16) u (|g| + mean|g| + |xh| mean|g xh|) and its rounding to storage.
Parameter gradients: every partial sum runs over at most `terms` values one
after another and the partial sums meet in at most 296 / 8 + 8 + 16 more steps:
(terms + 64) u of the sum of the terms' sizes, and 4 u of each term.
"""

import numpy as np
import pytest

import oracle as O
from fno_testlib import torch_dtype
from fourier_neural_spectral_fno_b200 import capi, synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}


def _dev(a, dtype="f32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.float64)).cuda().to(torch_dtype(dtype))


def _host(t):
    return t.double().cpu().numpy()


def _inputs(outer, C, inner, dtype, seed=5, offset=0.0):
    rng = np.random.default_rng(seed)
    q = lambda a: synth.quantize(a, dtype)  # noqa: E731
    x = q(rng.standard_normal((outer, C, inner)) * np.exp(0.5 * rng.standard_normal((1, C, 1)))
          + 0.7 * rng.standard_normal((1, C, 1)) + offset)
    return (x, q(1 + 0.2 * rng.standard_normal(C)), q(0.2 * rng.standard_normal(C)),
            q(0.3 * rng.standard_normal((outer, C, inner))))


def _bands(shape, dtype):
    """A tensor of that shape inside a buffer of sentinels, and the buffer."""
    import torch
    n = int(np.prod(shape))
    buf = torch.full((n + 64,), 7.0, dtype=torch_dtype(dtype), device="cuda")
    return buf[32:32 + n].view(*shape), buf


def _untouched(buf, n):
    return bool((buf[:32] == 7).all()) and bool((buf[32 + n:] == 7).all())


def _check_fwd(y, mean, rstd, x, gamma, beta, dtype, eps=EPS):
    C = x.shape[1]
    ry, rm, rr = O.layer_norm_fwd(x, gamma, beta, eps)
    xh = (x - rm[:, None]) * rr[:, None]
    ga = 1.0 if gamma is None else np.abs(gamma)[None, :, None]
    tol = (2 * C + 16) * U * (1 + np.abs(xh)) * ga + 4 * U * np.abs(ry)
    tol = tol + HALF[dtype] * (np.abs(ry) + tol) + TINY[dtype]
    assert np.all(np.abs(_host(y) - ry) <= tol)
    if mean is not None:
        size = np.abs(x).mean(1)
        assert np.all(np.abs(_host(mean) - rm) <= (C + 4) * U * size)
        # d rstd / rstd = d var / (2 (var + eps)), var off by (C + 8) u of itself
        assert np.all(np.abs(_host(rstd) - rr) <= (C + 16) * U * rr)


def _check_bwd(dx, dgamma, dbeta, x, gamma, mean, rstd, dy, dtype, terms=None):
    C = x.shape[1]
    rdx, rdg, rdb = O.layer_norm_bwd(x, gamma, mean, rstd, dy)
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy if gamma is None else dy * gamma[None, :, None]
    tol = rstd[:, None] * (C + 16) * U * (np.abs(g) + np.abs(g).mean(1)[:, None]
                                          + np.abs(xh) * np.abs(g * xh).mean(1)[:, None])
    tol = tol + HALF[dtype] * (np.abs(rdx) + tol) + TINY[dtype]
    assert np.all(np.abs(_host(dx) - rdx) <= tol)
    points = x.shape[0] * x.shape[2]
    terms = min(points, 4096) if terms is None else terms
    for got, ref, each in ((dgamma, rdg, dy * xh), (dbeta, rdb, dy)):
        if got is not None:
            tol = (terms + 68) * U * np.abs(each).sum((0, 2)) + 1e-45
            assert np.all(np.abs(_host(got) - ref) <= tol)


# rows, grids with odd and even sides, one channel, one point, channel counts on
# both sides of every internal limit
SHAPES = [(1, 1, 1), (5, 3, 1), (3, 1, 7), (2, 2, 9), (7, 8, 1), (1, 20, 256), (2, 20, 1023),
          (3, 32, 64), (2, 33, 68), (2, 64, 1000), (2, 65, 132), (1, 100, 33), (2, 300, 40),
          (1, 520, 24), (1, 1025, 12), (2, 2100, 6), (33, 64, 1), (130, 100, 1), (9, 1000, 1),
          (4, 1001, 1), (3, 2048, 1), (5, 2052, 1), (2, 4097, 1), (2, 8192, 1), (1, 33000, 1),
          (40, 24, 2), (50, 16, 3), (3, 24, 4096), (1, 4, 100003)]
# rows that start anywhere: every channel count the kernels round up to and its
# neighbours, the shortest rows, rows that end inside a warp's points, rows of a
# multiple of four values (pieces of float32, none of 16-bit gradients)
SHAPES += [(2, 1, 257), (3, 7, 1021), (2, 8, 4099), (3, 9, 259), (1, 16, 2047), (2, 17, 385),
           (3, 21, 449), (2, 24, 4099), (2, 25, 321), (1, 32, 4097), (5, 32, 1444), (2, 33, 513),
           (2, 47, 767), (2, 48, 1023), (2, 49, 1025), (700, 12, 291), (2, 40, 1444),
           (1, 57, 4099), (3, 64, 289), (2, 65, 257), (1, 73, 1021), (2, 81, 259), (2, 96, 517),
           (3, 97, 345), (2, 105, 299), (1, 113, 777), (1, 128, 2049), (2, 129, 301),
           (650, 33, 257)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_layer_norm_matches_oracle(shape, dtype):
    outer, C, inner = shape
    x, gamma, beta, dy = _inputs(outer, C, inner, dtype)
    d = capi.layer_norm_desc(outer, C, inner, dtype, EPS)
    n, pts = x.size, outer * inner
    y, ybuf = _bands(x.shape, dtype)
    mean, mbuf = _bands((outer, inner), "f32")
    rstd, rbuf = _bands((outer, inner), "f32")
    xd, gd, bd, dyd = _dev(x, dtype), _dev(gamma, dtype), _dev(beta, dtype), _dev(dy, dtype)
    capi.fno_layer_norm_fwd(d, xd, gd, bd, y, mean, rstd)
    _check_fwd(y, mean, rstd, x, gamma, beta, dtype)
    assert _untouched(ybuf, n) and _untouched(mbuf, pts) and _untouched(rbuf, pts)

    dx, dxbuf = _bands(x.shape, dtype)
    dg, dgbuf = _bands((C,), "f32")
    db, dbbuf = _bands((C,), "f32")
    capi.fno_layer_norm_bwd(d, xd, gd, mean, rstd, dyd, dx, dg, db)
    m64, r64 = _host(mean), _host(rstd)
    _check_bwd(dx, dg, db, x, gamma, m64, r64, dy, dtype)
    assert _untouched(dxbuf, n) and _untouched(dgbuf, C) and _untouched(dbbuf, C)
    # the inputs are as they were
    assert np.array_equal(_host(xd), x) and np.array_equal(_host(dyd), dy)


def _check_large(got, ref, tol, what):
    """On the device: |got - ref| <= tol everywhere."""
    worst = ((got.double() - ref).abs() - tol).max().item()
    assert worst <= 0, f"{what}: {worst} beyond its tolerance"


# sizes from a million values on, where the copies run as pipelines: every
# channel count they round up to and odd ones between, rows that end inside a
# tile, one sample and many, one tile per sample
LARGE = [(3, 5, 281000), (17, 8, 33000), (2, 13, 163848), (5, 16, 53000), (1, 17, 250008),
         (3, 20, 70008), (4, 23, 46000), (7, 24, 25000), (2, 31, 68008), (540, 32, 256),
         (3, 45, 31512), (2, 48, 44000), (3, 61, 23000), (2, 64, 33000), (130, 64, 520),
         (4, 65, 16392), (2, 96, 9000), (1, 97, 40008), (3, 127, 5000), (33, 128, 256)]


@pytest.mark.parametrize("shape", LARGE, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_layer_norm_large_matches_float64(shape, dtype):
    """The formulas in float64 torch operations, with the tolerances above; guard
    bands, and dx over dy giving the same bits."""
    import torch
    outer, C, inner = shape
    g = torch.Generator(device="cuda").manual_seed(13)
    dt = torch_dtype(dtype)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = (rnd(outer, C, inner) * torch.exp(0.5 * rnd(1, C, 1)) + 0.7 * rnd(1, C, 1)).to(dt)
    gamma, beta = (1 + 0.2 * rnd(C)).to(dt), (0.2 * rnd(C)).to(dt)
    dy = (0.3 * rnd(outer, C, inner)).to(dt)
    d = capi.layer_norm_desc(outer, C, inner, dtype, EPS)
    y, ybuf = _bands(x.shape, dtype)
    mean, mbuf = _bands((outer, inner), "f32")
    rstd, rbuf = _bands((outer, inner), "f32")
    capi.fno_layer_norm_fwd(d, x, gamma, beta, y, mean, rstd)
    assert _untouched(ybuf, x.numel())
    assert _untouched(mbuf, mean.numel()) and _untouched(rbuf, mean.numel())
    x6, ga, be = x.double(), gamma.double()[:, None], beta.double()[:, None]
    rm = x6.mean(1)
    rr = 1 / ((x6 - rm[:, None]).square().mean(1) + EPS).sqrt()
    xh = (x6 - rm[:, None]) * rr[:, None]
    ry = xh * ga + be
    tol = (2 * C + 16) * U * (1 + xh.abs()) * ga.abs() + 4 * U * ry.abs()
    _check_large(y, ry, tol + HALF[dtype] * (ry.abs() + tol) + TINY[dtype], "y")
    _check_large(mean, rm, (C + 4) * U * x6.abs().mean(1), "mean")
    _check_large(rstd, rr, (C + 16) * U * rr, "rstd")
    y2 = torch.empty_like(x)
    capi.fno_layer_norm_fwd(d, x, gamma, beta, y2)
    assert torch.equal(y2, y)
    same = x.clone()
    capi.fno_layer_norm_fwd(d, same, gamma, beta, same)
    assert torch.equal(same, y)

    dx, dxbuf = _bands(x.shape, dtype)
    dg, db = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    capi.fno_layer_norm_bwd(d, x, gamma, mean, rstd, dy, dx, dg, db)
    assert _untouched(dxbuf, x.numel())
    mu, r, dy6 = mean.double()[:, None], rstd.double()[:, None], dy.double()
    xh = (x6 - mu) * r
    gg = dy6 * ga
    rdx = r * (gg - gg.mean(1, keepdim=True) - xh * (gg * xh).mean(1, keepdim=True))
    tol = r * (C + 16) * U * (gg.abs() + gg.abs().mean(1, keepdim=True)
                              + xh.abs() * (gg * xh).abs().mean(1, keepdim=True))
    _check_large(dx, rdx, tol + HALF[dtype] * (rdx.abs() + tol) + TINY[dtype], "dx")
    for got, each, name in ((dg, dy6 * xh, "dgamma"), (db, dy6, "dbeta")):
        _check_large(got, each.sum((0, 2)), (4096 + 68) * U * each.abs().sum((0, 2)), name)
    dg2, db2, dx2 = torch.empty_like(dg), torch.empty_like(db), torch.empty_like(x)
    capi.fno_layer_norm_bwd(d, x, gamma, mean, rstd, dy, dx2, None, db2)
    assert torch.equal(dx2, dx) and torch.equal(db2, db)
    capi.fno_layer_norm_bwd(d, x, gamma, mean, rstd, dy, dx2)
    assert torch.equal(dx2, dx)
    capi.fno_layer_norm_bwd(d, x, gamma, mean, rstd, dy, dy, dg2, db2)
    assert torch.equal(dy, dx) and torch.equal(dg2, dg) and torch.equal(db2, db)


@pytest.mark.parametrize("shape", [(2, 20, 96), (3, 20, 35), (6, 40, 1), (3, 41, 1), (2, 1100, 5),
                                   (2, 200, 12), (1, 33001, 1)], ids=str)
def test_layer_norm_optional_arguments_and_in_place(shape):
    """gamma, beta, the statistics and the parameter gradients may be missing;
    y may be x and dx may be dy: the same bits as with everything given."""
    import torch
    outer, C, inner = shape
    x, gamma, beta, dy = _inputs(outer, C, inner, "f32", seed=6)
    d = capi.layer_norm_desc(outer, C, inner, "f32", EPS)
    xd, gd, bd, dyd = _dev(x), _dev(gamma), _dev(beta), _dev(dy)
    y, mean, rstd = torch.empty_like(xd), _dev(np.zeros((outer, inner))), _dev(np.zeros((outer, inner)))
    capi.fno_layer_norm_fwd(d, xd, None, None, y, mean, rstd)
    _check_fwd(y, mean, rstd, x, None, None, "f32")
    capi.fno_layer_norm_fwd(d, xd, gd, None, y)
    _check_fwd(y, None, None, x, gamma, None, "f32")
    capi.fno_layer_norm_fwd(d, xd, None, bd, y)
    _check_fwd(y, None, None, x, None, beta, "f32")
    capi.fno_layer_norm_fwd(d, xd, gd, bd, y)
    same = xd.clone()
    capi.fno_layer_norm_fwd(d, same, gd, bd, same)
    assert torch.equal(same, y)

    m64, r64 = _host(mean), _host(rstd)
    dx, dg, db = torch.empty_like(xd), torch.empty_like(gd), torch.empty_like(gd)
    capi.fno_layer_norm_bwd(d, xd, None, mean, rstd, dyd, dx, dg, db)
    _check_bwd(dx, dg, db, x, None, m64, r64, dy, "f32")
    capi.fno_layer_norm_bwd(d, xd, gd, mean, rstd, dyd, dx, dg, db)
    for a, b in ((dg, None), (None, db), (None, None), (dg, db)):
        dx2 = torch.empty_like(xd)
        a2, b2 = None if a is None else torch.empty_like(a), None if b is None else torch.empty_like(b)
        capi.fno_layer_norm_bwd(d, xd, gd, mean, rstd, dyd, dx2, a2, b2)
        assert torch.equal(dx2, dx)
        assert a is None or torch.equal(a2, a)
        assert b is None or torch.equal(b2, b)
    dg2, db2 = torch.empty_like(dg), torch.empty_like(db)
    capi.fno_layer_norm_bwd(d, xd, gd, mean, rstd, dyd, dyd, dg2, db2)
    assert torch.equal(dyd, dx) and torch.equal(dg2, dg) and torch.equal(db2, db)


@pytest.mark.parametrize("shape", [(2, 20, 64), (2, 20, 35), (8, 64, 1), (4, 1001, 1),
                                   (1, 1100, 8), (1, 33001, 1), (2, 200, 16), (2, 20, 1023),
                                   (2, 77, 1023), (4, 96, 4096), (1, 128, 8196)], ids=str)
def test_layer_norm_large_offset(shape):
    """A common offset of 4096 against a spread of one: the tolerances hold
    unchanged (for the mean they grow with the values' size), because the
    deviations are taken about a first mean and corrected by their own mean.
    First mean off by at most (C u 4096) from the true one; its square against
    the variance is below (C u 4096)^2 <= 2^-4 at C = 1024 and enters the
    variance with a relative error of C u only."""
    import torch
    outer, C, inner = shape
    x, gamma, beta, _ = _inputs(outer, C, inner, "f32", seed=7, offset=4096.0)
    d = capi.layer_norm_desc(outer, C, inner, "f32", EPS)
    y = torch.empty(x.shape, device="cuda")
    mean, rstd = torch.empty(outer, inner, device="cuda"), torch.empty(outer, inner, device="cuda")
    capi.fno_layer_norm_fwd(d, _dev(x), _dev(gamma), _dev(beta), y, mean, rstd)
    _check_fwd(y, mean, rstd, x, gamma, beta, "f32")


@pytest.mark.parametrize("shape", [(2, 20, 1023), (3, 32, 4099), (2, 48, 777), (2, 97, 777), (4, 96, 4096),
                                   (2, 128, 4104), (9, 32, 16384)], ids=str)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_layer_norm_non_finite_grid_points_stay_alone(shape, dtype):
    """One point's NaN or infinity makes that point NaN in y, dx and dgamma, and
    leaves every other point of y and dx, and dbeta, as they were."""
    import torch
    outer, C, inner = shape
    g = torch.Generator(device="cuda").manual_seed(31)
    dt = torch_dtype(dtype)
    x, dy = (torch.randn(shape, generator=g, device="cuda").to(dt) for _ in range(2))
    gamma = (1 + 0.2 * torch.randn(C, generator=g, device="cuda")).to(dt)
    d = capi.layer_norm_desc(outer, C, inner, dtype, EPS)

    def both(v):
        y, dx = torch.empty_like(v), torch.empty_like(v)
        mean, rstd = (torch.empty((outer, inner), device="cuda") for _ in range(2))
        dg, db = (torch.empty(C, device="cuda") for _ in range(2))
        capi.fno_layer_norm_fwd(d, v, gamma, None, y, mean, rstd)
        capi.fno_layer_norm_bwd(d, v, gamma, mean, rstd, dy, dx, dg, db)
        return y, dx, dg, db

    y, dx, dg, db = both(x)
    assert bool(torch.isfinite(dg).all())
    for bad in (np.nan, np.inf, -np.inf):
        for b, at in ((0, 0), (outer - 1, inner - 1), (outer // 2, inner // 2)):
            z = x.clone()
            z[b, C // 3, at] = bad
            y2, dx2, dg2, db2 = both(z)
            for got, clean in ((y2, y), (dx2, dx)):
                assert bool(torch.isnan(got[b, :, at]).all())
                got[b, :, at] = clean[b, :, at]
                assert torch.equal(got, clean)
            assert bool(torch.isnan(dg2).all()) and torch.equal(db2, db)


@pytest.mark.parametrize("shape", [(2, 20, 64), (2, 20, 35), (8, 64, 1), (4, 1001, 1),
                                   (1, 1100, 8), (2, 33001, 1), (2, 200, 16)], ids=str)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_layer_norm_constant_and_non_finite_points(shape, dtype):
    """A constant point gives beta (its deviations vanish); a point with a NaN or
    an infinity becomes NaN and leaves every other point's bits alone."""
    import torch
    outer, C, inner = shape
    x, gamma, beta, _ = _inputs(outer, C, inner, dtype, seed=8)
    x[0, :, 0] = 3.0
    d = capi.layer_norm_desc(outer, C, inner, dtype, EPS)
    gd, bd = _dev(gamma, dtype), _dev(beta, dtype)
    clean = torch.empty(x.shape, dtype=torch_dtype(dtype), device="cuda")
    capi.fno_layer_norm_fwd(d, _dev(x, dtype), gd, bd, clean)
    # deviations of a constant point: at most C u 3 from the first mean's
    # rounding, corrected by their own mean to C u of that; rstd <= eps^-1/2
    tol = (C * U * 3.0) * (C + 4) * U * EPS ** -0.5 * np.abs(gamma) + HALF[dtype] * np.abs(beta)
    assert np.all(np.abs(_host(clean)[0, :, 0] - beta) <= tol + 4 * U * np.abs(beta) + TINY[dtype])
    pts = outer * inner
    for bad in (np.nan, np.inf, -np.inf):
        z = x.copy()
        flat = z.transpose(0, 2, 1).reshape(pts, C)
        at = pts // 2
        flat[at, C // 3] = bad
        z = flat.reshape(outer, inner, C).transpose(0, 2, 1)
        y = torch.empty_like(clean)
        capi.fno_layer_norm_fwd(d, _dev(z, dtype), gd, bd, y)
        got = y.permute(0, 2, 1).reshape(pts, C)
        ref = clean.permute(0, 2, 1).reshape(pts, C)
        assert bool(torch.isnan(got[at]).all())
        keep = torch.arange(pts, device="cuda") != at
        assert torch.equal(got[keep], ref[keep])


def test_layer_norm_gradient_by_differences():
    """The kernels' gradients against differences of the kernels' own forward,
    float32: the loss is summed in float64 on the host; a step of 2^-6 leaves a
    truncation error of h^2 / 6 of third derivatives of order one (4e-5) and a
    rounding error of 64 values' 2^-22 over h (below 1e-3 in all)."""
    import torch
    outer, C, inner = 1, 12, 5
    x, gamma, beta, dy = _inputs(outer, C, inner, "f32", seed=9)
    d = capi.layer_norm_desc(outer, C, inner, "f32", EPS)
    y = torch.empty(x.shape, device="cuda")
    mean, rstd = torch.empty(outer, inner, device="cuda"), torch.empty(outer, inner, device="cuda")
    capi.fno_layer_norm_fwd(d, _dev(x), _dev(gamma), _dev(beta), y, mean, rstd)
    dx, dg, db = torch.empty_like(y), torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    capi.fno_layer_norm_bwd(d, _dev(x), _dev(gamma), mean, rstd, _dev(dy), dx, dg, db)

    def loss(x_, g_, b_):
        capi.fno_layer_norm_fwd(d, _dev(x_), _dev(g_), _dev(b_), y)
        return float((_host(y) * dy).sum())

    h = 2.0 ** -6
    for args, grad in ((0, dx), (1, dg), (2, db)):
        base = [x, gamma, beta]
        for idx in list(np.ndindex(base[args].shape))[::7]:
            up, dn = [a.copy() for a in base], [a.copy() for a in base]
            up[args][idx] += h
            dn[args][idx] -= h
            step = float(np.float32(up[args][idx])) - float(np.float32(dn[args][idx]))
            num = (loss(*up) - loss(*dn)) / step
            assert abs(num - _host(grad)[idx]) <= 3e-3 * max(1.0, abs(num))


@pytest.mark.parametrize("shape", [(4, 20, 4096), (3, 64, 4099), (500, 96, 1), (4, 2050, 1),
                                   (3, 64, 24008), (2, 20, 120000)], ids=str)
def test_layer_norm_on_streams_and_in_a_graph(shape):
    """Two calls at once on two streams with their own workspaces, and a captured
    forward + backward replayed on new inputs: the same bits as plain calls."""
    import torch
    outer, C, inner = shape
    d = capi.layer_norm_desc(outer, C, inner, "bf16", EPS)
    sets = [_inputs(outer, C, inner, "bf16", seed=s) for s in (10, 11)]

    def buffers():
        e = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
        b = torch.bfloat16
        return dict(y=e(outer, C, inner, dt=b), mean=e(outer, inner), rstd=e(outer, inner),
                    dx=e(outer, C, inner, dt=b), dg=e(C), db=e(C),
                    ws=e(capi.fno_layer_norm_workspace_size(d), dt=torch.uint8))

    def call(i, o, stream=None):
        capi.fno_layer_norm_fwd(d, i[0], i[1], i[2], o["y"], o["mean"], o["rstd"], stream=stream)
        capi.fno_layer_norm_bwd(d, i[0], i[1], o["mean"], o["rstd"], i[3], o["dx"], o["dg"],
                                o["db"], ws=o["ws"], stream=stream)

    ins = [[_dev(a, "bf16") for a in s] for s in sets]
    want = []
    for i in ins:
        o = buffers()
        call(i, o)
        want.append(o)
    torch.cuda.synchronize()
    outs = [buffers(), buffers()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for i, o, s in zip(ins, outs, streams):
            call(i, o, s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(o[k], w[k]) for k in w if k != "ws")
    live = [t.clone() for t in ins[0]]
    o = buffers()
    call(live, o)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(live, o)
    for t, src in zip(live, ins[1]):
        t.copy_(src)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o[k], want[1][k]) for k in want[1] if k != "ws")


@pytest.mark.parametrize("dtype,shape", [("bf16", (8, 32, 1 << 16)), ("bf16", (4, 64, 1 << 16)),
                                         ("f32", (16, 8, 1 << 16)), ("f32", (4, 64, 1 << 16))])
def test_layer_norm_expired_wait_is_reported(dtype, shape):
    """With the wait limit at a single probe some of the pipelines' waits give up: the
    call reports it, and the next one with the default limit gives the same bits as
    before."""
    import torch
    outer, C, inner = shape
    g = torch.Generator(device="cuda").manual_seed(5)
    dt = torch_dtype(dtype)
    x, dy = (torch.randn(shape, generator=g, device="cuda").to(dt) for _ in range(2))
    gamma = torch.ones(C, device="cuda", dtype=dt)
    d = capi.layer_norm_desc(outer, C, inner, dtype, EPS)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = (torch.empty((outer, inner), device="cuda") for _ in range(2))
    dg, db = (torch.empty(C, device="cuda") for _ in range(2))
    fwd = lambda: capi.fno_layer_norm_fwd(d, x, gamma, None, y, mean, rstd)  # noqa: E731
    bwd = lambda: capi.fno_layer_norm_bwd(d, x, gamma, mean, rstd, dy, dx, dg, db)  # noqa: E731
    capi.fno_device_error(clear=True)
    fwd()
    bwd()
    capi.fno_device_error(clear=True)
    kept = [t.clone() for t in (y, mean, rstd, dx, dg, db)]
    for call in (bwd, fwd) if dtype != "f32" else (bwd,):
        prev = capi.fno_set_wait_limit(0)
        try:
            call()
            torch.cuda.synchronize()
            with pytest.raises(capi.FnoError) as info:
                capi.fno_device_error(clear=True)
            assert info.value.code == capi.FNO_ERR_TIMEOUT
        finally:
            capi.fno_set_wait_limit(prev)
    fwd()
    bwd()
    capi.fno_device_error(clear=True)
    for a, b in zip(kept, (y, mean, rstd, dx, dg, db)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("shape", [(33, 64, 1 << 20), ((1 << 20) + 3, 2049, 1)], ids=str)
def test_layer_norm_offsets_beyond_32_bits(shape):
    """More than 2^31 elements: the last points against the oracle, and the
    parameter gradient of a cotangent that is nonzero there alone."""
    import torch
    outer, C, inner = shape
    d = capi.layer_norm_desc(outer, C, inner, "bf16", EPS)
    x, gamma, beta, dy = _inputs(1, C, 64 if inner > 1 else 1, "bf16", seed=12)
    big = torch.zeros(outer, C, inner, dtype=torch.bfloat16, device="cuda")
    tail = big[-1:, :, -64:]
    tail.copy_(_dev(x, "bf16"))
    gd, bd = _dev(gamma, "bf16"), _dev(beta, "bf16")
    y = torch.empty_like(big)
    mean, rstd = torch.empty(outer, inner, device="cuda"), torch.empty(outer, inner, device="cuda")
    capi.fno_layer_norm_fwd(d, big, gd, bd, y, mean, rstd)
    n = x.shape[2]
    _check_fwd(y[-1:, :, -64:], mean[-1:, -n:], rstd[-1:, -n:], x, gamma, beta, "bf16")
    assert torch.equal(y[0, :, 0], bd) and torch.equal(y[outer // 2, :, 0], bd)
    m64, r64 = _host(mean[-1:, -n:]), _host(rstd[-1:, -n:])
    y.zero_()                                       # now the cotangent
    y[-1:, :, -64:].copy_(_dev(dy, "bf16"))
    dg, db = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    capi.fno_layer_norm_bwd(d, big, gd, mean, rstd, y, y, dg, db)
    _check_bwd(y[-1:, :, -64:], dg, db, x, gamma, m64, r64, dy, "bf16", terms=4096)
    assert not bool(y[0].any())


# ---------------------------------------------------------------------------
# gradient norm and clipping
# ---------------------------------------------------------------------------

LISTS = {
    "one": [1], "empty": [0], "empties": [0, 0, 5, 0], "pair": [7, 4099],
    "chunks": [8192, 8191, 8193, 16384, 16385, 3], "large": [3_000_001, 12, 1_500_000],
    "many": [1 + (i * 37) % 977 for i in range(700)],
    # around the numbers of tensors and of 4 KB chunks that one launch takes
    "few": [5] * 64, "few+1": [5] * 65, "few+0": [5] * 64 + [0] * 3,
    "one-cta": [1 << 15], "one-cta+1": [1 << 15, 1], "one-cta-many": [700] * 32,
    "some": [1300] * 384, "some+1": [1300] * 385, "medium": [1 << 20, 1],
    "table": [1100] * 1024, "table+1": [1100] * 1025, "table+0": [1100] * 1024 + [0, 0],
    "tables": [3 + (i * 91) % 5000 for i in range(2300)],
}


def _grad_arrays(sizes, dtype, seed=3):
    rng = np.random.default_rng(seed)
    return [synth.quantize(rng.standard_normal(n) * np.exp(rng.uniform(-4, 2)), dtype)
            for n in sizes]


# Relative tolerances of the norm: float64 sums of groups whose squares are off
# by at most 8 u each (a group of 8 in float32), halved by the root, and one
# rounding to float32; the factor adds one rounding.
NORM_TOL = 6 * U


@pytest.mark.parametrize("name", list(LISTS))
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_grad_norm_and_clip_match_oracle(name, dtype):
    import torch
    arrays = _grad_arrays(LISTS[name], dtype)
    full, _ = O.grad_norm(arrays)
    for max_norm, scale in ((0.3 * full, 1.0), (2.0 * full, 1.0), (0.25 * full, -0.5),
                            (np.inf, 0.125), (0.0, 1.0)):
        ref, factor = O.grad_norm(arrays, np.float64(np.float32(max_norm)), scale)
        grads = [_dev(a, dtype) for a in arrays]
        norm = torch.full((2,), 9.0, device="cuda")
        capi.fno_grad_norm(grads, max_norm, norm, grad_scale=scale)
        got = _host(norm)
        assert abs(got[0] - ref) <= NORM_TOL * ref
        assert abs(got[1] - factor) <= 2 * NORM_TOL * factor
        # into other tensors, then in place: the same bits
        outs = [_bands((max(n, 1),), dtype) for n in LISTS[name]]
        outs = [(o[:n], buf) for (o, buf), n in zip(outs, LISTS[name])]
        norm2 = torch.empty(2, device="cuda")
        capi.fno_clip_grads(capi.grad_list(grads, [o for o, _ in outs]), max_norm, norm2,
                            grad_scale=scale)
        assert torch.equal(norm2, norm)
        for a, (o, buf) in zip(arrays, outs):
            want = a * scale * got[1]
            # the multiplier's rounding, the product's, the storage's
            tol = 2 * U * np.abs(want) + HALF[dtype] * np.abs(want) * (1 + 4 * U) + TINY[dtype]
            assert np.all(np.abs(_host(o) - want) <= tol)
            assert bool((buf[:32] == 7).all()) and bool((buf[32 + max(a.size, 1):] == 7).all())
        norm3 = torch.empty(2, device="cuda")
        capi.fno_clip_grads(grads, max_norm, norm3, grad_scale=scale)
        assert torch.equal(norm3, norm)
        assert all(torch.equal(g, o) for g, (o, _) in zip(grads, outs))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e-30, 1e-22, 1e30, 1e18])
def test_grad_norm_squares_beyond_float32(dtype, size):
    """Squares that float32 flushes to zero or overflows: the norm is exact to
    the same tolerance, and the clipped gradients are finite."""
    import torch
    rng = np.random.default_rng(4)
    arrays = [synth.quantize(rng.standard_normal(n) * size, dtype) for n in (1000, 5, 8193)]
    ref, factor = O.grad_norm(arrays, np.float64(np.float32(1e-3 * size)))
    grads = [_dev(a, dtype) for a in arrays]
    norm = torch.empty(2, device="cuda")
    capi.fno_clip_grads(grads, 1e-3 * size, norm)
    got = _host(norm)
    assert abs(got[0] - ref) <= NORM_TOL * ref
    assert abs(got[1] - factor) <= 2 * NORM_TOL * factor
    assert all(bool(torch.isfinite(g).all()) for g in grads)


@pytest.mark.parametrize("bad,norm,factor", [(np.nan, np.nan, np.nan), (np.inf, np.inf, 0.0),
                                             (-np.inf, np.inf, 0.0)])
def test_clip_non_finite_gradients(bad, norm, factor):
    """A NaN makes the norm, the factor and every gradient NaN; an infinity gives
    the norm infinity and the factor 0: finite gradients become 0, it becomes NaN."""
    import torch
    g = [torch.ones(5000, device="cuda"), torch.ones(3, device="cuda")]
    g[0][4097] = bad
    out = torch.empty(2, device="cuda")
    capi.fno_clip_grads(g, 1.0, out)
    np.testing.assert_array_equal(_host(out), [norm, factor])
    got = np.concatenate([_host(t) for t in g])
    want = np.zeros(5003) * (np.nan if np.isnan(bad) else 1.0)
    want[4097] = np.nan
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_clip_unaligned_views(dtype):
    """Tensors at any element offset (views into one buffer), in and out offset
    differently; the elements between them stay as they were."""
    import torch
    rng = np.random.default_rng(5)
    offs, sizes = [1, 11, 40, 20003], [7, 23, 19950, 9001]
    base = synth.quantize(rng.standard_normal(30000), dtype)
    src = _dev(base, dtype)
    dst = torch.full((30010,), 7.0, dtype=torch_dtype(dtype), device="cuda")
    grads = [src[o:o + n] for o, n in zip(offs, sizes)]
    outs = [dst[o + 3:o + 3 + n] for o, n in zip(offs, sizes)]
    arrays = [base[o:o + n] for o, n in zip(offs, sizes)]
    ref, factor = O.grad_norm(arrays, 2.0)
    norm = torch.empty(2, device="cuda")
    capi.fno_clip_grads(capi.grad_list(grads, outs), 2.0, norm)
    assert abs(float(norm[0]) - ref) <= NORM_TOL * ref
    mask = np.ones(30010, bool)
    for o, n, a in zip(offs, sizes, arrays):
        mask[o + 3:o + 3 + n] = False
        want = a * float(norm[1])
        got = _host(dst[o + 3:o + 3 + n])
        assert np.all(np.abs(got - want) <= (HALF[dtype] + 2 * U) * np.abs(want) + TINY[dtype])
    assert bool((dst[torch.from_numpy(mask).cuda()] == 7).all())
    assert np.array_equal(_host(src), base)


def test_grad_norm_beyond_32_bits_and_repeatable():
    """A tensor of more than 2^31 elements, nonzero at its end alone; and two
    calls on the same values give the same bits."""
    import torch
    g = torch.zeros((1 << 31) + 9, dtype=torch.bfloat16, device="cuda")
    g[-3:] = 2.0
    norm = torch.empty(2, device="cuda")
    capi.fno_clip_grads([g], 1.0, norm)
    np.testing.assert_allclose(_host(norm), [np.sqrt(12), 1 / np.sqrt(12)], rtol=2 * U)
    np.testing.assert_allclose(_host(g[-4:]), [0] + [2 / np.sqrt(12)] * 3, rtol=HALF["bf16"] + 2 * U)
    del g
    h = [torch.randn(n, device="cuda") for n in (1 << 22, 1001, 77777)]
    a, b = torch.empty(2, device="cuda"), torch.empty(2, device="cuda")
    capi.fno_grad_norm(h, 1.0, a)
    capi.fno_grad_norm(h, 1.0, b)
    assert torch.equal(a, b)


def test_clip_on_streams_and_in_graphs():
    """Concurrent calls on two streams with their own workspaces; two captured
    graphs that share one workspace, replayed one after the other."""
    import torch
    arrays = [_grad_arrays([70000, 33, 4100], "f32", seed=s) for s in (20, 21)]
    want = []
    for arr in arrays:
        g = [_dev(a) for a in arr]
        norm = torch.empty(2, device="cuda")
        capi.fno_clip_grads(g, 1.0, norm)
        want.append((g, norm))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for arr, s in zip(arrays, streams):
        src = [_dev(a) for a in arr]
        out = [torch.empty_like(t) for t in src]
        got.append((capi.grad_list(src, out), out, torch.empty(2, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(4):
        for (gl, _, norm), s in zip(got, streams):
            capi.fno_clip_grads(gl, 1.0, norm, stream=s)      # workspaces from the binding
    torch.cuda.synchronize()
    for (_, out, norm), (wg, wn) in zip(got, want):
        assert torch.equal(norm, wn) and all(torch.equal(a, b) for a, b in zip(out, wg))
    ws = torch.empty(capi.fno_grad_norm_workspace_size(got[0][0]), dtype=torch.uint8, device="cuda")
    graphs = []
    for gl, out, norm in got:
        for t in out:
            t.zero_()
        norm.zero_()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            capi.fno_clip_grads(gl, 1.0, norm, ws=ws)
        graphs.append(gr)
    for _ in range(2):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    for (_, out, norm), (wg, wn) in zip(got, want):
        assert torch.equal(norm, wn) and all(torch.equal(a, b) for a, b in zip(out, wg))


# ---------------------------------------------------------------------------
# the clipped Adam step
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("n", [1, 7, 4099, (1 << 20) + 3])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_adam_step_clipped_matches_oracle(n, dtype):
    """Three steps, the second and third clipped.  Bounds as for the plain Adam
    step: moments to a few units of the largest |g|, theta to 1e-5 of lr per step."""
    import torch
    rng = np.random.default_rng(21)
    theta = rng.standard_normal(n).astype(np.float32)
    lr, b1, b2, eps, wd, scale = 3e-3, 0.9, 0.99, 1e-6, 0.01, 0.5
    t_d = torch.from_numpy(theta).cuda()
    m_d, v_d = torch.zeros_like(t_d), torch.zeros_like(t_d)
    out = torch.empty(n, dtype=torch_dtype(dtype), device="cuda")
    norm = torch.empty(2, device="cuda")
    th, m, v = theta.astype(np.float64), np.zeros(n), np.zeros(n)
    gmax = 0.0
    for step, part in ((1, 3.0), (2, 0.4), (3, 0.1)):
        g = (rng.standard_normal(n) * np.exp(rng.uniform(-3, 1, n))).astype(np.float32)
        g_d = torch.from_numpy(g).cuda()
        limit = float(np.float32(part * scale * np.linalg.norm(g.astype(np.float64))))
        capi.fno_grad_norm([g_d], limit, norm, grad_scale=scale)
        capi.fno_adam_step_clipped(t_d, m_d, v_d, g_d, out, step, lr, norm, b1, b2, eps, wd, scale)
        _, factor = O.grad_norm([g], limit, scale)
        gmax = max(gmax, float(np.abs(g).max()) * scale)
        th, m, v = O.adam_update(th, m, v, g.astype(np.float64) * scale * factor, step, lr, b1, b2,
                                 eps, wd)
    torch.cuda.synchronize()
    np.testing.assert_allclose(m_d.cpu().numpy(), m, rtol=1e-5, atol=2.0 ** -21 * gmax)
    np.testing.assert_allclose(v_d.cpu().numpy(), v, rtol=1e-5, atol=2.0 ** -21 * gmax ** 2)
    np.testing.assert_allclose(t_d.cpu().numpy(), th, rtol=2.0 ** -20, atol=3 * 1e-5 * lr)
    np.testing.assert_array_equal(_host(out), O.round_to_storage(t_d.cpu().numpy(), dtype))


@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_adam_step_skips_a_norm_that_is_not_finite(bad):
    import torch
    n = 5001
    t, m, v, g = (torch.randn(n, device="cuda") for _ in range(4))
    v = v.abs()
    before = [a.clone() for a in (t, m, v)]
    g[77] = bad
    norm = torch.empty(2, device="cuda")
    out = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    capi.fno_grad_norm([g], 1.0, norm)
    capi.fno_adam_step_clipped(t, m, v, g, out, 3, 1e-3, norm, skip_nonfinite=True)
    assert all(torch.equal(a, b) for a, b in zip((t, m, v), before))
    assert torch.equal(out, t.bfloat16())
    capi.fno_adam_step_clipped(t, m, v, g, out, 3, 1e-3, norm)     # not skipped: NaN as the formula
    assert bool(torch.isnan(t[77])) and bool(torch.isnan(out[77]))
    # a finite norm is stepped with the flag as without it
    g[77] = 0.5
    capi.fno_grad_norm([g], 1.0, norm)
    a = [b.clone() for b in before]
    b = [x.clone() for x in before]
    capi.fno_adam_step_clipped(*a, g, None, 3, 1e-3, norm, skip_nonfinite=True)
    capi.fno_adam_step_clipped(*b, g, None, 3, 1e-3, norm)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and not torch.equal(a[0], before[0])
