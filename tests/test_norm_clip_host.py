"""Layer norm, gradient norm and clipping on the CPU: the oracle's formulas against
closed forms and finite differences, and every refused argument (validation runs
before anything touches a device)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import oracle as O
from fourier_neural_spectral_fno_b200 import build, capi


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


# ---------------------------------------------------------------- the oracle

def test_oracle_layer_norm_closed_forms():
    # two channels: xh = +-d / sqrt(d^2 + eps), d half their difference
    x = np.array([[[3.0, 1.0], [1.0, 1.0]]])
    y, mean, rstd = O.layer_norm_fwd(x, eps=0.5)
    np.testing.assert_allclose(mean, [[2.0, 1.0]])
    np.testing.assert_allclose(rstd, [[1 / math.sqrt(1.5), 1 / math.sqrt(0.5)]])
    np.testing.assert_allclose(y, [[[1 / math.sqrt(1.5), 0.0], [-1 / math.sqrt(1.5), 0.0]]])
    y, _, _ = O.layer_norm_fwd(x, np.array([2.0, 3.0]), np.array([0.5, -1.0]), eps=0.5)
    np.testing.assert_allclose(y[0, :, 0], [0.5 + 2 / math.sqrt(1.5), -1 - 3 / math.sqrt(1.5)])
    # mean 0 and variance C / (C + C eps / var) over the channels
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 7, 4, 5)) * 2 + 9
    y, mean, rstd = O.layer_norm_fwd(x)
    np.testing.assert_allclose(y.mean(1), 0, atol=1e-12)
    np.testing.assert_allclose((y ** 2).mean(1), x.var(1) / (x.var(1) + 1e-5))


def test_oracle_layer_norm_gradient_by_differences():
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((2, 6, 3)), rng.standard_normal((2, 6, 3))
    gamma, beta = rng.standard_normal(6), rng.standard_normal(6)
    _, mean, rstd = O.layer_norm_fwd(x, gamma, beta)
    dx, dgamma, dbeta = O.layer_norm_bwd(x, gamma, mean, rstd, dy)

    def loss(x_, g_, b_):
        return float((O.layer_norm_fwd(x_, g_, b_)[0] * dy).sum())

    h = 1e-6
    for idx in [(0, 0, 0), (1, 5, 2), (0, 3, 1)]:
        d = np.zeros_like(x)
        d[idx] = h
        num = (loss(x + d, gamma, beta) - loss(x - d, gamma, beta)) / (2 * h)
        assert abs(num - dx[idx]) < 1e-7
    for c in range(6):
        d = np.zeros(6)
        d[c] = h
        assert abs((loss(x, gamma + d, beta) - loss(x, gamma - d, beta)) / (2 * h) - dgamma[c]) < 1e-7
        assert abs((loss(x, gamma, beta + d) - loss(x, gamma, beta - d)) / (2 * h) - dbeta[c]) < 1e-7


def test_oracle_grad_norm():
    assert O.grad_norm([np.array([3.0]), np.zeros(0), np.array([[4.0]])]) == (5.0, 1.0)
    assert O.grad_norm([np.array([3.0, 4.0])], max_norm=2.0) == (5.0, 0.4)
    assert O.grad_norm([np.array([3.0, 4.0])], max_norm=2.0, scale=-0.5) == (2.5, 0.8)
    assert O.grad_norm([np.zeros(3)], max_norm=0.0) == (0.0, 1.0)
    assert O.grad_norm([np.array([3 + 4j])]) == (5.0, 1.0)      # complex weights: (re, im)


# --------------------------------------------------------- C entry points

def _desc(**kw):
    d = capi.layer_norm_desc(2, 8, 16)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw,code,word", [
    ({"dtype": 3}, capi.FNO_ERR_INVALID_ARG, "dtype"),
    ({"dtype": -1}, capi.FNO_ERR_INVALID_ARG, "dtype"),
    ({"outer": 0}, capi.FNO_ERR_INVALID_ARG, "outer 0"),
    ({"inner": 0}, capi.FNO_ERR_INVALID_ARG, "inner 0"),
    ({"inner": -4}, capi.FNO_ERR_INVALID_ARG, "inner -4"),
    ({"channels": 0}, capi.FNO_ERR_INVALID_ARG, "channels 0"),
    ({"channels": (1 << 20) + 1}, capi.FNO_ERR_UNSUPPORTED, "channels"),
    ({"outer": 1 << 40}, capi.FNO_ERR_UNSUPPORTED, "elements"),
    ({"outer": 1 << 62, "inner": 1 << 62}, capi.FNO_ERR_UNSUPPORTED, "elements"),
    ({"eps": 0.0}, capi.FNO_ERR_INVALID_ARG, "eps"),
    ({"eps": -1.0}, capi.FNO_ERR_INVALID_ARG, "eps"),
    ({"eps": float("nan")}, capi.FNO_ERR_INVALID_ARG, "eps"),
    ({"eps": float("inf")}, capi.FNO_ERR_INVALID_ARG, "eps"),
])
def test_layer_norm_refuses_descriptors(lib, kw, code, word):
    d = ctypes.byref(_desc(**kw))
    assert lib.fno_layer_norm_workspace_size(d) == 0
    assert word in capi.last_error()
    assert lib.fno_layer_norm_fwd(d, 256, 256, 256, 256, None, None, None) == code
    assert lib.fno_layer_norm_bwd(d, 256, 256, 256, 256, 256, 512, 256, 256, 256, 1 << 30,
                                  None) == code
    assert word in capi.last_error()


def test_layer_norm_refuses_pointers(lib):
    d = _desc()
    need = capi.fno_layer_norm_workspace_size(d)
    r = ctypes.byref(d)
    fwd = dict(x=256, gamma=256, beta=256, y=256, mean=256, rstd=256)
    bwd = dict(x=256, gamma=256, mean=256, rstd=256, dy=256, dx=512, dgamma=256, dbeta=256, ws=256)

    def f(**kw):
        return lib.fno_layer_norm_fwd(r, *dict(fwd, **kw).values(), None)

    def b(nb=need, **kw):
        return lib.fno_layer_norm_bwd(r, *dict(bwd, **kw).values(), nb, None)

    assert lib.fno_layer_norm_fwd(None, *fwd.values(), None) == capi.FNO_ERR_INVALID_ARG
    assert lib.fno_layer_norm_bwd(None, *bwd.values(), need, None) == capi.FNO_ERR_INVALID_ARG
    for name in ("x", "y"):
        assert f(**{name: None}) == capi.FNO_ERR_INVALID_ARG and name in capi.last_error()
    for name in fwd:
        assert f(**{name: 0x108}) == capi.FNO_ERR_INVALID_ARG
        assert f"{name} is not 16-byte aligned" in capi.last_error()
    for kw in ({"mean": None}, {"rstd": None}):
        assert f(**kw) == capi.FNO_ERR_INVALID_ARG and "both or neither" in capi.last_error()
    for name in ("x", "mean", "rstd", "dy", "dx", "ws"):
        assert b(**{name: None}) == capi.FNO_ERR_INVALID_ARG and name in capi.last_error()
    for name in bwd:
        assert b(**{name: 0x108}) == capi.FNO_ERR_INVALID_ARG
        assert f"{name} is not 16-byte aligned" in capi.last_error()
    assert b(dx=256, x=256) == capi.FNO_ERR_INVALID_ARG and "overlaps" in capi.last_error()
    assert b(nb=need - 1) == capi.FNO_ERR_WORKSPACE


def _grad_args(sizes=(4, 0, 7), ptrs=(256, 0, 512)):
    n = len(sizes)
    return n, (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*sizes)


def test_grad_norm_refuses(lib):
    n, g, s = _grad_args()
    need = capi.fno_grad_norm_workspace_size(n)
    assert lib.fno_grad_norm_workspace_size(0) == 0 and "n_tensors 0" in capi.last_error()
    assert capi.fno_grad_norm_workspace_size(2000) > need

    def call(n=n, g=g, s=s, dtype=0, scale=1.0, mx=1.0, norm=256, ws=256, nb=need):
        rc = lib.fno_grad_norm(n, g, s, dtype, scale, mx, norm, ws, nb, None)
        out = (ctypes.c_void_p * 3)(256, 0, 512)
        assert lib.fno_clip_grads(n, g, out, s, dtype, scale, mx, norm, ws, nb, None) == rc
        return rc

    bad = capi.FNO_ERR_INVALID_ARG
    for kw, word in [({"n": 0}, "n_tensors 0"), ({"n": -1}, "n_tensors -1"), ({"g": None}, "grads"),
                     ({"s": None}, "sizes"), ({"dtype": 3}, "dtype"),
                     ({"scale": float("inf")}, "grad_scale"), ({"scale": float("nan")}, "grad_scale"),
                     ({"mx": -1.0}, "max_norm"), ({"mx": float("nan")}, "max_norm"),
                     ({"norm": None}, "norm"), ({"norm": 0x102}, "norm"),
                     ({"ws": None}, "ws"), ({"ws": 0x108}, "ws"),
                     ({"s": _grad_args((4, -1, 7))[2]}, "sizes[1]"),
                     ({"g": _grad_args(ptrs=(256, 0, 0))[1]}, "grads[2]"),
                     ({"g": _grad_args(ptrs=(0x102, 0, 512))[1]}, "grads[0]"),
                     ({"g": _grad_args(ptrs=(0x101, 0, 512))[1], "dtype": 2}, "grads[0]")]:
        assert call(**kw) == bad, kw
        assert word in capi.last_error(), kw
    assert call(nb=need - 1) == capi.FNO_ERR_WORKSPACE
    assert call(s=_grad_args((1 << 40, 0, 1))[2]) == capi.FNO_ERR_UNSUPPORTED
    assert call(s=_grad_args((1 << 62, 1 << 62, 1 << 62))[2]) == capi.FNO_ERR_UNSUPPORTED
    assert lib.fno_clip_grads(n, g, None, s, 0, 1.0, 1.0, 256, 256, need, None) == bad
    for ptrs, word in [((256, 0, 0), "out[2]"), ((0x101, 0, 256), "out[0]")]:
        out = (ctypes.c_void_p * 3)(*ptrs)
        assert lib.fno_clip_grads(n, g, out, s, 0, 1.0, 1.0, 256, 256, need, None) == bad
        assert word in capi.last_error()


def test_adam_step_clipped_refuses(lib):
    def call(**kw):
        a = dict(n=8, theta=256, m=256, v=256, grad=256, out=256, od=2, step=1, lr=1e-3, b1=0.9,
                 b2=0.999, eps=1e-8, wd=0.0, scale=1.0, norm=256, skip=0)
        a.update(kw)
        return lib.fno_adam_step_clipped(*a.values(), None)

    for kw, word in [({"n": 0}, "n 0"), ({"theta": None}, "theta"), ({"grad": None}, "grad"),
                     ({"norm": None}, "norm"), ({"norm": 0x102}, "norm"), ({"step": 0}, "step 0"),
                     ({"eps": 0.0}, "eps"), ({"od": 5}, "out_dtype"), ({"b2": 1.0}, "betas"),
                     ({"scale": float("nan")}, "grad_scale")]:
        assert call(**kw) == capi.FNO_ERR_INVALID_ARG, kw
        assert word in capi.last_error(), kw


# ------------------------------------------------------------- the binding

@pytest.fixture
def host_tensors(monkeypatch):
    """Let host tensors pass the binding's device check, for calls that the library
    refuses before anything touches a device."""
    monkeypatch.setattr(capi, "_device_index", lambda t, name: t.get_device())


def test_binding_refuses_host_tensors(lib):
    d = capi.layer_norm_desc(2, 8, 16)
    x, c, s = torch.zeros(2, 8, 16), torch.zeros(8), torch.zeros(2, 16)
    with pytest.raises(ValueError, match="x is on cpu"):
        capi.fno_layer_norm_fwd(d, x, c, c, x)
    with pytest.raises(ValueError, match="x is on cpu"):
        capi.fno_layer_norm_bwd(d, x, c, s, s, x, x.clone())
    with pytest.raises(ValueError, match="grads.0. is on cpu"):
        capi.fno_clip_grads([x], 1.0, torch.zeros(2))
    with pytest.raises(ValueError, match="theta is on cpu"):
        capi.fno_adam_step_clipped(c, c, c, c, None, 1, 1e-3, torch.zeros(2))


def test_binding_refuses_layer_norm_tensors(lib, host_tensors):
    d = capi.layer_norm_desc(2, 8, 16)
    x = torch.zeros(2, 8, 16)
    c, s = torch.zeros(8), torch.zeros(2, 16)
    for kw, word in [({"x": x.double()}, "x is"), ({"y": x[:, :4]}, "y has"),
                     ({"y": torch.zeros(8, 2, 16).transpose(0, 1)}, "y is not contiguous"),
                     ({"gamma": c.half()}, "gamma is"), ({"beta": c[:4]}, "beta has"),
                     ({"mean": s.half()}, "mean is"), ({"rstd": s[:1]}, "rstd has")]:
        args = dict(x=x, gamma=c, beta=c, y=x.clone(), mean=s, rstd=s)
        args.update(kw)
        with pytest.raises(ValueError, match=word):
            capi.fno_layer_norm_fwd(d, stream=0, **args)
    for kw, word in [({"dy": x.half()}, "dy is"), ({"dx": x[:1]}, "dx has"),
                     ({"dgamma": c.half()}, "dgamma is"), ({"dbeta": c[:4]}, "dbeta has")]:
        args = dict(x=x, gamma=c, mean=s, rstd=s, dy=x.clone(), dx=x.clone(), dgamma=c, dbeta=c)
        args.update(kw)
        with pytest.raises(ValueError, match=word):
            capi.fno_layer_norm_bwd(d, stream=0, **args)


@pytest.mark.parametrize("fn,arg", [("fwd", a) for a in ("x", "gamma", "beta", "y", "mean", "rstd")]
                         + [("bwd", a) for a in ("x", "gamma", "mean", "rstd", "dy", "dx",
                                                 "dgamma", "dbeta")])
def test_binding_passes_each_pointer_in_place(lib, host_tensors, fn, arg):
    d = capi.layer_norm_desc(2, 8, 16)
    n = {"gamma": 8, "beta": 8, "dgamma": 8, "dbeta": 8, "mean": 32, "rstd": 32}

    def buf(name):
        t = torch.zeros(n.get(name, 256) + 1)
        return t[1:] if name == arg else t[:-1]

    names = ("x", "gamma", "beta", "y", "mean", "rstd") if fn == "fwd" else \
        ("x", "gamma", "mean", "rstd", "dy", "dx", "dgamma", "dbeta")
    with pytest.raises(capi.FnoError, match=f": {arg} is not 16-byte aligned"):
        getattr(capi, "fno_layer_norm_" + fn)(d, stream=0, **{k: buf(k) for k in names})


def test_binding_refuses_gradient_lists(lib, host_tensors):
    g = [torch.zeros(5), torch.zeros(0), torch.zeros(3, 2)]
    assert capi.grad_list(g).n == 3
    flat = torch.zeros(16)
    for grads, out, word in [
            ([], None, "no gradients"), ([torch.zeros(3, dtype=torch.float64)], None, "dtype"),
            ([g[0], g[2].half()], None, "grads.1. is"),
            ([torch.zeros(4, 4).t()], None, "contiguous"),
            (g, g[:2], "2 outputs for 3"), (g, [g[0], g[1], torch.zeros(5)], "out.2. has"),
            ([g[0], g[0]], None, "overlaps"), ([flat[:8], flat[7:]], None, "overlaps"),
            ([flat[:8], flat[8:]], [flat[8:], flat[:8]], "overlaps"),
            ([flat[:8]], [flat[4:12]], "overlaps"),
            ([flat[:2], flat[8:10]], [flat[4:6], flat[4:6]], "overlaps")]:
        with pytest.raises(ValueError, match=word):
            capi.grad_list(grads, out)
    capi.grad_list([flat[:8], flat[8:]])                       # neighbours may touch
    capi.grad_list([flat[:4], flat[4:8]], [flat[8:12], flat[12:]])
    with pytest.raises(ValueError, match="norm has"):
        capi.fno_grad_norm(g, 1.0, torch.zeros(1), stream=0)
    with pytest.raises(ValueError, match="norm is"):
        capi.fno_clip_grads(g, 1.0, torch.zeros(2).half(), stream=0)
    with pytest.raises(capi.FnoError, match="max_norm -1"):
        capi.fno_grad_norm(g, -1.0, torch.zeros(2), stream=0)
    with pytest.raises(capi.FnoError, match="grad_scale"):
        capi.fno_clip_grads(g, 1.0, torch.zeros(2), grad_scale=float("inf"), stream=0)


def test_binding_refuses_clipped_adam_tensors(lib, host_tensors):
    t = [torch.zeros(8) for _ in range(4)]
    norm = torch.zeros(2)
    for k, word in enumerate(("theta", "m", "v", "grad")):
        bad = list(t)
        bad[k] = torch.zeros(8).half()
        with pytest.raises(ValueError, match=word + " is"):
            capi.fno_adam_step_clipped(*bad, None, 1, 1e-3, norm, stream=0)
    with pytest.raises(ValueError, match="param_out has"):
        capi.fno_adam_step_clipped(*t, torch.zeros(4).half(), 1, 1e-3, norm, stream=0)
    with pytest.raises(ValueError, match="norm has"):
        capi.fno_adam_step_clipped(*t, None, 1, 1e-3, torch.zeros(3), stream=0)
    for kw, word in [({"step": 0}, "step 0"), ({"beta1": 1.5}, "betas"), ({"eps": -1.0}, "eps -1"),
                     ({"weight_decay": -3.0}, "weight_decay"), ({"grad_scale": math.inf},
                                                                "grad_scale")]:
        args = dict(step=1, lr=1e-3, norm=norm)
        args.update(kw)
        with pytest.raises(capi.FnoError, match=word):
            capi.fno_adam_step_clipped(*t, None, stream=0, **args)
