"""Skipped optimiser steps on the CPU: the trainer's host logic over a stand-in library,
and the refused arguments of fno_adam_step_skipping."""

import math

import numpy as np
import pytest
import torch

from fourier_neural_spectral_fno_b200 import build, capi
from fourier_neural_spectral_fno_b200.train import PrecisionSchedule
from test_norm_network_host import _FakeWithNorm, _network


class _FakeSkipping(_FakeWithNorm):
    """The stand-in whose clipped step keeps the count of skipped steps."""

    def fno_adam_step_clipped(self, theta, m, v, grad, out, step, lr, norm, beta1, beta2, eps,
                              weight_decay, grad_scale, skip_nonfinite):
        if isinstance(skip_nonfinite, capi.SkippedSteps):
            step -= skip_nonfinite.count()
            if not np.isfinite(float(norm[0])):
                skip_nonfinite.state[0] += 1
        super().fno_adam_step_clipped(theta, m, v, grad, out, step, lr, norm, beta1, beta2, eps,
                                      weight_decay, grad_scale, skip_nonfinite)


def _trainer(monkeypatch, inp, **kw):
    from fourier_neural_spectral_fno_b200 import train as T
    monkeypatch.setattr(T, "capi", _FakeSkipping((2, 2)))
    return T.Trainer((8, 6), (2, 2), 3, 4, inp["params"], PrecisionSchedule([(0, "f32")]),
                     hidden=5, n_layers=2, lr=1e-2, device="cpu", **kw)


def _batches(inp):
    a = torch.from_numpy(np.asarray(inp["a"], np.float32))
    good = torch.from_numpy(np.asarray(inp["target"], np.float32))
    bad = good.clone()
    bad[0, 0, 0, 0] = math.inf
    return a, good, bad


def _same(x, y):
    return all(torch.equal(getattr(x, k), getattr(y, k)) for k in ("master", "m", "v"))


def test_skipped_steps_leave_no_trace(monkeypatch):
    """[bad, bad, good, bad, good] gives the bits of [good, good]."""
    _, inp = _network()
    a, good, bad = _batches(inp)
    tr, ref = (_trainer(monkeypatch, inp, skip_nonfinite=True) for _ in range(2))
    for t in (bad, bad, good, bad, good):
        tr.step(a, t)
    for _ in range(2):
        ref.step(a, good)
    assert _same(tr, ref) and tr.step_count == 5
    assert tr.skipped_steps() == 3 and ref.skipped_steps() == 0


def test_skipped_steps_survive_a_checkpoint(monkeypatch):
    _, inp = _network()
    a, good, bad = _batches(inp)
    ref = _trainer(monkeypatch, inp, skip_nonfinite=True)
    for _ in range(3):
        ref.step(a, good)
    tr = _trainer(monkeypatch, inp, skip_nonfinite=True)
    for t in (bad, good, bad):
        tr.step(a, t)
    state = tr.state_dict()
    assert state["skipped"] == 2 and state["step"] == 3
    for kw in ({}, {"skip_nonfinite": True}):
        other = _trainer(monkeypatch, inp, **kw)
        if kw:
            other.step(a, bad)                  # a count of its own, which the load replaces
        other.load_state_dict(state)
        assert other.skipped_steps() == 2
        other.step(a, good)
        other.step(a, bad)
        other.step(a, good)
        assert _same(other, ref) and other.skipped_steps() == 3
    # a checkpoint from before the count
    other = _trainer(monkeypatch, inp, skip_nonfinite=True)
    other.load_state_dict({k: v for k, v in state.items() if k != "skipped"})
    assert other.skipped_steps() == 0


def test_the_count_holds_when_the_flag_is_taken_back(monkeypatch):
    _, inp = _network()
    a, good, bad = _batches(inp)
    ref = _trainer(monkeypatch, inp)
    for _ in range(3):
        ref.step(a, good)
    tr = _trainer(monkeypatch, inp, skip_nonfinite=True)
    tr.step(a, bad)
    tr.step(a, good)
    tr.skip_nonfinite = False
    tr.step(a, good)
    tr.skip_nonfinite = True
    tr.step(a, bad)
    tr.step(a, good)
    assert _same(tr, ref) and tr.skipped_steps() == 2


def test_adam_step_skipping_refuses():
    build.build()
    lib = capi.load()

    def call(**kw):
        a = dict(n=8, theta=256, m=256, v=256, grad=256, out=256, od=2, step=1, lr=1e-3, b1=0.9,
                 b2=0.999, eps=1e-8, wd=0.0, scale=1.0, norm=256, skipped=256)
        a.update(kw)
        return lib.fno_adam_step_skipping(*a.values(), None)

    for kw, word in [({"n": 0}, "n 0"), ({"theta": None}, "theta"), ({"grad": None}, "grad"),
                     ({"norm": None}, "norm"), ({"norm": 0x102}, "norm"), ({"step": 0}, "step 0"),
                     ({"eps": 0.0}, "eps"), ({"od": 5}, "out_dtype"), ({"b2": 1.0}, "betas"),
                     ({"scale": float("nan")}, "grad_scale"), ({"skipped": None}, "skipped is NULL"),
                     ({"skipped": 0x104}, "skipped is not 16-byte aligned")]:
        assert call(**kw) == capi.FNO_ERR_INVALID_ARG, kw
        assert word in capi.last_error(), kw


def test_binding_refuses_a_count_on_the_host(monkeypatch):
    build.build()
    t = [torch.zeros(8) for _ in range(4)]
    monkeypatch.setattr(capi, "_device_index", lambda t, name: 0)
    monkeypatch.setattr(capi, "_check_tensor", lambda t, name, *a: None if "state" not in name else
                        _refuse(t, name, *a))
    with pytest.raises(ValueError, match="skip_nonfinite.state is on cpu"):
        capi.fno_adam_step_clipped(*t, None, 1, 1e-3, torch.zeros(2), stream=0,
                                   skip_nonfinite=capi.SkippedSteps("cpu"))


_refuse = capi._check_tensor
