"""The network with layer norm and the clipped trainer on the CPU: the oracle's
gradients against differences, the library's argument checks, the parameter
layout and the trainer's calls (with a stand-in for the library)."""

import ctypes

import numpy as np
import pytest
import torch

import oracle as O
from fourier_neural_spectral_fno_b200 import build, capi, synth
from fourier_neural_spectral_fno_b200.train import ALIGN, ParamLayout, PrecisionSchedule
from test_train_host import _FakeLibrary


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


def _network(dtype="f32", grid=(8, 6), modes=(2, 2), width=4, batch=2, seed=3):
    wl = synth.Workload("tiny", "network", dtype, batch, grid, modes, width, in_ch=3, hidden=5,
                        n_layers=2, backward=True)
    inp = synth.make_network_inputs(wl)
    rng = np.random.default_rng(seed)
    inp["params"]["ln_g"] = [synth.quantize(1 + 0.3 * rng.standard_normal(width), dtype)
                             for _ in range(2)]
    inp["params"]["ln_b"] = [synth.quantize(0.3 * rng.standard_normal(width), dtype)
                             for _ in range(2)]
    return wl, inp


def test_oracle_network_gradients_by_differences():
    wl, inp = _network()
    a, p, t = inp["a"], inp["params"], inp["target"]

    def loss(params):
        return O.mse(O.forward(a, params, wl.modes, O.LAYER_NORM), t)[0]

    u, saves = O.forward(a, p, wl.modes, O.LAYER_NORM, save=True)
    grads = O.backward(a, p, saves, O.mse(u, t)[1], wl.modes, O.LAYER_NORM)
    assert not np.allclose(u, O.forward(a, p, wl.modes))     # the flag does something
    h = 1e-5
    for key, idx in (("ln_g", (0, 1)), ("ln_g", (1, 3)), ("ln_b", (0, 2)), ("ln_b", (1, 0)),
                     ("W", (0, 1, 2)), ("b", (1, 1))):
        vals = []
        for s in (h, -h):
            q = {**p, key: [x.copy() for x in p[key]]}
            q[key][idx[0]][idx[1:]] += s
            vals.append(loss(q))
        num = (vals[0] - vals[1]) / (2 * h)
        assert abs(num - grads[key][idx[0]][idx[1:]]) <= 1e-6 * max(1.0, abs(num)), (key, idx)
    q = {**p, "P": p["P"].copy()}
    q["P"][1, 2] += h
    up = loss(q)
    q["P"][1, 2] -= 2 * h
    assert abs((up - loss(q)) / (2 * h) - grads["P"][1, 2]) <= 1e-6


def test_flag_is_for_networks_alone_and_needs_its_parameters(lib):
    d = capi.block_desc(2, 4, 4, (16, 16), (4, 4), flags=capi.FNO_LAYER_NORM)
    assert lib.fno_workspace_size(ctypes.byref(d), capi.FNO_OP_BLOCK_FWD) == 0
    assert "flag" in capi.last_error()
    plain = capi.net_desc(2, (16, 16), (4, 4), 3, 8, hidden=16, n_layers=2)
    d = capi.net_desc(2, (16, 16), (4, 4), 3, 8, hidden=16, n_layers=2, flags=capi.FNO_LAYER_NORM)
    # the norm's input and statistics are saved too
    act, stat = 2 * 8 * 256 * 4, 2 * 256 * 4
    assert capi.fno_net_saves_size(d) == capi.fno_net_saves_size(plain) + 2 * (act + 2 * stat)

    def buf():
        return torch.zeros(1 << 14)

    params = {k: buf() for k in ("P", "p", "Q1", "q1", "Q2", "q2")}
    params.update({k: [buf(), buf()] for k in ("R", "W", "b", "ln_g", "ln_b")})
    for key in ("ln_g", "ln_b"):
        for bad, word in (([buf()], f"{key}.l. is NULL"),
                          ([buf(), buf()[1:]], f"{key}.l. is not 16-byte aligned")):
            with pytest.raises(capi.FnoError, match=word):
                capi.fno_forward(d, buf(), capi.make_params({**params, key: bad}), buf(), buf(),
                                 stream=0)
    for key, word in (("ln_g", "dln_g"), ("ln_b", "dln_b")):
        with pytest.raises(capi.FnoError, match=word):
            capi.fno_backward(d, buf(), capi.make_params(params), buf(), buf(),
                              capi.make_grads({**params, key: []}), stream=0)
    with pytest.raises(capi.FnoError, match="ln_g"):
        capi.fno_backward(d, buf(), capi.make_params({**params, "ln_g": []}), buf(), buf(),
                          capi.make_grads(params), stream=0)


def test_layout_with_layer_norm():
    lay = ParamLayout(3, 6, 9, 2, 3, 40, layer_norm=True)
    assert [k for k, *_ in lay.slots] == ["P", "p"] + ["R", "W", "b", "ln_g", "ln_b"] * 3 + \
        ["Q1", "q1", "Q2", "q2"]
    assert all(off % ALIGN == 0 for *_, off, _ in lay.slots)
    # a layer's group holds its norm too, and the groups tile the buffer
    at = {(k, l): off for k, l, _, off, _ in lay.slots}
    bk = lay.buckets()
    assert bk[2][0] <= at[("ln_b", 1)] < bk[2][1] and bk[2][0] <= at[("ln_g", 1)]
    edges = sorted(bk)
    assert edges[0][0] == 0 and edges[-1][1] == lay.total
    assert all(a[1] == b[0] for a, b in zip(edges, edges[1:]))


def test_layout_pack_with_and_without_norm_parameters():
    _, inp = _network()
    lay = ParamLayout(3, 4, 5, 1, 2, synth._num_kept((8, 6), (2, 2)), layer_norm=True)
    flat = torch.zeros(lay.total)
    lay.pack(inp["params"], flat)
    back = lay.unpack(flat)
    for key in ("ln_g", "ln_b"):
        for l in range(2):
            np.testing.assert_array_equal(back[key][l], np.float32(inp["params"][key][l]))
    without = {k: v for k, v in inp["params"].items() if not k.startswith("ln_")}
    lay.pack(without, flat)
    back = lay.unpack(flat)
    assert all((g == 1).all() for g in back["ln_g"]) and all((b == 0).all() for b in back["ln_b"])


class _FakeWithNorm(_FakeLibrary):
    """The stand-in with layer norm, the gradient norm and the clipped step."""

    def fno_forward(self, d, a, params, u, saves, ws=None):
        p = self._np(params)
        uu, sv = O.forward(a.float().numpy().astype(np.float64), p, self.modes, d["flags"], save=True)
        self.saved[saves.data_ptr()] = sv
        u.copy_(torch.from_numpy(uu))

    def fno_backward(self, d, a, params, saves, du, grads, ws=None):
        g = O.backward(a.float().numpy().astype(np.float64), self._np(params),
                       self.saved[saves.data_ptr()], du.float().numpy().astype(np.float64),
                       self.modes, d["flags"])
        for key, val in grads.items():
            for l, t in enumerate(val if isinstance(val, list) else [val]):
                src = g[key][l] if isinstance(val, list) else g[key]
                if key == "R":
                    src = np.stack([src.real, src.imag], -1)
                t.copy_(torch.from_numpy(np.asarray(src, np.float32)))

    @staticmethod
    def grad_list(grads):
        return grads

    @staticmethod
    def fno_grad_norm_workspace_size(grads):
        return 64

    def fno_grad_norm(self, grads, max_norm, norm, grad_scale=1.0, ws=None):
        self.calls.append(("norm", max_norm, grad_scale))
        norm.copy_(torch.tensor(O.grad_norm([g.numpy() for g in grads], max_norm, grad_scale)))

    def fno_adam_step_clipped(self, theta, m, v, grad, out, step, lr, norm, beta1, beta2, eps,
                              weight_decay, grad_scale, skip_nonfinite):
        self.calls.append(("clipped", step, skip_nonfinite))
        if skip_nonfinite and not np.isfinite(float(norm[0])):
            out.copy_(theta.to(out.dtype))
            return
        self.fno_adam_step(theta, m, v, grad, out, step, lr, beta1, beta2, eps, weight_decay,
                           grad_scale * float(norm[1]))


def _trainer(fake, monkeypatch, inp, **kw):
    from fourier_neural_spectral_fno_b200 import train as T
    monkeypatch.setattr(T, "capi", fake)
    return T.Trainer((8, 6), (2, 2), 3, 4, inp["params"], PrecisionSchedule([(0, "f32")]),
                     hidden=5, n_layers=2, lr=1e-2, device="cpu", **kw)


def test_trainer_with_norm_and_clipping_matches_the_oracle_loop(monkeypatch):
    """eps = 1 makes the update nearly linear in the gradient, so a wrong factor shows."""
    _, inp = _network()
    fake = _FakeWithNorm((2, 2))
    limit = 1e-2
    tr = _trainer(fake, monkeypatch, inp, flags=capi.FNO_LAYER_NORM, eps=1.0, max_grad_norm=limit)
    a = torch.from_numpy(np.asarray(inp["a"], np.float32))
    t = torch.from_numpy(np.asarray(inp["target"], np.float32))
    start = tr.master.clone()
    losses = [float(tr.step(a, t)) for _ in range(3)]
    ref, ref_losses = O.train(inp["a"], inp["target"], inp["params"], (2, 2), [(0, "f32")], 3, 1e-2,
                              eps=1.0, flags=O.LAYER_NORM, max_grad_norm=limit)
    np.testing.assert_allclose(losses, ref_losses, rtol=1e-6)
    got = tr.params()
    moved = float((tr.master - start).abs().max())
    for key in ("ln_g", "ln_b", "W", "b", "R"):
        for l in range(2):
            np.testing.assert_allclose(got[key][l], ref[key][l], rtol=1e-5, atol=1e-3 * moved)
    assert float(tr.grad_norm[1]) < 1.0                           # the limit was reached
    assert [c for c in fake.calls if c[0] == "norm"] == [("norm", limit, 1.0)] * 3
    assert [c[1:] for c in fake.calls if c[0] == "clipped"] == [(1, False), (2, False), (3, False)]


def test_trainer_without_clipping_makes_no_norm_call(monkeypatch):
    _, inp = _network()
    fake = _FakeWithNorm((2, 2))
    tr = _trainer(fake, monkeypatch, inp)
    a = torch.from_numpy(np.asarray(inp["a"], np.float32))
    t = torch.from_numpy(np.asarray(inp["target"], np.float32))
    tr.step(a, t)
    assert tr.grad_norm is None and not [c for c in fake.calls if c[0] in ("norm", "clipped")]


def test_trainer_skips_a_step_that_overflowed(monkeypatch):
    _, inp = _network()
    fake = _FakeWithNorm((2, 2))
    tr = _trainer(fake, monkeypatch, inp, skip_nonfinite=True)
    a = torch.from_numpy(np.asarray(inp["a"], np.float32))
    t = torch.from_numpy(np.asarray(inp["target"], np.float32))
    tr.step(a, t)
    before = [x.clone() for x in (tr.master, tr.m, tr.v)]
    bad = t.clone()
    bad[0, 0, 0, 0] = float("inf")
    tr.step(a, bad)
    assert not np.isfinite(float(tr.grad_norm[0]))
    assert all(torch.equal(x, y) for x, y in zip((tr.master, tr.m, tr.v), before))
    tr.step(a, t)
    assert not torch.equal(tr.master, before[0])
    assert [c[1] for c in fake.calls if c[0] == "norm"] == [float("inf")] * 3


def test_trainer_checkpoint_holds_the_clipping(monkeypatch):
    _, inp = _network()
    fake = _FakeWithNorm((2, 2))
    tr = _trainer(fake, monkeypatch, inp, flags=capi.FNO_LAYER_NORM, max_grad_norm=0.5,
                  skip_nonfinite=True)
    state = tr.state_dict()
    other = _trainer(fake, monkeypatch, inp, flags=capi.FNO_LAYER_NORM)
    other.load_state_dict(state)
    assert other.max_grad_norm == 0.5 and other.skip_nonfinite is True
    # a checkpoint from before clipping leaves the trainer's own setting
    old = {k: v for k, v in state.items() if k not in ("max_grad_norm", "skip_nonfinite")}
    third = _trainer(fake, monkeypatch, inp, flags=capi.FNO_LAYER_NORM, max_grad_norm=2.0)
    third.load_state_dict(old)
    assert third.max_grad_norm == 2.0 and third.skip_nonfinite is False
    # without layer norm the slots differ
    with pytest.raises(ValueError):
        _trainer(fake, monkeypatch, inp).load_state_dict(state)
    with pytest.raises(ValueError, match="max_grad_norm"):
        _trainer(fake, monkeypatch, inp, max_grad_norm=-1.0)
    with pytest.raises(ValueError, match="max_grad_norm"):
        _trainer(fake, monkeypatch, inp, max_grad_norm=float("nan"))
