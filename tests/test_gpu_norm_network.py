"""The network with layer norm and the clipped, norm-taking trainer on the GPU
against the oracle: a run of the operators together.

Tolerances (relative L2).  float32: 1e-5, the library's own bound.  bfloat16: a
stored value is off by at most 2^-8 of itself, and by less than 2^-9 in the root
mean square over a binade; between the input and u of two layers lie 7 stored arrays (input, lift,
and per layer the normalised input, pre-activation's store and output), and a
norm enlarges a relative error by |v| / std(v) <= 2 here: 7 2^-9 2 = 2.8e-2.
The backward runs through as many again: 6e-2 for the gradients.
"""

import numpy as np
import pytest

import oracle as O
from fno_testlib import (assert_close, dev, empty, grads_like, host, host_complex,
                         params_to_device, rel_l2)
from fourier_neural_spectral_fno_b200 import capi, synth

pytestmark = pytest.mark.gpu

U_TOL = {"f32": 1e-5, "bf16": 3e-2}
G_TOL = {"f32": 1e-5, "bf16": 6e-2}


def _network(grid, modes, dtype, batch=2, width=6, hidden=9, layers=2):
    wl = synth.Workload("tiny", "network", dtype, batch, tuple(grid), tuple(modes), width,
                        in_ch=1 + len(grid), hidden=hidden, n_layers=layers, backward=True)
    inp = synth.make_network_inputs(wl)
    p = inp["params"]
    rng = np.random.default_rng(31)
    p["R"] = [synth.quantize_complex(r * width * width / np.sqrt(width), dtype) for r in p["R"]]
    p["b"] = [synth.quantize(np.linspace(-0.3, 0.3, width), dtype) for _ in p["b"]]
    p["ln_g"] = [synth.quantize(1 + 0.3 * rng.standard_normal(width), dtype) for _ in p["b"]]
    p["ln_b"] = [synth.quantize(0.3 * rng.standard_normal(width), dtype) for _ in p["b"]]
    return wl, inp


CASES = [((16, 12), (4, 5), 6), ((15, 9), (5, 4), 7), ((6, 10, 12), (2, 3, 4), 6), ((100,), (20,), 6),
         ((64, 64), (10, 12), 32), ((128, 64), (8, 8), 64)]


@pytest.mark.parametrize("grid,modes,width", CASES, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_network_with_layer_norm(grid, modes, width, dtype):
    import torch
    wl, inp = _network(grid, modes, dtype, width=width)
    a, params, tgt = inp["a"], inp["params"], inp["target"]
    fl = capi.FNO_LAYER_NORM
    d = capi.net_desc(wl.batch, grid, modes, wl.in_ch, width, wl.hidden, 1, wl.n_layers, dtype, fl)
    pd = params_to_device(params, dtype)
    cp = capi.make_params(pd)
    saves = torch.empty(capi.fno_net_saves_size(d), dtype=torch.uint8, device="cuda")
    u = empty((wl.batch, 1) + grid, dtype)
    a_d = dev(a, dtype)
    capi.fno_forward(d, a_d, cp, u, saves)
    u_ref, sv = O.forward(a, params, modes, O.LAYER_NORM, save=True)
    assert_close(host(u), u_ref, U_TOL[dtype], "u")
    u2 = empty(u.shape, dtype)
    capi.fno_forward(d, a_d, cp, u2)              # nothing saved: the norm runs in place
    assert torch.equal(u, u2)
    loss = torch.empty(1, dtype=torch.float32, device="cuda")
    du = empty(u.shape, dtype)
    capi.fno_mse(u, dev(tgt, dtype), loss, du, dtype)
    gd = grads_like(params)
    ready = [torch.cuda.Event() for _ in range(wl.n_layers + 2)]
    capi.fno_backward(d, a_d, cp, saves, du, capi.make_grads(gd), ready=ready)
    g_ref = O.backward(a, params, sv, host(du), modes, O.LAYER_NORM)
    tol = G_TOL[dtype]
    for key in ("P", "p", "Q1", "q1", "Q2", "q2"):
        assert_close(host(gd[key]), g_ref[key], tol, key)
    for key in ("R", "W", "b", "ln_g", "ln_b"):
        for l in range(wl.n_layers):
            got = host_complex(gd[key][l]) if key == "R" else host(gd[key][l])
            assert_close(got, g_ref[key][l], tol, f"{key}[{l}]")


def test_training_step_replays_as_cuda_graph():
    """Forward, loss, backward, gradient norm and clipped Adam captured as one
    graph: replays give the bits of the same calls made one by one."""
    import torch
    grid, modes = (64, 64), (10, 12)
    wl, inp = _network(grid, modes, "bf16", width=64, hidden=32)
    d = capi.net_desc(wl.batch, grid, modes, wl.in_ch, 64, 32, 1, wl.n_layers, "bf16",
                      capi.FNO_LAYER_NORM)
    from fourier_neural_spectral_fno_b200.train import ParamLayout
    lay = ParamLayout(wl.in_ch, 64, 32, 1, wl.n_layers, capi.num_modes(grid, modes), layer_norm=True)

    def buffers():
        z = lambda: torch.zeros(lay.total, device="cuda")  # noqa: E731
        b = dict(theta=z(), m=z(), v=z(), grad=z(), norm=torch.empty(2, device="cuda"),
                 w=torch.empty(lay.total, dtype=torch.bfloat16, device="cuda"),
                 u=empty((wl.batch, 1) + grid, "bf16"), du=empty((wl.batch, 1) + grid, "bf16"),
                 loss=torch.zeros(1, device="cuda"),
                 saves=torch.empty(capi.fno_net_saves_size(d), dtype=torch.uint8, device="cuda"),
                 wf=torch.empty(capi.fno_net_workspace_size(d, capi.FNO_OP_NET_FWD),
                                dtype=torch.uint8, device="cuda"),
                 wb=torch.empty(capi.fno_net_workspace_size(d, capi.FNO_OP_NET_BWD),
                                dtype=torch.uint8, device="cuda"),
                 wn=torch.empty(capi.fno_grad_norm_workspace_size(1), dtype=torch.uint8,
                                device="cuda"))
        lay.pack(inp["params"], b["theta"])
        b["w"].copy_(b["theta"])
        b["gl"] = capi.grad_list([b["grad"]])
        return b

    a_d, t_d = dev(inp["a"], "bf16"), dev(inp["target"], "bf16")

    def step(b):
        cp, cg = capi.make_params(lay.views(b["w"])), capi.make_grads(lay.views(b["grad"]))
        capi.fno_forward(d, a_d, cp, b["u"], b["saves"], ws=b["wf"])
        capi.fno_mse(b["u"], t_d, b["loss"], b["du"], dtype="bf16")
        capi.fno_backward(d, a_d, cp, b["saves"], b["du"], cg, ws=b["wb"])
        capi.fno_grad_norm(b["gl"], 1e-2, b["norm"], ws=b["wn"])
        capi.fno_adam_step_clipped(b["theta"], b["m"], b["v"], b["grad"], b["w"], 1, 1e-3, b["norm"],
                                   skip_nonfinite=True)

    plain, graphed = buffers(), buffers()
    for _ in range(3):
        step(plain)
    step(graphed)                       # the first of its three steps, outside the graph
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        step(graphed)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert float(plain["norm"][1]) < 1.0
    for key in ("theta", "m", "v", "grad", "norm", "w"):
        assert torch.equal(plain[key], graphed[key]), key


@pytest.mark.parametrize("grid,modes,width", [((16, 12), (4, 5), 6), ((64, 64), (10, 12), 32)], ids=str)
def test_trainer_with_norm_and_clipping_matches_oracle(grid, modes, width):
    """Three clipped steps, eps = 1 (a step nearly linear in the gradient, so that a
    wrong factor shows).  The weights move by about lr g: the gradients' own 1e-5
    bound and one of 2^-20 for the master copy's roundings, over three steps."""
    import torch
    from fourier_neural_spectral_fno_b200.train import PrecisionSchedule, Trainer
    wl, inp = _network(grid, modes, "f32", width=width)
    steps, lr, limit = 3, 0.5, 1e-2
    tr = Trainer(grid, modes, wl.in_ch, width, inp["params"], PrecisionSchedule([(0, "f32")]),
                 hidden=wl.hidden, n_layers=wl.n_layers, lr=lr, eps=1.0, flags=capi.FNO_LAYER_NORM,
                 max_grad_norm=limit)
    start = tr.params()
    a = torch.from_numpy(np.asarray(inp["a"], np.float32)).cuda()
    t = torch.from_numpy(np.asarray(inp["target"], np.float32)).cuda()
    losses = [float(tr.step(a, t).item()) for _ in range(steps)]
    ref, ref_losses = O.train(inp["a"], inp["target"], inp["params"], modes, [(0, "f32")], steps, lr,
                              eps=1.0, flags=O.LAYER_NORM, max_grad_norm=limit)
    np.testing.assert_allclose(losses, ref_losses, rtol=1e-4)
    assert float(tr.grad_norm[1]) < 1.0
    got = tr.params()
    for key in ("P", "Q1", "ln_g", "ln_b", "W", "R"):
        for x, y, s in zip(*[np.asarray(q[key])[None] if key in ("P", "Q1") else q[key]
                             for q in (got, ref, start)]):
            moved = np.linalg.norm(np.ravel(y - s))
            off = np.linalg.norm(np.ravel(x - y))
            assert off <= 1e-3 * moved + 2.0 ** -22 * np.linalg.norm(np.ravel(y)), key


def test_trainer_half_precision_overflow_is_skipped():
    """A target beyond float16's range makes the loss and gradients overflow: with
    skip_nonfinite the weights stay, and the next good step moves them."""
    import torch
    from fourier_neural_spectral_fno_b200.train import PrecisionSchedule, Trainer
    wl, inp = _network((16, 12), (4, 5), "f16")
    tr = Trainer((16, 12), (4, 5), wl.in_ch, 6, inp["params"], PrecisionSchedule([(0, "f16")]),
                 hidden=wl.hidden, n_layers=wl.n_layers, flags=capi.FNO_LAYER_NORM,
                 max_grad_norm=1.0, skip_nonfinite=True)
    a = torch.from_numpy(np.asarray(inp["a"], np.float32)).cuda()
    t = torch.from_numpy(np.asarray(inp["target"], np.float32)).cuda()
    tr.step(a, t)
    before = [x.clone() for x in (tr.master, tr.m, tr.v, tr.weights)]
    tr.step(a, t * 1e6)
    assert not np.isfinite(float(tr.grad_norm[0]))
    assert all(torch.equal(x, y) for x, y in zip((tr.master, tr.m, tr.v, tr.weights), before))
    tr.step(a, t)
    assert np.isfinite(float(tr.grad_norm[0])) and not torch.equal(tr.master, before[0])
    assert rel_l2(host(tr.weights), host(tr.master)) < 2.0 ** -11
