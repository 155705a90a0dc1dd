"""Skipped Adam steps on the GPU: the count on the device and the bias correction of the
steps that are taken."""

import numpy as np
import pytest

import oracle as O
from fno_testlib import torch_dtype
from fourier_neural_spectral_fno_b200 import capi
from test_gpu_norm_network import _network

pytestmark = pytest.mark.gpu

BETAS = (0.9, 0.999)


def _state(n, seed=5):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    theta = torch.randn(n, generator=g, device="cuda")
    return [theta, torch.zeros_like(theta), torch.zeros_like(theta)]


@pytest.mark.parametrize("n", [1, 4099, (1 << 20) + 3])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("bad", [np.nan, np.inf], ids=str)
def test_adam_skipped_steps_leave_no_trace(n, dtype, bad):
    """Bad steps among good ones against the good ones alone.  m and v do not depend on t:
    the same bits.  theta: 1 / (1 - beta^t) comes from the device's pow, off by 2 units of
    2^-52 of beta^t, which 1 - beta^t enlarges by at most 1000: one rounding to float32
    more or less, u = 2^-24 in m_hat and half of it in v_hat's root, so 4 u of each of the
    three steps lr m_hat / (v_hat^1/2 + eps) <= 10 lr, and theta's own roundings."""
    import torch
    steps = ["good", "bad", "bad", "good", "bad", "good"]
    a, b = _state(n), _state(n)
    lr = 1e-2
    skips = capi.SkippedSteps("cuda")
    norm = torch.empty(2, device="cuda")
    outs = [torch.empty(n, dtype=torch_dtype(dtype), device="cuda") for _ in range(2)]
    t, host = 0, [x.double().cpu().numpy() for x in a]
    for k, kind in enumerate(steps):
        g = torch.randn(n, generator=torch.Generator(device="cuda").manual_seed(70 + k), device="cuda")
        if kind == "bad":
            g[n // 2] = bad
        capi.fno_grad_norm([g], 0.7 * n ** 0.5, norm)
        capi.fno_adam_step_clipped(*a, g, outs[0], k + 1, lr, norm, *BETAS, skip_nonfinite=skips)
        if kind == "good":
            t += 1
            capi.fno_adam_step_clipped(*b, g, outs[1], t, lr, norm, *BETAS)
            host = list(O.adam_update(*host, g.double().cpu().numpy() * float(norm[1]), t, lr, *BETAS,
                                      1e-8, 0.0))
        else:
            assert torch.equal(outs[0], a[0].to(outs[0].dtype))
    assert skips.count() == 3
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    u = 2.0 ** -24
    assert bool(((a[0] - b[0]).abs() <= 3 * (4 * u * 10 * lr) + 6 * u * b[0].abs()).all())
    np.testing.assert_allclose(a[0].cpu().numpy(), host[0], rtol=2.0 ** -20, atol=3 * 1e-5 * lr)


def test_adam_without_a_skip_gives_the_same_bits():
    import torch
    n = 70001
    a, b = _state(n), _state(n)
    skips, norm = capi.SkippedSteps("cuda"), torch.empty(2, device="cuda")
    for k in range(4):
        g = torch.randn(n, generator=torch.Generator(device="cuda").manual_seed(80 + k), device="cuda")
        capi.fno_grad_norm([g], 1.0, norm)
        capi.fno_adam_step_clipped(*a, g, None, k + 1, 1e-3, norm, skip_nonfinite=skips)
        capi.fno_adam_step_clipped(*b, g, None, k + 1, 1e-3, norm)
    assert skips.count() == 0 and all(torch.equal(x, y) for x, y in zip(a, b))


def test_adam_skipping_in_a_graph_and_on_a_stream():
    """A captured norm and step, replayed on good and bad gradients: the count goes on
    from replay to replay, and a bad one changes nothing."""
    import torch
    n = 4099
    s = _state(n)
    skips, norm = capi.SkippedSteps("cuda"), torch.empty(2, device="cuda")
    good = torch.randn(n, device="cuda")
    g = good.clone()
    gl = capi.grad_list([g])
    ws = torch.empty(capi.fno_grad_norm_workspace_size(gl), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        capi.fno_grad_norm(gl, 1.0, norm, ws=ws, stream=stream)
        capi.fno_adam_step_clipped(*s, g, None, 9, 1e-3, norm, skip_nonfinite=skips, stream=stream)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    assert skips.count() == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for k in range(1, 4):
        before = [x.clone() for x in s]
        g[7] = float("inf")
        graph.replay()
        torch.cuda.synchronize()
        assert skips.count() == 2 * k - 1 and all(torch.equal(x, y) for x, y in zip(s, before))
        step(side)
        torch.cuda.synchronize()
        assert skips.count() == 2 * k and all(torch.equal(x, y) for x, y in zip(s, before))
        g.copy_(good)
        graph.replay()
        torch.cuda.synchronize()
        assert skips.count() == 2 * k and not torch.equal(s[0], before[0])


@pytest.mark.parametrize("clip", [None, 1.0], ids=str)
def test_trainer_skipped_steps_leave_no_trace(clip):
    """A float16 trainer whose first steps overflow takes its first real step as if they
    had not been: the same bits as a trainer without them (t = 1 for both: beta^1 is
    exact)."""
    import torch
    from fourier_neural_spectral_fno_b200.train import PrecisionSchedule, Trainer
    wl, inp = _network((16, 12), (4, 5), "f16")

    def trainer():
        return Trainer((16, 12), (4, 5), wl.in_ch, 6, inp["params"], PrecisionSchedule([(0, "f16")]),
                       hidden=wl.hidden, n_layers=wl.n_layers, flags=capi.FNO_LAYER_NORM,
                       max_grad_norm=clip, skip_nonfinite=True)

    a = torch.from_numpy(np.asarray(inp["a"], np.float32)).cuda()
    t = torch.from_numpy(np.asarray(inp["target"], np.float32)).cuda()
    tr, ref = trainer(), trainer()
    for _ in range(9):
        tr.step(a, t * 1e6)
    assert not np.isfinite(float(tr.grad_norm[0])) and tr.skipped_steps() == 9
    tr.step(a, t)
    ref.step(a, t)
    assert tr.skipped_steps() == 9 and ref.skipped_steps() == 0
    for key in ("master", "m", "v", "weights"):
        assert torch.equal(getattr(tr, key), getattr(ref, key)), key
