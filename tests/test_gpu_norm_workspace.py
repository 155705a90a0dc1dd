"""The layer norm backward in a workspace of exactly the size asked for: it is enough, and
what lies around it stays as it was."""

import pytest

from fno_testlib import torch_dtype
from fourier_neural_spectral_fno_b200 import capi
from test_gpu_norm_clip import LARGE, SHAPES

pytestmark = pytest.mark.gpu

# few points a CTA, where the partial rows are as many as the points allow
FEW = [(1, 8192, 1), (1, 8191, 1), (7, 4096, 1), (64, 1001, 1), (65, 4099, 1), (600, 8192, 1),
       (8, 7, 1), (300, 513, 1), (1, 256, 31), (19, 129, 32), (600, 32, 8), (31, 9, 257),
       (600, 96, 256), (1, 1 << 20, 1), (17, 33000, 1), (1, 300, 1025)]


@pytest.mark.parametrize("shape", FEW + SHAPES + LARGE, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_layer_norm_backward_keeps_to_its_workspace(shape, dtype):
    import torch
    outer, C, inner = shape
    g = torch.Generator(device="cuda").manual_seed(61)
    dt = torch_dtype(dtype)
    x = torch.randn(shape, generator=g, device="cuda").to(dt)
    dy = torch.randint(-3, 4, shape, generator=g, device="cuda")
    d = capi.layer_norm_desc(outer, C, inner, dtype)
    n = capi.fno_layer_norm_workspace_size(d)
    buf = torch.full((n + 8192,), 0x5a, dtype=torch.uint8, device="cuda")
    mean, rstd = torch.zeros(outer, inner, device="cuda"), torch.ones(outer, inner, device="cuda")
    dx = torch.empty_like(x)
    dg, db = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    capi.fno_layer_norm_bwd(d, x, None, mean, rstd, dy.to(dt), dx, dg, db, ws=buf[4096:4096 + n])
    assert bool((buf[:4096] == 0x5a).all()) and bool((buf[4096 + n:] == 0x5a).all())
    assert torch.equal(db.long(), dy.sum((0, 2)))          # whole numbers: exact in any order
