"""The layer norm backward's sums over all points, on data that adds up exactly.

With mean and xh small whole numbers, rstd = 1 and dy in 1 .. 4 every product and
every partial sum of dgamma = sum dy xh and dbeta = sum dy is a whole number below
2^24 (at most 12 a point, at most 1.3 million points): exact in float32 in any order.
dbeta then shows one point lost or taken twice, and dgamma a dy that met another
point's x.
"""

import pytest

from fno_testlib import torch_dtype
from fourier_neural_spectral_fno_b200 import capi
from test_gpu_norm_clip import LARGE, SHAPES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", SHAPES + LARGE, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_layer_norm_parameter_gradients_take_every_point_once(shape, dtype):
    import torch
    outer, C, inner = shape
    assert 12 * outer * inner < 1 << 24
    g = torch.Generator(device="cuda").manual_seed(47)
    ints = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g, device="cuda")  # noqa: E731
    xh, mean, dy = ints(-3, 3, *shape), ints(-4, 4, outer, inner), ints(1, 4, *shape)
    dt = torch_dtype(dtype)
    d = capi.layer_norm_desc(outer, C, inner, dtype)
    x = (xh + mean[:, None]).to(dt)
    dx = torch.empty_like(x)
    dg, db = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    ones = torch.ones(outer, inner, device="cuda")
    capi.fno_layer_norm_bwd(d, x, None, mean.float(), ones, dy.to(dt), dx, dg, db)
    assert torch.equal(dg.long(), (dy * xh).sum((0, 2)))
    assert torch.equal(db.long(), dy.sum((0, 2)))
