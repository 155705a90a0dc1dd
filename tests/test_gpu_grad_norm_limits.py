"""The gradient norm and its factor at the ends of their range."""

import numpy as np
import pytest

import oracle as O
from fourier_neural_spectral_fno_b200 import capi

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
LISTS = {"one-cta": [300, 5], "two-launches": [40000, 9, 70001], "tables": [40] * 1030}


def _grads(name, value):
    import torch
    return [torch.full((n,), value, device="cuda") for n in LISTS[name]]


@pytest.mark.parametrize("name", list(LISTS))
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan], ids=str)
@pytest.mark.parametrize("max_norm", [np.inf, 1.0], ids=str)
def test_factor_of_a_norm_that_is_not_finite(name, bad, max_norm):
    """Infinity: 1 where the limit is infinity, else 0; a NaN: NaN.  Without a limit the
    gradients stay as they are."""
    import torch
    g = _grads(name, 1.0)
    g[-1][3] = bad
    before = [t.clone() for t in g]
    want = O.grad_norm([np.array([bad, 1.0])], max_norm)
    factor = np.nan if np.isnan(bad) else 1.0 if max_norm == np.inf else 0.0
    norm = torch.zeros(2, device="cuda")
    capi.fno_grad_norm(g, max_norm, norm)
    np.testing.assert_array_equal(norm.cpu().numpy(), [abs(bad), factor])
    np.testing.assert_array_equal(want, [abs(bad), factor])
    capi.fno_clip_grads(g, max_norm, norm)
    np.testing.assert_array_equal(norm.cpu().numpy(), [abs(bad), factor])
    if max_norm == np.inf and not np.isnan(bad):
        assert all(torch.equal(a, b) for a, b in zip(g, before))


@pytest.mark.parametrize("name", list(LISTS))
def test_norm_beyond_float32(name):
    """Values of 2^127: the norm reads as infinity, the factor is the limit over the norm
    itself (each square exact, the sum's and the root's float64 roundings below u: one
    rounding to float32), and the clipped values have the limit as their norm."""
    import torch
    g = _grads(name, 2.0 ** 127)
    total = sum(LISTS[name])
    limit = 2.0 ** 10
    norm = torch.zeros(2, device="cuda")
    capi.fno_clip_grads(g, limit, norm)
    factor = limit / (2.0 ** 127 * total ** 0.5)
    got = norm.double().cpu().numpy()
    assert got[0] == np.inf and abs(got[1] - factor) <= 2 * U * factor
    each = limit / total ** 0.5
    assert all(bool(((t.double() - each).abs() <= 4 * U * each).all()) for t in g)
    capi.fno_grad_norm(g, np.inf, norm)
    np.testing.assert_allclose(norm.double().cpu().numpy(), [limit, 1.0], rtol=6 * U)
