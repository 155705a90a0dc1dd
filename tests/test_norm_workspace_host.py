"""The layer norm backward's workspace on the CPU: it follows the points."""

import pytest

from fourier_neural_spectral_fno_b200 import build, capi


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


def _ws(outer, channels, inner, dtype):
    return capi.fno_layer_norm_workspace_size(capi.layer_norm_desc(outer, channels, inner, dtype))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_layer_norm_workspace_follows_the_points(lib, dtype):
    """8 bytes per channel and partial row: as many rows as the points can fill, 592 at
    most, never fewer for a larger batch or a larger grid."""
    for c in (1, 8, 33, 64, 256, 257, 1001, 8192, 8191, 33000):
        for inner in (1, 7, 32, 257, 4096):
            sizes = [_ws(outer, c, inner, dtype) for outer in (1, 2, 3, 8, 31, 100, 700, 20000, 10**6)
                     if outer * c * inner <= 1 << 40]     # more elements are refused
            assert sizes == sorted(sizes)
            assert 8 * c <= sizes[0] <= 592 * 8 * c + 255
            assert sizes[-1] <= 592 * 8 * c + 255
        for outer in (1, 5):
            sizes = [_ws(outer, c, inner, dtype) for inner in (2, 3, 31, 32, 33, 1000, 10**5, 10**7)
                     if outer * c * inner <= 1 << 40]
            assert sizes == sorted(sizes)
    # one row, or one point, of very many channels: no gigabytes
    assert _ws(1, 1 << 20, 1, dtype) == 8 << 20
    assert _ws(1, 1 << 20, 2, dtype) == 8 << 20
    assert _ws(1, 8192, 1, dtype) == 8 * 8192
    assert _ws(40, 8192, 1, dtype) <= 40 * 8 * 8192
