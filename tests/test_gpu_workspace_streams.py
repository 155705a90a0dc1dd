"""The workspaces that the binding makes for calls on a stream other than the current one."""

import pytest

from fourier_neural_spectral_fno_b200 import capi

pytestmark = pytest.mark.gpu


def _pending(nbytes):
    """The address of memory that was freed with work on it still queued on the current
    stream: PyTorch hands it out again to that stream alone, ordered behind the work."""
    import torch
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    t = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(1_000_000)
    t.fill_(7)
    return t.data_ptr()


def _layer_norm(stream):
    import torch
    d = capi.layer_norm_desc(40, 64, 4096)
    x, s = torch.ones(40, 64, 4096, device="cuda"), torch.ones(40, 4096, device="cuda")
    g = torch.ones(64, device="cuda")
    dx, dg, db = torch.empty_like(x), torch.empty_like(g), torch.empty_like(g)
    return capi.fno_layer_norm_workspace_size(d), lambda: capi.fno_layer_norm_bwd(
        d, x, g, s, s, x, dx, dg, db, stream=stream)


def _norm(stream):
    import torch
    gl, norm = capi.grad_list([torch.ones(100000, device="cuda")]), torch.empty(2, device="cuda")
    return capi.fno_grad_norm_workspace_size(gl), lambda: capi.fno_grad_norm(gl, 1.0, norm,
                                                                             stream=stream)


def _clip(stream):
    import torch
    gl, norm = capi.grad_list([torch.ones(100000, device="cuda")]), torch.empty(2, device="cuda")
    return capi.fno_grad_norm_workspace_size(gl), lambda: capi.fno_clip_grads(gl, 1.0, norm,
                                                                              stream=stream)


def _block(stream):
    import torch
    d = capi.block_desc(2, 8, 8, (16, 16), (4, 4))
    x = torch.ones(2, 8, 16, 16, device="cuda")
    r, w = torch.ones(8, 8, capi.num_modes((16, 16), (4, 4)), 2, device="cuda"), torch.ones(8, 8, device="cuda")
    b, y = torch.ones(8, device="cuda"), torch.empty_like(x)
    return capi.fno_workspace_size(d, capi.FNO_OP_BLOCK_FWD), lambda: capi.fno_block_fwd(
        d, x, r, w, b, y, stream=stream)


@pytest.mark.parametrize("make", [_layer_norm, _norm, _clip, _block])
@pytest.mark.parametrize("kind", ["stream", "handle"])
def test_workspace_is_not_one_that_the_current_stream_still_uses(make, kind, monkeypatch):
    """Nor is it handed back to the current stream when the call returns."""
    import torch
    side = torch.cuda.Stream()
    size, call = make(side if kind == "stream" else side.cuda_stream)
    made = []
    plain = capi._workspace

    def watched(*args):
        made.append(plain(*args)[0].data_ptr())     # freed here, as when the call returns
        return plain(*args)

    monkeypatch.setattr(capi, "_workspace", watched)
    busy = _pending(size)
    call()
    again = torch.empty(size, dtype=torch.uint8, device="cuda").data_ptr()
    torch.cuda.synchronize()
    assert len(made) == 1
    for at in (busy, again):
        assert not (at <= made[0] < at + size or made[0] <= at < made[0] + size)
