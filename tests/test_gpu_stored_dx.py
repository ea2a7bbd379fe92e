"""The layer norm's gradient from 8 bits where neither the weights' nor the biases' is wanted, which
the C interface allows: the same dx, whatever the width and alignment."""
import pytest
import torch

from top_gradient_compression_gb300 import _lib, api

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", list(api.TYPES), ids=str)
@pytest.mark.parametrize("rows,dim", [(1, 16), (5, 128), (333, 1024), (1, 8192), (2000, 333),
                                      (3, 9001)])
def test_dx_alone(t, rows, dim):
    gen = torch.Generator(device=DEV).manual_seed(rows + dim)
    x, dy = (torch.randn(rows, dim, generator=gen, device=DEV).to(t) for _ in range(2))
    w = torch.randn(dim, generator=gen, device=DEV).to(t)
    kept = api.checkpoint8(x)
    _, mean, rstd = api.layer_norm(x)
    want, dw, db = api.layer_norm_backward(dy, kept, mean, rstd, w)
    size = api.layer_norm_backward_workspace_size(rows, dim)
    ws, dx = api.workspace(size, DEV), torch.full_like(x, 7.0)
    code = api.TYPES[t]
    args = (dy.data_ptr(), dim, code, kept.codes.data_ptr(), kept.codes.shape[-1],
            kept.exponents.data_ptr(), kept.exponents.shape[-1], w.data_ptr(), code,
            mean.data_ptr(), rstd.data_ptr(), rows, dim, dx.data_ptr(), dim)
    last = (0, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    backward = _lib.load().sparcml_layer_norm_backward8
    assert backward(*args, None, None, *last) == 0
    assert torch.equal(dx, want)
    for sums in ((dw, None), (None, db)):  # or one of the two
        got = [None if s is None else torch.full_like(s, 7.0) for s in sums]
        assert backward(*args, *(None if g is None else g.data_ptr() for g in got), *last) == 0
        assert torch.equal(dx, want)
        assert all(s is None or torch.equal(g, s) for g, s in zip(got, sums))
