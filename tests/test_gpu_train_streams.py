"""The training-step operators on a stream that the caller names: what a call allocates for
itself stays its own until that stream has used it."""
import pytest
import torch

from top_gradient_compression_gb300 import api

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu


def norm_case():
    gen = torch.Generator(device=DEV).manual_seed(3)
    x, dy = (torch.randn(64, 512, generator=gen, device=DEV) for _ in range(2))
    w = torch.randn(512, generator=gen, device=DEV)
    _, mean, rstd = api.layer_norm(x, w)
    return (api.layer_norm_backward_workspace_size(64, 512),
            lambda s: (*api.layer_norm(x, w, stream=s),
                       *api.layer_norm_backward(dy, x, mean, rstd, w, stream=s)))


def orthogonal_case():
    gen = torch.Generator(device=DEV).manual_seed(4)
    g = torch.randn(2, 96, 200, generator=gen, device=DEV)
    return (api.orthogonalize_workspace_size(2, 96, 200),
            lambda s: (api.orthogonalize(g, stream=s),))


def step_case():
    gen = torch.Generator(device=DEV).manual_seed(5)
    g, w, m = (torch.randn(96, 200, generator=gen, device=DEV) for _ in range(3))
    # the copies are ready before the busy stream gets to them
    sets = [(w.clone(), m.clone()) for _ in range(2)]
    return (api.orthogonalize_workspace_size(1, 96, 200),
            lambda s: api.muon_step(sets[s is not None][0], g, sets[s is not None][1], 0.1,
                                    stream=s))


@pytest.mark.parametrize("case", [norm_case, orthogonal_case, step_case])
def test_memory_of_a_call_on_another_stream(case):
    size, call = case()
    want = call(None)
    big = torch.ones(64 << 20, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(100):  # the call below begins long after it has returned
            big.mul_(1.0)
    got = call(side)
    # on the current stream meanwhile: memory of the workspace's size, filled at once
    junk = [torch.full((size,), 255, dtype=torch.uint8, device=DEV) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(int(j[0]) == 255 and int(j[-1]) == 255 and bool((j == 255).all()) for j in junk)
    for p, q in zip(want, got):
        assert torch.equal(p, q)
