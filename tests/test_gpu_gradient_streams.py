"""The operators that make a gradient on a stream that the caller names: what a call allocates for
itself stays its own until that stream has used it."""
import pytest
import torch

from top_gradient_compression_gb300 import api

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu


def normal(seed, *shape, dtype=torch.bfloat16):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=gen, device=DEV).to(dtype)


def stored_case():
    x, dy, w = normal(1, 64, 520), normal(2, 64, 520), normal(3, 520)
    _, mean, rstd = api.layer_norm(x, w)

    def call(s):
        c = api.checkpoint8(x, stream=s)
        return (c.codes, c.exponents, api.restore8(c, stream=s),
                *api.layer_norm_backward(dy, c, mean, rstd, w, stream=s))
    return api.layer_norm_backward_workspace_size(64, 520), call


def expert_case(k, stored):
    x, w, dy = normal(1, 300, k), normal(2, 3, 264, k), normal(3, 300, 264)
    off = torch.tensor([0, 100, 100, 300], dtype=torch.int32, device=DEV)
    kept = api.checkpoint8(x) if stored else x
    return (api.expert_linear_workspace_size(300, 3, 264, k),
            lambda s: (api.expert_linear(x, w, off, stream=s),
                       *api.expert_linear_backward(dy, kept, w, off, stream=s)))


def head_case():
    both, g = normal(1, 200, 7, 64), normal(2, 200, 6, 64)
    q, k = both[:, :4], both[:, 4:6]
    at = torch.arange(200, dtype=torch.int32, device=DEV)
    f = normal(3, 32, dtype=torch.float32)
    return (api.head_norm_rotary_backward_workspace_size(200, 4, 2, 64),
            lambda s: (*api.head_norm_rotary(q, k, at, f, stream=s),
                       *api.head_norm_rotary_backward(g[:, :4], g[:, 4:], q, k, at, f, stream=s)))


@pytest.mark.parametrize("case", [stored_case, lambda: expert_case(136, False),
                                  lambda: expert_case(136, True), lambda: expert_case(133, False),
                                  head_case],
                         ids=["stored", "experts", "experts from 8 bits", "odd experts", "heads"])
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
    assert all(bool((j == 255).all()) for j in junk)
    for p, q in zip(want, got):
        assert torch.equal(p, q)


def test_graphs_that_share_a_workspace():
    """Replayed one after the other, in any order and with eager calls between them."""
    x, w, dy = normal(1, 5000, 72), normal(2, 2, 264, 72), normal(3, 5000, 264)
    off = [torch.tensor(o, dtype=torch.int32, device=DEV) for o in ([0, 4000, 5000], [0, 7, 4900])]
    ws = api.workspace(api.expert_linear_workspace_size(5000, 2, 264, 72), DEV)
    out = [torch.zeros(5000, 264, dtype=torch.bfloat16, device=DEV) for _ in off]

    def call(i):
        dx = torch.zeros_like(x)
        y = api.expert_linear(x, w, off[i], out=out[i], ws=ws)
        return (y, *api.expert_linear_backward(dy, x, w, off[i], dx=dx, ws=ws))
    want = [[t.clone() for t in call(i)] for i in range(2)]
    graphs, got = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(call(i))
        graphs.append(graph)
    for order in ((0, 1), (1, 0), (0, 0)):
        for t in got[0] + got[1]:
            t.zero_()
        for i in order:
            graphs[i].replay()
            call(1 - i)
        torch.cuda.synchronize()
        for i in set(order):
            assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))
    assert api.get_status(ws) == 0
