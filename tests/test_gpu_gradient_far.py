"""The operators that make a gradient on operands whose rows are 2^31 elements apart, against the same
ones with their rows together."""
import pytest
import torch

from top_gradient_compression_gb300 import api

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

FAR = 1 << 31


def normal(seed, *shape, dtype=torch.bfloat16):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=gen, device=DEV).to(dtype)


def apart(x):
    """x with its first axis 2^31 elements a step, in memory of its own."""
    room = torch.empty(FAR * (x.shape[0] - 1) + x[0].numel(), dtype=x.dtype, device=DEV)
    return room.as_strided(x.shape, (FAR, *x.stride()[1:])).copy_(x)


def same(a, b):
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dim", [520, 523, 8200])
def test_rows(dim):
    x, dy, w = normal(1, 3, dim), normal(2, 3, dim), normal(3, dim)
    _, mean, rstd = api.layer_norm(x, w)
    kept = api.checkpoint8(x)
    got = api.checkpoint8(apart(x))
    same((got.codes, got.exponents), (kept.codes, kept.exponents))
    same((api.restore8(kept, out=apart(x)),), (api.restore8(kept),))
    want = api.layer_norm_backward(dy, kept, mean, rstd, w)
    out = apart(dy)
    same(api.layer_norm_backward(out, kept, mean, rstd, w, dx=out), want)


@pytest.mark.parametrize("k", [72, 75])
def test_experts(k):
    x, w, dy = normal(1, 3, k), normal(2, 2, 40, k), normal(3, 3, 40)
    off = torch.tensor([0, 1, 3], dtype=torch.int32, device=DEV)
    y, dx = torch.zeros(3, 40, dtype=x.dtype, device=DEV), torch.zeros_like(x)
    same((api.expert_linear(apart(x), apart(w), off, out=apart(y)),),
         (api.expert_linear(x, w, off),))
    want = api.expert_linear_backward(dy, x, w, off)
    same(api.expert_linear_backward(apart(dy), x, w, off, dx=apart(dx),
                                    dweight=apart(torch.zeros(2, 40, k, device=DEV))), want)


@pytest.mark.parametrize("t, dim", [(torch.bfloat16, 128), (torch.float16, 37)])
def test_heads(t, dim):
    q, k = normal(1, 3, 4, dim, dtype=t), normal(2, 3, 2, dim, dtype=t)
    g, h = normal(3, 3, 4, dim, dtype=t), normal(4, 3, 2, dim, dtype=t)
    at = torch.tensor([5, 0, 1 << 40], device=DEV)
    f = normal(5, dim // 2, dtype=torch.float32)
    out = apart(q)
    same(api.head_norm_rotary(out, k, at, f, q_out=out), api.head_norm_rotary(q, k, at, f))
    out = apart(g)
    same(api.head_norm_rotary_backward(out, h, apart(q), k, at, f, dq_out=out),
         api.head_norm_rotary_backward(g, h, q, k, at, f))
