"""The example that runs the operators that make a gradient together, with the sparse exchange and
the weight steps."""
import os
import runpy

import pytest
import torch

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "expert_step.py")
SIZES = [dict(), dict(dim=77, q=3, kv=1, head=22, out=33, experts=4, tokens=150),
         dict(dim=128, q=4, kv=4, head=32, out=264, experts=1, tokens=64)]


def model(b, p, x):
    """The block in 64 bits, for autograd."""
    mean = x.mean(1, keepdim=True)
    h = (x - mean) / (x.var(1, unbiased=False, keepdim=True) + 1e-5).sqrt()
    h = h * p["weight"] + p["bias"]
    qkv = (h @ p["project"].t()).view(b.tokens, -1, b.head)

    def turned(v, w):
        v = v / (v.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        angle = b.positions.double()[:, None, None] * b.freqs.double()
        u0, u1 = v.chunk(2, -1)
        return torch.cat([u0 * angle.cos() - u1 * angle.sin(),
                          u0 * angle.sin() + u1 * angle.cos()], -1)
    q = turned(qkv[:, :b.q], p["q_weight"]).view(b.tokens, b.kv, -1, b.head).permute(1, 2, 0, 3)
    k = turned(qkv[:, b.q:b.q + b.kv], p["k_weight"]).transpose(0, 1)[:, None]
    v = qkv[:, b.q + b.kv:].transpose(0, 1)[:, None]
    score = q @ k.mT / b.head ** 0.5
    later = torch.ones_like(score, dtype=torch.bool).triu(1)
    o = (score.masked_fill(later, float("-inf")).softmax(-1) @ v).permute(2, 0, 1, 3)
    o = o.reshape(b.tokens, -1)
    at = b.offsets.tolist()
    runs = [o[i:j] @ p["experts"][e].t() for e, (i, j) in enumerate(zip(at, at[1:]))]
    return torch.cat(runs + [o.new_zeros(b.tokens - at[-1], b.out)])


@pytest.mark.parametrize("sizes", SIZES)
def test_gradients(sizes):
    """Every parameter's gradient and x's against autograd in 64 bits. What is kept in 8 bits is off
    by up to 1 / 63.5 / sqrt(12) of its group's largest, 1.3 % of a normal's root mean square; eight
    roundings to bf16 on the way of the gradient are 2^-9 each, 0.2 %; 5 % allows for both to add up
    and for the softmax."""
    b = runpy.run_path(PATH)["Block"](**sizes)
    x = b.normal(b.tokens, b.dim)
    dy = b.normal(b.tokens, b.out).to(torch.bfloat16)
    flat = torch.full((int(b.begin[-1]),), 7.0, device=DEV)
    y, kept = b.forward(x)
    dx = b.backward(dy, kept, flat)
    p = {k: v.double().requires_grad_() for k, v in b.params.items()}
    xd = x.double().requires_grad_()
    want = model(b, p, xd)
    (want * dy.double()).sum().backward()

    def off(a, c):
        return float((a.double() - c).norm() / c.norm())
    assert off(y, want.detach()) < 0.02  # bf16 alone
    assert off(dx, xd.grad) < 0.05
    for name, g in b.views(flat).items():
        assert off(g, p[name].grad) < 0.05, name


def test_the_step_runs_and_repeats():
    """All of it, twice: every sum of the path has a fixed order."""
    train = runpy.run_path(PATH)["train"]
    first = train(steps=6)
    assert all(v == v and v < 1e3 for v in first)
    assert train(steps=6) == first
    train(steps=2, nodes=3, **SIZES[1])
