"""The sums of experts' linear layers over deep axes, where what an accumulator of the tensor cores
drops would show in a result of 16 bits.

Tolerance. An accumulator takes 1024 of the summed axis: 64 additions of 16 products and two for
their alignment, each of which may drop 2^-22 of the sum. The accumulators' sums are added in fp32,
a rounding of 2^-24 at most each. The result is rounded once, half a step of its own binade."""
import math

import pytest
import torch

from top_gradient_compression_gb300 import api

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

ROWS, SIDE = 64, 16


def positive(seed, *shape):
    """Between 2^-5 and 2^-4, so that 2^20 products of them stay within fp16's range."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.rand(*shape, generator=gen, device=DEV).add_(1.0).mul_(2.0 ** -5)


def near(got, want, depth):
    t = got.dtype
    digits = 1 - int(math.log2(torch.finfo(t).eps))  # of the significand
    half = torch.ldexp(torch.ones_like(want), torch.frexp(want)[1] - digits - 1)
    bound = half + (66 * 2.0 ** -22 + math.ceil(depth / 1024) * 2.0 ** -24) * want
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("depth", [2 ** 17 + 72, 2 ** 20])
def test_deep_sums_of_one_sign(t, depth):
    """A row for each of 64 experts that share a matrix: tiles enough that no sum is taken in
    parts."""
    off = torch.arange(ROWS + 1, dtype=torch.int32, device=DEV)
    x = positive(1, ROWS, depth).to(t)
    w = positive(2, SIDE, depth).to(t)
    y = api.expert_linear(x, w.expand(ROWS, SIDE, depth), off)
    near(y, x.double() @ w.double().t(), depth)
    w = w.t().contiguous()
    dx, _ = api.expert_linear_backward(x, y, w.expand(ROWS, depth, SIDE), off, need_dweight=False)
    near(dx, x.double() @ w.double(), depth)
