"""Linear layers of experts against the formulas in 64 bits.

Tolerances. A result is rounded once, by half a step at most; before that, its sum in fp32 adds 16
products at a time to the accumulator, and each such addition may drop what is below the last of
24 bits of the sum so far, which the sum of the products' magnitudes bounds: (depth / 16 + 2) 2^-22
of that, with a factor of two for the alignment of the products among themselves."""
import math

import pytest
import torch

from top_gradient_compression_gb300 import api

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]


def normal(seed, *shape):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=gen, device=DEV)


def offsets_of(sizes, start=0):
    at, out = start, [start]
    for s in sizes:
        at += s
        out.append(at)
    return torch.tensor(out, dtype=torch.int32, device=DEV)


def slack(depth):
    return (math.ceil(depth / 16) + 2) * 2.0 ** -22


def near(got, want, magnitude, depth, t):
    """got within its rounding to t and the sum's error; `magnitude`: of the products."""
    half = 0.0 if t == torch.float32 else torch.finfo(t).eps / 2
    least = 0.0 if t == torch.float32 else torch.finfo(t).smallest_normal * half
    bound = half * want.abs() + (1 + half) * slack(depth) * magnitude + least
    if t == torch.float32:
        bound = bound + 2.0 ** -24 * want.abs()
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), float((off / bound.clamp_min(1e-300)).max())


class Case:
    """Operands, and results in 64 bits with the sums of the products' magnitudes."""

    def __init__(self, t, sizes, n, k, before=0, behind=0, seed=0):
        self.t, self.n, self.k, self.sizes, self.before = t, n, k, sizes, before
        self.rows = before + sum(sizes) + behind
        self.offsets = offsets_of(sizes, before)
        self.x = normal(seed, self.rows, k).to(t)
        self.w = normal(seed + 1, len(sizes), n, k).mul_(0.1).to(t)
        self.dy = normal(seed + 2, self.rows, n).to(t)

    def runs(self):
        at = self.before
        for e, s in enumerate(self.sizes):
            yield e, slice(at, at + s)
            at += s

    def want(self, x=None, dy=None):
        x = (self.x if x is None else x).double()
        dy, w = (self.dy if dy is None else dy).double(), self.w.double()
        y, dx, dw = (torch.zeros(2, *s, dtype=torch.float64, device=DEV)
                     for s in ((self.rows, self.n), (self.rows, self.k), self.w.shape))
        for e, r in self.runs():
            for i, f in enumerate((lambda v: v, torch.abs)):
                y[i, r] = f(x[r]) @ f(w[e]).t()
                dx[i, r] = f(dy[r]) @ f(w[e])
                dw[i, e] = f(dy[r]).t() @ f(x[r])
        return y, dx, dw

    def check(self, y=None, dx=None, dw=None, want=None):
        wy, wdx, wdw = self.want() if want is None else want
        for e, r in self.runs():
            if y is not None:
                near(y[r], wy[0, r], wy[1, r], self.k, self.t)
            if dx is not None:
                near(dx[r], wdx[0, r], wdx[1, r], self.n, self.t)
            if dw is not None:
                near(dw[e], wdw[0, e], wdw[1, e], self.sizes[e], torch.float32)


SIZES = [
    ([1], 8, 8), ([1], 1, 1), ([3], 2, 5), ([64], 64, 64), ([300], 256, 64), ([65], 257, 129),
    ([0, 1, 0, 255, 0], 128, 72), ([256, 257, 63, 64, 65], 264, 200), ([7, 0, 130], 777, 333),
    ([513], 1000, 96), ([1] * 40, 136, 80), ([2, 30, 0, 1] * 12, 40, 24),
    ([16, 17, 15, 33, 1], 512, 512),
]


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("sizes,n,k", SIZES)
def test_all_three_products(t, sizes, n, k):
    c = Case(t, sizes, n, k, before=3, behind=5)
    ws = api.workspace(api.expert_linear_workspace_size(c.rows, len(sizes), n, k), DEV)
    y = torch.full((c.rows, n), 7.0, dtype=t, device=DEV)
    dx = torch.full((c.rows, k), 7.0, dtype=t, device=DEV)
    assert api.expert_linear(c.x, c.w, c.offsets, out=y, ws=ws) is y
    _, dw = api.expert_linear_backward(c.dy, c.x, c.w, c.offsets, dx=dx, ws=ws)
    assert api.get_status(ws) == 0
    c.check(y, dx, dw)
    for out in (y, dx):  # rows of no expert
        assert bool((out[:3] == 7.0).all()) and bool((out[c.rows - 5:] == 7.0).all())
