"""Norm and rotation of queries and keys against the formulas in 64 bits.

Tolerances. A result is rounded once, by half a step. Before that, in units of 2^-24 of the sizes
of a pair's two terms: the sum of squares 20 (half of it in the root), the root 4, products 6, the
sine and cosine 4 each and their angle, of 2^-26 of a turn, 6.3: 40 with what rounding adds up to.
The gradients have two sums over a head: 80. The weights' gradients add one for each token of a
warp and 350 for the blocks."""
import decimal

import pytest
import torch

from top_gradient_compression_gb300 import api

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
UNIT = 2.0 ** -24
EPS = 1e-6


def normal(seed, *shape):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=gen, device=DEV)


def frequencies(pairs, base=10000.0):
    i = torch.arange(pairs, dtype=torch.float64, device=DEV)
    return (base ** (-i / max(1, pairs))).float()


class Case:
    def __init__(self, t, tokens, q, k, dim, turned, pairs, layout="packed", weights=True,
                 seed=0, start=0, wide=False):
        self.pairs, self.turned, self.t = pairs, turned, t
        self.positions = torch.arange(tokens, device=DEV) * 3 + start
        self.positions = self.positions.to(torch.int64 if wide else torch.int32)
        self.freqs = frequencies(turned // 2)
        self.x = self.arrays(layout, seed, tokens, q, k, dim)
        self.g = self.arrays("own", seed + 1, tokens, q, k, dim)
        self.w = [(1 + 0.1 * normal(seed + 2 + i, dim)).to(t) if weights else None
                  for i in range(2)]

    def arrays(self, layout, seed, tokens, q, k, dim):
        x = normal(seed + 10, tokens, q + k + 1, dim).to(self.t)
        if layout == "own":
            both = x[:, :q].contiguous(), x[:, q:q + k].contiguous()
        elif layout == "shifted":  # heads one element off every alignment
            flat = torch.zeros(tokens * (q + k + 1) * dim + 1, dtype=self.t, device=DEV)
            x = flat[1:].view(x.shape).copy_(x)
            both = x[:, :q], x[:, q:q + k]
        elif layout == "heads first":
            x = x.transpose(0, 1).contiguous().transpose(0, 1)
            both = x[:, :q], x[:, q:q + k]
        else:
            both = x[:, :q], x[:, q:q + k]
        return [v if n else None for v, n in zip(both, (q, k))]

    def phase(self):
        angle = self.positions.double()[:, None] * self.freqs.double()
        return angle.cos()[:, None], angle.sin()[:, None]

    def split(self, x):
        r = x[..., :self.turned]
        a, b = (r[..., 0::2], r[..., 1::2]) if self.pairs else r.chunk(2, -1)
        return a, b, x[..., self.turned:]

    def join(self, a, b, rest):
        r = torch.stack([a, b], -1).flatten(-2) if self.pairs else torch.cat([a, b], -1)
        return torch.cat([r, rest], -1)

    def turn(self, x, back=False):
        """x turned, and the sum of the sizes of a pair's members at both."""
        c, s = self.phase()
        s = -s if back else s
        a, b, rest = self.split(x)
        size = a.abs() + b.abs()
        return (self.join(a * c - b * s, a * s + b * c, rest),
                self.join(size, size, rest.abs()))

    def root(self, x):
        return 1.0 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()

    def forward(self, **more):
        return api.head_norm_rotary(*self.x, self.positions, self.freqs, *self.w, EPS, self.pairs,
                                    **more)

    def backward(self, **more):
        return api.head_norm_rotary_backward(*self.g, *self.x, self.positions, self.freqs, *self.w,
                                             EPS, self.pairs, **more)

    def near(self, got, want, size, units):
        half = 0 if self.t == torch.float32 else torch.finfo(self.t).eps / 2
        least = 0 if self.t == torch.float32 else torch.finfo(self.t).smallest_normal * half
        bound = half * want.abs() + (1 + half) * units * UNIT * size + least
        off = (got.double() - want).abs()
        assert bool((off <= bound).all()), float((off / bound.clamp_min(1e-300)).max())

    def check_forward(self, got):
        for x, w, y in zip(self.x, self.w, got):
            if x is None:
                assert y is None
                continue
            u = x.double() * self.root(x.double()) * (1.0 if w is None else w.double())
            want, size = self.turn(u)
            self.near(y, want, size, 40)

    def check_backward(self, got, before=0.0):
        for i, (x, g, w) in enumerate(zip(self.x, self.g, self.w)):
            if x is None:
                assert got[i] is None and got[2 + i] is None
                continue
            v = x.double()
            r = self.root(v)
            t, tsize = self.turn(g.double(), back=True)
            f = 1.0 if w is None else w.double()
            wsize = 1.0 if w is None else w.double().abs()
            xh, d, dsize = v * r, t * f, tsize * wsize
            dx = r * (d - xh * (d * xh).mean(-1, keepdim=True))
            size = r * (dsize + xh.abs() * (dsize * xh.abs()).mean(-1, keepdim=True))
            self.near(got[i], dx, size, 80)
            dw, mag = (t * xh).sum((0, 1)), (tsize * xh.abs()).sum((0, 1))
            off = (got[2 + i].double() - before - dw).abs()
            n = x.shape[0] * x.shape[1]
            assert bool((off <= (n / 300 + 400) * UNIT * mag + 4 * UNIT * abs(before)).all())


SHAPES = [
    # tokens, q heads, k heads, elements, turned
    (1, 1, 1, 2, 2), (1, 32, 8, 128, 128), (5, 3, 1, 64, 64), (4, 2, 2, 80, 80), (4, 2, 2, 80, 40),
    (3, 5, 2, 96, 48), (6, 4, 1, 256, 256), (3, 2, 1, 512, 512), (3, 1, 1, 264, 264),
    (7, 6, 2, 37, 12), (5, 2, 1, 7, 6), (4, 1, 2, 1, 0), (9, 2, 2, 66, 66), (3, 3, 1, 511, 100),
    (200, 7, 1, 112, 112), (3, 2, 2, 128, 0), (2, 1, 1, 192, 64), (41, 1, 1, 16, 16),
]


@pytest.mark.parametrize("pairs", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_both_passes(shape, t, pairs):
    c = Case(t, *shape, pairs, start=17)
    c.check_forward(c.forward())
    c.check_backward(c.backward())


@pytest.mark.parametrize("layout", ["own", "shifted", "heads first"])
@pytest.mark.parametrize("t", TYPES, ids=str)
def test_layouts(layout, t):
    for dim, turned in ((128, 128), (72, 24)):
        c = Case(t, 11, 4, 2, dim, turned, False, layout, seed=3)
        c.check_forward(c.forward())
        c.check_backward(c.backward())


def test_outputs_of_other_strides_and_in_place():
    c = Case(torch.bfloat16, 13, 4, 2, 64, 64, False, "packed")
    want = c.forward()
    # heads first
    out = [torch.zeros(h, 13, 64, dtype=c.t, device=DEV).transpose(0, 1) for h in (4, 2)]
    got = c.forward(q_out=out[0], k_out=out[1])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    gwant = c.backward()
    got = c.backward(dq_out=out[0], dk_out=out[1])
    assert all(torch.equal(a, b) for a, b in zip(got, gwant))
    dq, dk = c.backward(dq_out=c.g[0], dk_out=c.g[1])[:2]  # over the results' gradients
    assert dq is c.g[0] and torch.equal(dq, gwant[0]) and torch.equal(dk, gwant[1])
    got = c.forward(q_out=c.x[0], k_out=c.x[1])  # in the projection itself
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_one_side_alone():
    c = Case(torch.float16, 9, 3, 0, 48, 48, True)
    c.check_forward(c.forward())
    c.check_backward(c.backward())
    c = Case(torch.float16, 9, 0, 3, 48, 48, True)
    c.check_forward(c.forward())
    c.check_backward(c.backward())


def test_weights_of_another_type_or_none():
    c = Case(torch.bfloat16, 9, 3, 2, 64, 64, False)
    c.w = [w.float() for w in c.w]
    c.check_forward(c.forward())
    c.check_backward(c.backward())
    c.w = [None, c.w[1]]
    c.check_forward(c.forward())
    c.w = [None, None]
    c.check_forward(c.forward())
    c.check_backward(c.backward())


def test_gradients_added_into_slices():
    c = Case(torch.float32, 70, 4, 2, 40, 40, False)
    flat = torch.full((85,), 0.25, device=DEV)
    got = c.backward(dq_weight=flat[1:41], dk_weight=flat[43:83], accumulate=True)
    c.check_backward(got, 0.25)
    assert float(flat[0]) == float(flat[41]) == float(flat[42]) == float(flat[83]) == 0.25


def exact_angle(position, freq):
    """position * freq without whole turns, from 80 digits."""
    with decimal.localcontext() as ctx:
        ctx.prec = 80
        two_pi = 2 * decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097"
                                     "49445923078164062862090")
        return float(decimal.Decimal(position) * decimal.Decimal(freq) % two_pi)


@pytest.mark.parametrize("position", [0, 1, -1, 12345, -98765, (1 << 20) + 1, (1 << 31) - 1,
                                      -(1 << 31), (1 << 38) + 12347])
def test_far_positions(position):
    """The angle of any position: against cosines and sines of the exact one. A head of one pair at
    a time, (1, 0) before it is normed: r = sqrt(2) after. The angle is off by 2^-26 of a turn
    and 2^-64 of one for each position, cosine and sine by 2^-22."""
    freqs = [1.0, 0.7310585, 0.1, 1e-4, 3.0, 123.456]
    f = torch.tensor(freqs, dtype=torch.float32, device=DEV)
    x = torch.zeros(1, 1, 12, device=DEV)
    x[..., :6] = 1.0
    p = torch.tensor([position], dtype=torch.int64, device=DEV)
    got = api.head_norm_rotary(x, None, p, f, eps=0.0)[0][0, 0].double() / 2 ** 0.5
    angles = torch.tensor([exact_angle(position, float(v)) for v in f.tolist()],
                          dtype=torch.float64, device=DEV)
    bound = 6.2832 * (2.0 ** -26 + abs(position) * 2.0 ** -64) + 2.0 ** -22
    assert bool(((got[:6] - angles.cos()).abs() <= bound).all())
    assert bool(((got[6:] - angles.sin()).abs() <= bound).all())
    if -(1 << 31) <= position < 1 << 31:
        narrow = api.head_norm_rotary(x, None, p.to(torch.int32), f, eps=0.0)[0]
        assert torch.equal(narrow[0, 0].double() / 2 ** 0.5, got)


@pytest.mark.parametrize("position", [12345, (1 << 31) - 1, (1 << 40) + 12347])
def test_frequencies_of_either_sign(position):
    """-f turns the other way by the same angle, at far positions too; bounds as above."""
    f = torch.tensor([0.7310585, 1e-4, 3.0, 1.1e-7], dtype=torch.float32, device=DEV)
    x = torch.zeros(1, 1, 16, device=DEV)
    x[..., :8] = 1.0
    p = torch.tensor([position], dtype=torch.int64, device=DEV)
    got = api.head_norm_rotary(x, None, p, torch.cat([f, -f]), eps=0.0)[0][0, 0].double() / 2 ** 0.5
    angles = torch.tensor([exact_angle(position, float(v)) for v in f.tolist()],
                          dtype=torch.float64, device=DEV)
    want = torch.cat([angles.cos(), angles.cos(), angles.sin(), -angles.sin()])
    bound = 6.2832 * (2.0 ** -26 + position * 2.0 ** -64) + 2.0 ** -22
    assert bool(((got - want).abs() <= bound).all())


@pytest.mark.parametrize("t", TYPES, ids=str)
def test_no_epsilon(t, monkeypatch):
    """With heads that leave lanes idle, which must add nothing to the weights' gradients."""
    monkeypatch.setitem(globals(), "EPS", 0.0)
    for dim in (64, 40, 6):
        c = Case(t, 3, 3, 1, dim, dim // 4 * 2, False)
        c.check_forward(c.forward())
        c.check_backward(c.backward())


def test_nan_stays_in_its_head():
    c = Case(torch.bfloat16, 6, 4, 2, 64, 64, False)
    c.x[0][3, 1, 5] = float("nan")
    c.x[1][2, 0, 7] = float("inf")
    q, k = c.forward()
    assert q.isnan().flatten(2).any(2).nonzero().tolist() == [[3, 1]]
    assert (~k.isfinite()).any(2).nonzero().tolist() == [[2, 0]]
    dq, dk, wq, wk = c.backward()
    assert dq.isnan().any(2).nonzero().tolist() == [[3, 1]]
    assert dk.isnan().any(2).nonzero().tolist() == [[2, 0]]
    assert bool(wq.isnan().all()) and bool(wk.isnan().any())


def test_no_tokens():
    c = Case(torch.float32, 3, 2, 1, 16, 16, False)
    x = [v[:0] for v in c.x]
    q, k = api.head_norm_rotary(*x, c.positions[:0], c.freqs)
    assert q.shape == (0, 2, 16) and k.shape == (0, 1, 16)
    dq, dk, wq, wk = api.head_norm_rotary_backward(*x, *x, c.positions[:0], c.freqs)
    assert dq.shape == (0, 2, 16) and float(wq.abs().sum() + wk.abs().sum()) == 0.0


def test_against_differences():
    """The gradient along a direction against the change of the forward pass, both in fp32: steps of
    2^-6 leave a third of its square of the third derivative (below 1e-3 of the sum of sizes here)
    and rounding errors of 80 units over the step."""
    for pairs in (False, True):
        c = Case(torch.float32, 20, 3, 2, 24, 16, pairs, "own")
        h = 2.0 ** -6
        dq, dk, wq, wk = c.backward()
        x, w = c.x, [v.clone() for v in c.w]
        for i, d in ((0, dq), (1, dk)):
            v = normal(40 + i, *d.shape)
            ends = []
            for s in (h, -h):
                c.x = list(x)
                c.x[i] = x[i] + s * v
                ends.append((c.forward()[i].double() * c.g[i].double()).sum())
            c.x = x
            size = (d.double() * v).abs().sum()
            assert abs((ends[0] - ends[1]) / (2 * h) - (d.double() * v).sum()) <= \
                1e-3 * size + 80 * UNIT / h * c.g[i].double().abs().sum()
        for i, d in ((0, wq), (1, wk)):
            v = normal(50 + i, 24)
            ends = []
            for s in (1.0, -1.0):
                c.w = list(w)
                c.w[i] = w[i] + s * v
                ends.append((c.forward()[i].double() * c.g[i].double()).sum())
            c.w = w
            size = c.g[i].double().abs().sum() * 6
            assert abs((ends[0] - ends[1]) / 2 - (d.double() * v).sum()) <= 500 * UNIT * size


def test_the_same_bits_every_time_and_captured():
    c = Case(torch.bfloat16, 700, 8, 2, 128, 128, False)
    ws = api.workspace(api.head_norm_rotary_backward_workspace_size(700, 8, 2, 128), DEV)
    want, gwant = c.forward(), c.backward(ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = c.forward()
        g = c.backward(ws=ws)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(y + g, want + gwant))
    c.positions.add_(1)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(y[0], want[0])
    c.check_forward(y)
