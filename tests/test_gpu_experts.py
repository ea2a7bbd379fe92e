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


@pytest.mark.parametrize("t", TYPES, ids=str)
def test_wide_and_tall_tiles(t):
    """Several tiles each way, rows in several tiles, and bands of tiles."""
    c = Case(t, [700, 0, 1500, 9], 600, 520)
    y = api.expert_linear(c.x, c.w, c.offsets)
    c.check(y, *api.expert_linear_backward(c.dy, c.x, c.w, c.offsets))
    c = Case(t, [2600], 300, 2304)
    y = api.expert_linear(c.x, c.w, c.offsets)
    c.check(y, *api.expert_linear_backward(c.dy, c.x, c.w, c.offsets))


@pytest.mark.parametrize("sizes,n,k", [([1], 300, 9000), ([5, 0, 3], 256, 5000), ([40], 4100, 264),
                                       ([130], 9000, 72)])
def test_split_sums(sizes, n, k):
    """A long summed axis with few tiles, taken in parts: forward by k, dx by n."""
    c = Case(torch.bfloat16, sizes, n, k, before=1, behind=2)
    ws = api.workspace(api.expert_linear_workspace_size(c.rows, len(sizes), n, k), DEV)
    first = None
    for _ in range(3):
        y = api.expert_linear(c.x, c.w, c.offsets, ws=ws)
        dx, dw = api.expert_linear_backward(c.dy, c.x, c.w, c.offsets, ws=ws)
        c.check(y, dx, dw)
        rows = slice(1, c.rows - 2)
        got = (y[rows].clone(), dx[rows].clone(), dw)
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


@pytest.mark.parametrize("sizes,n,k", [([256], 4096, 1024), ([300], 8192, 2048),
                                       ([120, 0, 250, 65], 520, 640), ([333, 14], 1033, 4100)])
def test_fewer_rows_per_tile_where_tiles_are_few(sizes, n, k):
    """64, 128 and 256 rows, with and without parts of the summed axis."""
    c = Case(torch.bfloat16, sizes, n, k, before=2, behind=7)
    ws = api.workspace(api.expert_linear_workspace_size(c.rows, len(sizes), n, k), DEV)
    y = api.expert_linear(c.x, c.w, c.offsets, ws=ws)
    dx, _ = api.expert_linear_backward(c.dy, c.x, c.w, c.offsets, need_dweight=False, ws=ws)
    c.check(y, dx)
    assert api.get_status(ws) == 0


@pytest.mark.parametrize("sizes,n,k", [([5000], 264, 96), ([700, 0, 3000, 77], 256, 256),
                                       ([1025, 511, 512, 513], 300, 257), ([9000, 1], 40, 24)])
def test_split_weight_gradients(sizes, n, k):
    """Long runs of rows with few tiles, taken in parts, some experts' whole."""
    c = Case(torch.float16, sizes, n, k, before=3, behind=4)
    want = c.want()
    first = None
    for _ in range(3):
        _, dw = api.expert_linear_backward(c.dy, c.x, c.w, c.offsets, need_dx=False)
        c.check(dw=dw, want=want)
        first = dw if first is None else first
        assert torch.equal(first, dw)


def test_long_sums_are_not_biased():
    """Sums of 20,000 products of one sign, where an accumulator that drops bits would lose 2e-5."""
    x, dy = (normal(i, 20000, 72).abs().to(torch.bfloat16) for i in (1, 2))
    w = torch.zeros(72, 72, dtype=torch.bfloat16, device=DEV)
    _, dw = api.expert_linear_backward(dy, x, w, need_dx=False)
    want = dy.double().t() @ x.double()
    # 32 additions of 16 products to an accumulator, 40 rounded sums of accumulators
    assert float(((dw.double() - want) / want).abs().max()) <= 34 * 2.0 ** -22


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("sizes,n,k", [([300], 264, 200), ([65, 0, 129], 100, 333),
                                       ([1, 63, 64, 65, 700], 256, 384), ([3000], 40, 513)])
def test_from_8_bits(t, sizes, n, k):
    c = Case(t, sizes, n, k, before=2, behind=3)
    kept = api.checkpoint8(c.x)
    x = api.restore8(kept)
    ws = api.workspace(api.expert_linear_workspace_size(c.rows, len(sizes), n, k), DEV)
    dx, dw = api.expert_linear_backward(c.dy, kept, c.w, c.offsets, ws=ws)
    c.check(dx=dx, dw=dw, want=c.want(x=x))
    # c 2^e is an operand as it is: the same as from x restored
    _, same = api.expert_linear_backward(c.dy, x, c.w, c.offsets, need_dx=False, ws=ws)
    assert torch.equal(dw, same)


@pytest.mark.parametrize("stored", [False, True])
def test_what_is_not_finite_stays_with_its_expert(stored):
    c = Case(torch.bfloat16, [70, 30, 60], 136, 264, before=5, behind=6)
    for bad in (float("nan"), float("inf")):
        x, dy, w = c.x.clone(), c.dy.clone(), c.w.clone()
        x[:5], dy[:5] = bad, bad            # rows of no expert
        x[-6:], dy[-6:] = bad, bad
        x[80], dy[82] = bad, bad            # the second expert's, in the block of the first's end
        w[1, 3, 4] = bad
        y = api.expert_linear(x, w, c.offsets)
        dx, dw = api.expert_linear_backward(dy, api.checkpoint8(x) if stored else x, w, c.offsets)
        wy, wdx, wdw = c.want(x=api.restore8(api.checkpoint8(x)) if stored else x)
        for e, r in ((0, slice(5, 75)), (2, slice(105, 165))):
            near(y[r], c.want()[0][0, r], c.want()[0][1, r], c.k, c.t)
            near(dx[r], wdx[0, r], wdx[1, r], c.n, c.t)
            near(dw[e], wdw[0, e], wdw[1, e], c.sizes[e], torch.float32)
        assert not bool(y[80].isfinite().any()) and not bool(dx[82].isfinite().any())
        # other rows of the second expert: only where its own matrix is not finite
        assert bool(y[90, :3].isfinite().all()) and not bool(y[90, 3].isfinite())
        assert bool(dx[90, :4].isfinite().all()) and not bool(dx[90, 4].isfinite())


@pytest.mark.parametrize("offsets,want", [([0, 50, 30, 90], [0, 50, 50, 90]),
                                          ([-5, 20, 60, 200], [0, 20, 60, 100]),
                                          ([70, 60, 50, 40], [70, 70, 70, 70]),
                                          ([0, 2 ** 31 - 1, -2 ** 31, 100], [0, 100, 100, 100])])
def test_offsets_out_of_order_or_range(offsets, want):
    """They count as the nearest that are not, and the workspace says so."""
    c = Case(torch.bfloat16, [100, 0, 0], 72, 40)
    ws = api.workspace(api.expert_linear_workspace_size(100, 3, 72, 40), DEV)
    results = []
    for o in (offsets, want):
        off = torch.tensor(o, dtype=torch.int32, device=DEV)
        y = torch.full((100, 72), 5.0, dtype=c.t, device=DEV)
        dx = torch.full((100, 40), 5.0, dtype=c.t, device=DEV)
        api.expert_linear(c.x, c.w, off, out=y, ws=ws)
        status = api.get_status(ws)
        _, dw = api.expert_linear_backward(c.dy, c.x, c.w, off, dx=dx, ws=ws)
        assert api.get_status(ws) == status == (4 if o is offsets else 0)
        results.append((y, dx, dw))
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_one_matrix_without_offsets():
    c = Case(torch.float16, [333], 100, 88)
    y = api.expert_linear(c.x, c.w[0])
    dx, dw = api.expert_linear_backward(c.dy, c.x, c.w[0])
    assert dw.shape == (100, 88)
    c.check(y, dx, dw[None])


def test_strided_and_unaligned_operands():
    """Slices at any offset, rows and matrices apart, and matrices whose rows alternate."""
    t, sizes, n, k = torch.bfloat16, [40, 25, 70], 104, 72
    c = Case(t, sizes, n, k)
    want = c.want()
    for shift, pad in ((0, 8), (1, 0), (3, 5)):
        def place(v, pad):
            wide = torch.full((*v.shape[:-1], v.shape[-1] + pad), 9.0, dtype=v.dtype, device=DEV)
            flat = torch.zeros(wide.numel() + 8, dtype=v.dtype, device=DEV)
            out = flat[shift:shift + wide.numel()].view(wide.shape)[..., :v.shape[-1]]
            return out.copy_(v)
        x, w, dy = place(c.x, pad), place(c.w, pad), place(c.dy, pad)
        y, dx = place(torch.zeros_like(c.dy), pad), place(torch.zeros_like(c.x), pad)
        dw = place(torch.zeros(c.w.shape, device=DEV), pad)
        api.expert_linear(x, w, c.offsets, out=y)
        got = api.expert_linear_backward(dy, x, w, c.offsets, dx=dx, dweight=dw)
        assert got[0] is dx and got[1] is dw
        c.check(y, dx, dw, want=want)
    w = c.w.transpose(0, 1).contiguous().transpose(0, 1)  # [n][experts][k] in memory
    dw = torch.zeros(n, 3, k, device=DEV).transpose(0, 1)
    y = api.expert_linear(c.x, w, c.offsets)
    dx, dw = api.expert_linear_backward(c.dy, c.x, w, c.offsets, dweight=dw)
    c.check(y, dx, dw, want=want)
    shared = c.w[:1].expand(3, n, k)  # one matrix for all experts
    c.w = shared.contiguous()
    y = api.expert_linear(c.x, shared, c.offsets)
    c.check(y)


def test_weight_gradients_added_into_a_flat_gradient():
    c = Case(torch.bfloat16, [40, 0, 70], 56, 40)
    flat = torch.full((3 * 56 * 40 + 7,), 0.5, device=DEV)
    dw = flat[3:3 + 3 * 56 * 40].view(3, 56, 40)
    api.expert_linear_backward(c.dy, c.x, c.w, c.offsets, dweight=dw, accumulate=True)
    want = c.want()[2]
    near(dw - 0.5, want[0], want[1] + 4.0, 70, torch.float32)  # and 0.5's own rounding
    assert bool((dw[1] == 0.5).all())
    assert float(flat[:3].sum() + flat[-4:].sum()) == 3.5
    _, dw = api.expert_linear_backward(c.dy, c.x, c.w, c.offsets, need_dx=False)
    assert float(dw[1].abs().sum()) == 0.0


@pytest.mark.parametrize("sizes, n, k", [([40, 0, 70], 56, 40), ([3900, 1100], 264, 72),
                                         ([300] * 20, 520, 513)], ids=["short", "deep", "many"])
def test_what_is_added_is_what_would_be_written(sizes, n, k):
    """One addition, rounded once, whether the sums come in one piece or in parts."""
    c = Case(torch.bfloat16, sizes, n, k)
    plain = api.expert_linear_backward(c.dy, c.x, c.w, c.offsets, need_dx=False)[1]
    before = normal(9, len(sizes) * n * k + 5)
    flat = before.clone()
    dw = flat[1:-4].view(len(sizes), n, k)
    api.expert_linear_backward(c.dy, c.x, c.w, c.offsets, dweight=dw, accumulate=True,
                               need_dx=False)
    assert torch.equal(flat[1:-4], before[1:-4] + plain.view(-1))
    assert torch.equal(flat[:1], before[:1]) and torch.equal(flat[-4:], before[-4:])


@pytest.mark.parametrize("stored", [False, True])
def test_no_rows(stored):
    w = normal(1, 4, 72, 40).to(torch.bfloat16)
    x, dy = (torch.zeros(0, i, dtype=torch.bfloat16, device=DEV) for i in (40, 72))
    off = torch.zeros(5, dtype=torch.int32, device=DEV)
    assert api.expert_linear(x, w, off).shape == (0, 72)
    dx, dw = api.expert_linear_backward(dy, api.checkpoint8(x) if stored else x, w, off)
    assert dx.shape == (0, 40) and float(dw.abs().sum()) == 0.0
    dw.fill_(2.0)
    api.expert_linear_backward(dy, x, w, off, dweight=dw, accumulate=True)
    assert bool((dw == 2.0).all())
    # rows, but none of them an expert's
    dx, dw = api.expert_linear_backward(dy.new_ones(9, 72), x.new_ones(9, 40), w, off)
    assert float(dw.abs().sum()) == 0.0


def test_as_many_experts_as_there_may_be():
    gen = torch.Generator().manual_seed(3)
    sizes = torch.randint(0, 4, (1024,), generator=gen).tolist()
    c = Case(torch.bfloat16, sizes, 24, 16)
    y = api.expert_linear(c.x, c.w, c.offsets)
    c.check(y, *api.expert_linear_backward(c.dy, c.x, c.w, c.offsets))


def test_captured_and_replayed_with_other_offsets():
    c = Case(torch.bfloat16, [100, 20, 80], 264, 136)
    ws = api.workspace(api.expert_linear_workspace_size(200, 3, 264, 136), DEV)
    graph = torch.cuda.CUDAGraph()
    kept = api.checkpoint8(c.x)
    c.x = api.restore8(kept)
    with torch.cuda.graph(graph):
        y = api.expert_linear(c.x, c.w, c.offsets, ws=ws)
        dx, dw = api.expert_linear_backward(c.dy, c.x, c.w, c.offsets, ws=ws)
        _, dw8 = api.expert_linear_backward(c.dy, kept, c.w, c.offsets, need_dx=False, ws=ws)
    for sizes in ([100, 20, 80], [0, 200, 0], [1, 64, 135]):
        c.sizes = sizes
        c.offsets.copy_(offsets_of(sizes))
        graph.replay()
        torch.cuda.synchronize()
        c.check(y, dx, dw)
        assert torch.equal(dw8, dw)


def test_two_calls_at_once():
    """On two streams, with a workspace of its own each."""
    cases = [Case(torch.bfloat16, [300, 500], 512, 264, seed=s) for s in (0, 50)]
    want = [(api.expert_linear(c.x, c.w, c.offsets),
             *api.expert_linear_backward(c.dy, c.x, c.w, c.offsets)) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [(api.expert_linear(c.x, c.w, c.offsets, stream=s),
                *api.expert_linear_backward(c.dy, c.x, c.w, c.offsets, stream=s))
               for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_against_differences():
    """The products are linear in each operand, so that a difference over any step is the gradient
    itself but for y's rounding, half a step of each value at both ends."""
    c = Case(torch.bfloat16, [50, 0, 33], 72, 40)
    dx, dw = api.expert_linear_backward(c.dy, c.x, c.w, c.offsets)
    v, u = (normal(7, *c.x.shape).to(c.t), normal(8, *c.w.shape).to(c.t))
    dy = c.dy.double()
    y = api.expert_linear(c.x, c.w, c.offsets).double()
    for got, change in (((dx.double() * v.double()).sum(), dict(x=(c.x.float() + v).to(c.t))),
                        ((dw.double() * u.double()).sum(), dict(w=(c.w.float() + u).to(c.t)))):
        x, w = change.get("x", c.x), change.get("w", c.w)
        # the step as it is after the operand's own rounding
        if "x" in change:
            got = (dx.double() * (x.double() - c.x.double())).sum()
        else:
            got = (dw.double() * (w.double() - c.w.double())).sum()
        far = api.expert_linear(x, w, c.offsets).double()
        slip = (dy.abs() * (far.abs() + y.abs())).sum() * 2.0 ** -9
        half = 2.0 ** -9 * (dx.double().abs() * (x.double() - c.x.double()).abs()).sum()
        assert abs((dy * (far - y)).sum() - got) <= slip + half + 1e-4 * slip


def test_a_wait_that_runs_out():
    """With a fault injected the first pair of SMs withholds its products: the call ends, says so,
    and the next one is right."""
    c = Case(torch.bfloat16, [300, 0, 500], 600, 264)
    ws = api.workspace(api.expert_linear_workspace_size(800, 3, 600, 264), DEV)
    api.set_fault_injection(ws, api.INJECT_WITHHOLD_FIRST)
    api.expert_linear(c.x, c.w, c.offsets, ws=ws)
    assert api.STATUS[api.get_status(ws)] == "SPARCML_ERR_TIMEOUT"
    for x in (c.x, api.checkpoint8(c.x)):
        api.expert_linear_backward(c.dy, x, c.w, c.offsets, need_dx=False, ws=ws)
        assert api.STATUS[api.get_status(ws)] == "SPARCML_ERR_TIMEOUT"
    api.set_fault_injection(ws, 0)
    y = api.expert_linear(c.x, c.w, c.offsets, ws=ws)
    c.check(y, *api.expert_linear_backward(c.dy, c.x, c.w, c.offsets, ws=ws))
    assert api.get_status(ws) == 0
