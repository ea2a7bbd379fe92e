"""Layer norm and its gradients against the formulas in 64 bits, on the GPU.

Tolerances. With u the unit roundoff of the output's type (2^-24, 2^-8, 2^-11):
a sum over a row has at most 64 rounding steps of fp32 in sequence (32 in a
thread, 10 over the warps, a few scalings), so the mean is off by at most
64 * 2^-24 * mean|x|, and so is (x - mean) * rstd by that times rstd; every
other step adds a few relative 2^-24. The output adds u of itself. A column sum
of n terms in any fixed order is off by at most n * 2^-24 * sum|terms|; with
the sums split over blocks and joined, the longest chain is far shorter, and
128 + n / 128 steps bound it.
"""
import pytest
import torch

from top_gradient_compression_gb300 import api

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
F32 = 2.0 ** -24
TYPES = [torch.float32, torch.bfloat16, torch.float16]
# (rows, dim): one element, one warp's row, odd widths, the switch between a warp's and
# a block's rows, unaligned and long rows, rows beyond a block's registers
SHAPES = [(1, 1), (3, 2), (5, 7), (1, 1024), (33, 64), (257, 512), (9, 513), (64, 1023),
          (130, 1032), (17, 4096), (5, 8191), (4, 8200), (3, 16384), (2, 16389), (2, 40_000)]


def make(rows, dim, dtype, seed, pad=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)
    x = (normal(rows, dim + pad) * 2 + 3).to(dtype)[:, :dim]
    dy = normal(rows, dim + pad).to(dtype)[:, :dim]
    w, b = (1 + 0.2 * normal(dim)).to(dtype), (0.5 * normal(dim)).to(dtype)
    return x, dy, w, b


def reference(x, w, b, eps):
    x = x.double()
    mean = x.mean(-1, keepdim=True)
    rstd = ((x - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    xh = (x - mean) * rstd
    y = xh * (1.0 if w is None else w.double()) + (0.0 if b is None else b.double())
    return y, mean[..., 0], rstd[..., 0], xh


def check_forward(x, w, b, eps, got):
    y, mean, rstd = got
    ry, rmean, rrstd, xh = reference(x, w, b, eps)
    spread = x.double().abs().mean(-1)
    wa = torch.ones(x.shape[-1], device=DEV).double() if w is None else w.double().abs()
    off = 64 * F32 * (1 + spread * rrstd)[..., None] * (xh.abs() + 1) * wa
    assert ((mean.double() - rmean).abs() <= 64 * F32 * spread + 1e-37).all()
    assert ((rstd.double() - rrstd).abs() <= 64 * F32 * (1 + spread * rrstd) * rrstd).all()
    tol = off + (U[x.dtype] + 4 * F32) * ry.abs() + (2.0 ** -25 if x.dtype == torch.float16 else 0)
    assert ((y.double() - ry).abs() <= tol + (0 if b is None else 4 * F32 * b.double().abs())).all()


def check_backward(x, dy, w, mean, rstd, got, before=None):
    dx, dw, db = got
    x, dy, m, r = x.double(), dy.double(), mean.double()[:, None], rstd.double()[:, None]
    rows, dim = x.shape
    xh = (x - m) * r
    d = dy * (1.0 if w is None else w.double())
    c1, c2 = d.mean(1, keepdim=True), (d * xh).mean(1, keepdim=True)
    rdx = r * (d - c1 - xh * c2)
    # xh is off by a few roundings of x * rstd
    exh = 4 * F32 * ((x.abs() + m.abs()) * r)
    off = r * (8 * F32 * d.abs() + 64 * F32 * (d.abs().mean(1, keepdim=True)
               + (d * xh).abs().mean(1, keepdim=True) * (xh.abs() + 1))
               + exh * (c2.abs() + 1) + (d.abs() * exh).mean(1, keepdim=True) * (xh.abs() + 1))
    tol = off + U[got[0].dtype] * rdx.abs() + (2.0 ** -25 if got[0].dtype == torch.float16 else 0)
    assert ((dx.double() - rdx).abs() <= tol).all()
    steps = 128 + rows / 128
    rdw, rdb = (dy * xh).sum(0), dy.sum(0)
    edw = steps * F32 * (dy * xh).abs().sum(0) + (dy.abs() * exh).sum(0)
    edb = steps * F32 * dy.abs().sum(0)
    if before is not None:
        rdw, rdb = rdw + before[0].double(), rdb + before[1].double()
        edw, edb = edw + 2 * F32 * rdw.abs(), edb + 2 * F32 * rdb.abs()
    assert ((dw.double() - rdw).abs() <= edw + 1e-37).all()
    assert ((db.double() - rdb).abs() <= edb + 1e-37).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,dim", SHAPES)
def test_forward_and_backward(rows, dim, dtype):
    x, dy, w, b = make(rows, dim, dtype, rows * 131 + dim)
    got = api.layer_norm(x, w, b, 1e-5)
    check_forward(x, w, b, 1e-5, got)
    y, mean, rstd = got
    check_backward(x, dy, w, mean, rstd, api.layer_norm_backward(dy, x, mean, rstd, w))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,dim,pad", [(65, 768, 8), (65, 768, 5), (33, 100, 1), (6, 9000, 3)])
def test_strided_rows_and_unaligned_parameters(rows, dim, pad, dtype):
    """Rows of a wider array, weights and gradient slices at odd offsets of flat vectors."""
    x, dy, w, b = make(rows, dim, dtype, 5, pad)
    flat = torch.zeros(2 * dim + 3, dtype=dtype, device=DEV)
    flat[1:dim + 1], flat[dim + 2:2 * dim + 2] = w, b
    w, b = flat[1:dim + 1], flat[dim + 2:2 * dim + 2]
    wide = torch.full((rows, dim + pad), 7.0, dtype=dtype, device=DEV)
    y, mean, rstd = api.layer_norm(x, w, b, 1e-6, out=wide[:, :dim])
    check_forward(x, w, b, 1e-6, (y, mean, rstd))
    grad = torch.arange(2 * dim + 3, device=DEV, dtype=torch.float32) / dim
    before = grad.clone()
    dw, db = grad[1:dim + 1], grad[dim + 2:2 * dim + 2]
    wide2 = torch.full((rows, dim + pad), 7.0, dtype=dtype, device=DEV)
    got = api.layer_norm_backward(dy, x, mean, rstd, w, dx=wide2[:, :dim], dweight=dw, dbias=db,
                                  accumulate=True)
    check_backward(x, dy, w, mean, rstd, got, (before[1:dim + 1], before[dim + 2:2 * dim + 2]))
    assert (wide[:, dim:] == 7).all() and (wide2[:, dim:] == 7).all()
    for i in (0, dim + 1, 2 * dim + 2):
        assert grad[i] == before[i]


def test_types_of_weights_may_differ_and_be_missing():
    x, dy, w, b = make(40, 264, torch.bfloat16, 9)
    for wt in (w.float(), w.half(), None):
        for bt in (None, None if wt is None else b.to(wt.dtype)):
            got = api.layer_norm(x, wt, bt)
            check_forward(x, wt, bt, 1e-5, got)
        check_backward(x, dy, wt, got[1], got[2],
                       api.layer_norm_backward(dy, x, got[1], got[2], wt))


@pytest.mark.parametrize("rows,dim", [(40, 768), (40, 769), (5, 9000), (5, 9001)])
def test_in_place_gradients(rows, dim):
    """dx over dy or over x: the sums and dx come from what stood there before."""
    x, dy, w, b = make(rows, dim, torch.bfloat16, 21)
    y, mean, rstd = api.layer_norm(x, w, b)
    want = api.layer_norm_backward(dy, x, mean, rstd, w)
    for which in ("dy", "x"):
        args = {"dy": dy.clone(), "x": x.clone()}
        got = api.layer_norm_backward(args["dy"], args["x"], mean, rstd, w, dx=args[which])
        for p, q in zip(want, got):
            assert torch.equal(p, q)


def test_in_place_three_axes_and_no_rows():
    x, dy, w, b = make(24, 96, torch.float32, 3)
    y, mean, rstd = api.layer_norm(x, w, b)
    x3 = x.clone().view(4, 6, 96)
    y3, mean3, rstd3 = api.layer_norm(x3, w, b, out=x3)
    assert y3 is x3 and mean3.shape == (4, 6) and torch.equal(x3.view(24, 96), y)
    dx, dw, db = api.layer_norm_backward(dy, x, mean, rstd, w)
    dyc = dy.clone()
    dx2, dw2, db2 = api.layer_norm_backward(dyc, x, mean, rstd, w, dx=dyc)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)
    empty = x[:0]
    y0, m0, r0 = api.layer_norm(empty, w, b)
    assert y0.shape == (0, 96)
    _, dw0, db0 = api.layer_norm_backward(empty, empty, m0, r0, w)
    assert (dw0 == 0).all() and (db0 == 0).all()


@pytest.mark.parametrize("dim", [64, 1000, 1024, 40_000])
def test_nan_inf_and_constant_rows_stay_in_their_row(dim):
    x, dy, w, b = make(12, dim, torch.float32, 4)
    clean = api.layer_norm(x, w, b)
    x = x.clone()
    x[2, dim // 2], x[5, 0], x[7] = float("nan"), float("inf"), 4.0
    y, mean, rstd = api.layer_norm(x, w, b)
    for r in (2, 5):
        assert y[r].isnan().all()
    assert torch.equal(y[7], b) and mean[7] == 4.0
    keep = [r for r in range(12) if r not in (2, 5, 7)]
    assert torch.equal(y[keep], clean[0][keep])
    dx, dw, db = api.layer_norm_backward(dy, x, mean, rstd, w)
    assert dx[2].isnan().all() and dx[5].isnan().all() and not dx[keep + [7]].isnan().any()


def test_offset_much_larger_than_the_spread():
    """The variance is taken from the deviations, not from a difference of squares."""
    x, _, w, b = make(16, 2048, torch.float32, 6)
    x = x + 3000.0
    check_forward(x, w, b, 1e-5, api.layer_norm(x, w, b, 1e-5))


def test_gradients_against_differences():
    """Central differences of sum(y * v) in 64 bits, with a step of 1e-5: their own
    error is about 1e-10 + eps64 / 1e-5; the kernel's is fp32 rounding."""
    x, dy, w, b = make(3, 20, torch.float32, 8)
    y, mean, rstd = api.layer_norm(x, w, b)
    dx, dw, db = api.layer_norm_backward(dy, x, mean, rstd, w)

    def f(x, w, b):
        return float((reference(x, w, b, 1e-5)[0] * dy.double()).sum())
    for t, g in ((x, dx), (w, dw), (b, db)):
        base = t.double()
        for i in range(0, t.numel(), 7):
            ends = []
            for s in (1e-5, -1e-5):
                moved = base.clone()
                moved.view(-1)[i] += s
                args = [moved if t is q else q.double() for q in (x, w, b)]
                ends.append(f(*args))
            slope = (ends[0] - ends[1]) / 2e-5
            assert abs(slope - float(g.reshape(-1)[i])) <= 2e-5 * (1 + abs(slope))


def test_the_same_call_gives_the_same_bits_on_another_stream():
    x, dy, w, b = make(3001, 1023, torch.float16, 10)
    y, mean, rstd = api.layer_norm(x, w, b)
    first = api.layer_norm_backward(dy, x, mean, rstd, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        y2, mean2, rstd2 = api.layer_norm(x, w, b)
        again = api.layer_norm_backward(dy, x, mean2, rstd2, w)
    side.synchronize()
    assert torch.equal(y, y2)
    for p, q in zip(first, again):
        assert torch.equal(p, q)


def test_refusals():
    x, dy, w, b = make(4, 16, torch.float32, 1)
    y, mean, rstd = api.layer_norm(x, w, b)
    with pytest.raises(TypeError):
        api.layer_norm(x.double(), w, b)
    with pytest.raises(TypeError):
        api.layer_norm(x, w, b.half())
    with pytest.raises(TypeError):
        api.layer_norm(x.cpu(), w, b)
    with pytest.raises(ValueError):
        api.layer_norm(x.t(), w, b)
    with pytest.raises(ValueError):
        api.layer_norm(x, w[:8], b)
    with pytest.raises(ValueError):
        api.layer_norm(torch.zeros(4, 6, 16, device=DEV)[:, ::4].transpose(0, 1)[:, ::3], w, b)
    with pytest.raises(api.SparcmlError):
        api.layer_norm(x, w, b, -1.0)
    with pytest.raises(api.SparcmlError):
        api.layer_norm(x, w, b, out=x[:1].expand(4, 16))
    with pytest.raises(TypeError):
        api.layer_norm_backward(dy.half(), x, mean, rstd, w)
    with pytest.raises(ValueError):
        api.layer_norm_backward(dy, x, mean[:2], rstd, w)
    with pytest.raises(ValueError):
        api.layer_norm_backward(dy, x, mean, rstd, w, accumulate=True)
    with pytest.raises(api.SparcmlError):
        api.layer_norm_backward(dy, x, mean, rstd, w, ws=api.workspace(256, DEV))


# (rows, dim): many and few rows of one to 64 packs and of odd widths beside them, which share a
# warp in different ways; blocks' sums just within and beyond what the last block joins
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,dim", [(1217, 8), (1217, 40), (2049, 45), (1301, 72), (1300, 128),
                                      (1250, 130), (1219, 249), (1217, 256), (1217, 264),
                                      (1217, 512), (65, 512), (64, 512), (73, 512), (129, 129),
                                      (700, 16), (40, 104)])
def test_rows_that_share_warps_and_sums_that_are_joined(rows, dim, dtype):
    x, dy, w, b = make(rows, dim, dtype, rows + dim)
    got = api.layer_norm(x, w, b, 1e-5)
    check_forward(x, w, b, 1e-5, got)
    y, mean, rstd = got
    ws = api.workspace(api.layer_norm_backward_workspace_size(rows, dim), DEV)
    first = api.layer_norm_backward(dy, x, mean, rstd, w, ws=ws)
    check_backward(x, dy, w, mean, rstd, first)
    again = api.layer_norm_backward(dy, x, mean, rstd, w, ws=ws)  # the same workspace, and bits
    for p, q in zip(first, again):
        assert torch.equal(p, q)
