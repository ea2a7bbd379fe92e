"""Activations in 8 bits: codes, exponents and what they come back as bit for bit against the
definition in 64 bits, and the layer norm's gradients from them against the formula."""
import pytest
import torch

from top_gradient_compression_gb300 import api

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
RANGE = {torch.float32: (1, 248), torch.bfloat16: (1, 248), torch.float16: (103, 136)}


def normal(seed, *shape):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=gen, device=DEV)


def laid_out(x, t, pad, shift):
    """x in type t, its rows `pad` elements apart, from element `shift` of the memory on."""
    rows, dim = x.shape
    flat = torch.zeros(rows * (dim + pad) + shift + 8, dtype=t, device=DEV)
    v = flat[shift:shift + rows * (dim + pad)].view(rows, dim + pad)[:, :dim]
    return v.copy_(x)


def power(b):
    """2^(b - 127), exactly: powers on the device are off in their last bit."""
    table = torch.tensor([2.0 ** (i - 127) for i in range(256)], dtype=torch.float64, device=DEV)
    return table[b.long()]


def definition(x):
    """(codes, exponent bytes, values) in 64 bits, by trying the exponents one after the other."""
    rows, dim = x.shape
    least, most = RANGE[x.dtype]
    codes = torch.zeros(rows, (dim + 15) // 16 * 16, dtype=torch.int8, device=DEV)
    exponents = torch.zeros(rows, (dim + 127) // 128, dtype=torch.uint8, device=DEV)
    values = torch.zeros(rows, dim, dtype=torch.float64, device=DEV)
    v = x.double()
    for g in range(exponents.shape[1]):
        part = v[:, 128 * g:128 * g + 128]
        fine = part.isfinite().all(1)
        top = torch.where(fine, part.abs().amax(1), 0.0)
        b = torch.full_like(top, most)
        for e in range(most, least - 1, -1):
            b = torch.where(top * 2.0 ** (127 - e) < 127.5, float(e), b)
        c = torch.round(part / power(b)[:, None]).clamp(-127, 127)
        c = torch.where(fine[:, None], c, 0.0)
        codes[:, 128 * g:128 * g + part.shape[1]] = c.to(torch.int8)
        exponents[:, g] = torch.where(fine, b, 255.0).to(torch.uint8)
        values[:, 128 * g:128 * g + 128] = torch.where(fine[:, None], c * power(b)[:, None],
                                                       float("nan"))
    return codes, exponents, values


def same(a, b):
    return torch.equal(a.nan_to_num(0.125), b.nan_to_num(0.125)) and \
        torch.equal(a.isnan(), b.isnan())


def check(x):
    got = api.checkpoint8(x)
    codes, exponents, values = definition(x)
    assert torch.equal(got.exponents, exponents)
    assert torch.equal(got.codes, codes)
    assert got.dtype == x.dtype and got.shape == x.shape
    back = api.restore8(got)
    assert back.dtype == x.dtype and same(back.double(), values)
    return got


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("rows,dim,pad,shift", [
    (1, 1, 0, 0), (3, 15, 0, 0), (3, 16, 0, 0), (3, 17, 7, 1), (5, 127, 0, 0), (5, 128, 0, 0),
    (5, 129, 0, 0), (7, 777, 23, 0), (7, 776, 0, 3), (4, 1024, 8, 0), (4, 1024, 0, 1),
    (2, 8200, 0, 0), (2500, 264, 0, 0), (700, 500, 12, 2)])
def test_store_and_restore(t, rows, dim, pad, shift):
    spread = torch.exp2(torch.round(6 * normal(1, rows, 1)))
    check(laid_out(normal(2, rows, dim) * spread, t, pad, shift))


@pytest.mark.parametrize("t", TYPES, ids=str)
def test_borders(t):
    """The step's border, ties, signed zeros, the smallest and the largest numbers."""
    f = torch.finfo(t)
    rows = []
    for top in (127.0, 127.5, 127.4375, 128.0, 64.0, 63.5, 1.0, f.max, f.smallest_normal, 0.0):
        r = torch.zeros(128, dtype=torch.float64)
        r[0] = -top
        r[1:5] = torch.tensor([0.5, 1.5, 2.5, -0.0]) * (top / 128)
        r[5] = top / 300
        rows.append(r)
    tiny = torch.zeros(128, dtype=torch.float64)
    tiny[:4] = torch.tensor([1.0, 2.0, 3.0, -5.0]) * f.smallest_normal * f.eps  # subnormal
    rows.append(tiny)
    x = torch.stack(rows).to(device=DEV, dtype=t)
    got = check(x)
    assert int(got.codes.min()) >= -127
    assert bool(api.restore8(got).isfinite().all())
    # within half a step, but where the type's largest numbers saturate
    step = power(got.exponents)
    assert bool(((api.restore8(got).double() - x.double()).abs() <= step / 2)[x.abs() < f.max]
                .all())


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_a_group_that_is_not_finite(t, what):
    x = normal(3, 4, 300).to(t)
    x[1, 140] = what
    x[2, 299] = what
    got = check(x)
    back = api.restore8(got)
    assert bool(back[1, 128:256].isnan().all()) and bool(back[2, 256:].isnan().all())
    assert int(back.isnan().sum()) == 128 + 44


def test_other_shapes_and_types():
    x = normal(4, 3, 5, 200).to(torch.bfloat16)
    c = api.checkpoint8(x)
    assert c.codes.shape == (3, 5, 208) and c.exponents.shape == (3, 5, 2)
    flat = api.checkpoint8(x.view(15, 200))
    assert torch.equal(flat.codes, c.codes.view(15, 208))
    wide = api.restore8(c, dtype=torch.float32)
    assert torch.equal(wide, api.restore8(c).float())  # a bf16 number as it is
    out = torch.full((3, 5, 203), 9.0, device=DEV)[..., :200]
    assert api.restore8(c, out=out) is out and torch.equal(out, wide)
    again = api.checkpoint8(x, out=c)
    assert again is c
    empty = api.checkpoint8(x[:0])
    assert api.restore8(empty).shape == (0, 5, 200)
    vector = api.checkpoint8(x[0, 0])
    assert torch.equal(api.restore8(vector), api.restore8(c)[0, 0])


def test_codes_of_the_callers_own():
    """Any byte in either array stands for something."""
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).view(torch.int8).view(1, 256)
    for b in (0, 1, 100, 127, 254, 255):
        e = torch.tensor([[b, 127]], dtype=torch.uint8, device=DEV)
        got = api.restore8(api.Checkpoint8(codes, e, 256, torch.float32))[0].double()
        want = codes[0].double()
        want[:128] *= float("nan") if b == 255 else 2.0 ** (b - 127)
        want = torch.where(want.abs() < 2.0 ** 128, want, want.sign() * float("inf")) \
            if b != 255 else want
        assert same(got, want), b


# --------------------------------------------------------------------------- layer norm
def norm_case(t, rows, dim, pad, shift, seed=5):
    x = laid_out(normal(seed, rows, dim) * torch.exp(0.5 * normal(seed + 1, dim)) +
                 normal(seed + 2, dim), t, 0, 0)
    dy = laid_out(normal(seed + 3, rows, dim), t, pad, shift)
    w = (1 + 0.1 * normal(seed + 4, dim)).to(t)
    _, mean, rstd = api.layer_norm(x, w)
    return dy, api.checkpoint8(x), mean, rstd, w


def check_norm(dy, c, mean, rstd, w, got, before=(0.0, 0.0)):
    """dx is rounded once, by half a step. Before that: every product and sum of its own is
    rounded by 2^-24 of its size, a sum over the row by 64 of them at most (16 in a thread, the
    rest pairwise), the sums over rows by one for each row of a block and 330 for the blocks."""
    t, (rows, dim) = dy.dtype, dy.shape
    x, d0, r = api.restore8(c).double(), dy.double(), rstd.double()[:, None]
    xh = (x - mean.double()[:, None]) * r
    d = d0 * (1.0 if w is None else w.double())
    m0, m1 = d.mean(1, keepdim=True), (d * xh).mean(1, keepdim=True)
    dx = r * (d - m0 - xh * m1)
    unit = 2.0 ** -24
    size = r * (d.abs() + d.abs().mean(1, keepdim=True) +
                xh.abs() * (d * xh).abs().mean(1, keepdim=True))
    half = 0 if t == torch.float32 else torch.finfo(t).eps / 2
    least = 0 if t == torch.float32 else torch.finfo(t).smallest_normal * half
    assert bool(((got[0].double() - dx).abs() <= half * dx.abs() + 72 * unit * size + least).all())
    for g, want, mag, b in ((got[1], (d0 * xh).sum(0), (d0 * xh).abs().sum(0), before[0]),
                            (got[2], d0.sum(0), d0.abs().sum(0), before[1])):
        bound = (rows / 150 + 340) * unit * mag + 4 * unit * (want.abs() + b)
        assert bool(((g.double() - b - want).abs() <= bound).all())


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("rows,dim,pad,shift", [
    (1, 1, 0, 0), (2, 8, 0, 0), (9, 40, 0, 0), (3, 128, 0, 0), (70, 136, 0, 0), (33, 256, 8, 0),
    (1200, 96, 0, 0), (5, 264, 0, 0), (400, 1024, 0, 0), (7, 1023, 0, 0), (7, 1000, 5, 1),
    (3, 200, 0, 3), (650, 17, 0, 0), (20, 4096, 0, 0), (4, 4104, 0, 0), (3, 8192, 0, 0),
    (3, 8193, 0, 0), (5, 9000, 0, 1)])
def test_norm_gradients(t, rows, dim, pad, shift):
    case = norm_case(t, rows, dim, pad, shift)
    check_norm(*case, api.layer_norm_backward(*case))


@pytest.mark.parametrize("dim", [512, 777])
def test_norm_gradients_into_slices(dim):
    """Added into slices of a flat gradient at odd offsets, dx over dy, weights of another type."""
    dy, c, mean, rstd, _ = norm_case(torch.bfloat16, 60, dim, 0, 0)
    w = 1 + 0.1 * normal(9, dim)
    flat = torch.full((2 * dim + 5,), 0.5, device=DEV)
    kept = dy.clone()
    ws = api.workspace(api.layer_norm_backward_workspace_size(60, dim), DEV)
    got = api.layer_norm_backward(dy, c, mean, rstd, w, dx=dy, dweight=flat[1:1 + dim],
                                  dbias=flat[3 + dim:3 + 2 * dim], accumulate=True, ws=ws)
    assert got[0] is dy
    check_norm(kept, c, mean, rstd, w, got, (0.5, 0.5))
    assert float(flat[0]) == float(flat[1 + dim]) == float(flat[2 + dim]) == float(flat[-1]) == 0.5
    got = api.layer_norm_backward(kept, c, mean, rstd, None)
    check_norm(kept, c, mean, rstd, None, got)


def test_norm_gradients_of_no_rows_and_of_nan():
    dy, c, mean, rstd, w = norm_case(torch.float32, 6, 300, 0, 0)
    empty = api.Checkpoint8(c.codes[:0], c.exponents[:0], 300, torch.float32)
    dx, dw, db = api.layer_norm_backward(dy[:0], empty, mean[:0], rstd[:0], w)
    assert dx.shape == (0, 300) and float(dw.abs().sum() + db.abs().sum()) == 0.0
    c.exponents[2, 1] = 255  # a group that was not finite: its row's dx, its columns' dweight
    dx, dw, db = api.layer_norm_backward(dy, c, mean, rstd, w)
    bad = dx.isnan().any(1)
    assert bad.tolist() == [False, False, True, False, False, False]
    assert dw.isnan().nonzero()[:, 0].tolist() == list(range(128, 256))
    assert not bool(db.isnan().any())


def test_the_same_bits_every_time():
    case = norm_case(torch.bfloat16, 3000, 1024, 0, 0)
    first = api.layer_norm_backward(*case)
    for _ in range(3):
        for a, b in zip(first, api.layer_norm_backward(*case)):
            assert torch.equal(a, b)


def test_captured_and_replayed():
    dy, c, mean, rstd, w = norm_case(torch.float16, 50, 264, 0, 0)
    x = api.restore8(c)
    ws = api.workspace(api.layer_norm_backward_workspace_size(50, 264), DEV)
    want = api.layer_norm_backward(dy, c, mean, rstd, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = api.checkpoint8(x)
        back = api.restore8(kept)
        got = api.layer_norm_backward(dy, kept, mean, rstd, w, ws=ws)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(back, x)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    x.mul_(2.0)  # other inputs at the same place
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(back, x) and not torch.equal(got[1], want[1])


def test_a_type_that_the_output_does_not_have():
    c = api.checkpoint8(torch.ones(3, 40, dtype=torch.bfloat16, device=DEV))
    out = torch.zeros(3, 40, device=DEV)
    with pytest.raises(TypeError):
        api.restore8(c, out=out, dtype=torch.bfloat16)
    assert float(out.abs().sum()) == 0.0
    assert api.restore8(c, out=out, dtype=torch.float32) is out and bool((out == 1).all())
