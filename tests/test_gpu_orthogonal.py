"""Newton-Schulz orthogonalisation and the weight step built on it, against the
formulas in 64 bits, on the GPU.

Tolerances. The products take fp16 operands (unit roundoff u = 2^-11) with fp32
accumulators. In one step a singular value s is off by at most
(u |P| + u |b + 2 c s^2| s^2 + u |P|) s with |P| <= 2.9 and |b + 2 c s^2| s^2 <= 4.8,
relative to a result of at least 0.7 s: 15 u = 7e-3, and later steps multiply an
error by at most about 1. So one singular value alone, as in a matrix of a few
rows, may come out 3e-2 off at worst. Over a matrix the roundings are
independent: their root mean square is u / sqrt(3) or less each, and a
simulation of the roundings on the CPU gives 0.2e-3 to 1.8e-3 in the Frobenius
norm over flat, 1/i, 1/sqrt(i) and 1/i^2 spectra. The bf16 output adds
2^-8 / sqrt(3) / 1.4 = 1.6e-3. So 5e-3 is asked from 32 rows on.
"""
import pytest
import torch

from top_gradient_compression_gb300 import api

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

COEFFS = api.NEWTON_SCHULZ
# larger first steps, as sets that are fitted step by step have them
FITTED = ((8.2872, -23.5959, 17.3004), (4.1071, -2.9478, 0.5448), (3.9487, -2.9089, 0.5518),
          (3.3184, -2.4885, 0.5100), (2.3006, -1.6689, 0.4188))


def gradient(shape, seed, dtype=torch.float32, size=1e-3, power=0.5):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    *lead, m, n = shape
    r = min(m, n)
    decay = torch.arange(1, r + 1, device=DEV, dtype=torch.float32).pow(-power)
    left = torch.randn(*lead, m, r, generator=gen, device=DEV)
    right = torch.randn(*lead, r, n, generator=gen, device=DEV)
    return ((left * decay) @ right * size).to(dtype)


def reference(g, coeffs=COEFFS):
    """X <- a X + b (X X') X + c (X X')^2 X in 64 bits."""
    x = g.double()
    if x.shape[-2] > x.shape[-1]:
        return reference(g.transpose(-1, -2), coeffs).transpose(-1, -2)
    norm = torch.linalg.vector_norm(x, dim=(-2, -1), keepdim=True)
    x = torch.where(norm > 0, x / torch.where(norm > 0, norm, 1.0), 0.0)
    for a, b, c in coeffs:
        s = x @ x.transpose(-1, -2)
        x = a * x + b * (s @ x) + c * (s @ (s @ x))
    return x


def check(out, ref):
    out, ref = out.double(), ref.double()
    k = min(ref.shape[-2:])
    rel = (out - ref).norm() / ref.norm().clamp_min(1e-300)
    assert rel <= (5e-3 if k >= 32 else 3e-2), float(rel)
    rms = ref.square().mean().sqrt()
    worst = ((out - ref).abs() - 2.0 ** -7 * ref.abs()).max() / rms.clamp_min(1e-300)
    assert worst <= (0.04 if k >= 32 else 0.3), float(worst)


def check_small(out, ref, noise):
    """A side of at most 64: X is read in three products of its halves and the steps are
    fp32, so what is left beside the output's rounding is fp32's own in S, 2^-24, times
    what the steps multiply a small singular value by."""
    out, ref = out.double(), ref.double()
    assert (out - ref).norm() <= noise * ref.norm()


@pytest.mark.parametrize("power", [0.0, 0.5, 2.0, 4.0])
@pytest.mark.parametrize("m,n", [(16, 16), (17, 900), (33, 64), (64, 64), (64, 5000), (4100, 48),
                                 (20_000, 63)])
def test_small_sides(m, n, power):
    """An update in fp32, so that the result's error can be seen: 1e-3 of it at most (the
    simulated roundings give up to 8e-4, for the 1/i^4 spectrum)."""
    gen = torch.Generator(device=DEV).manual_seed(m + n)
    k = min(m, n)
    u, _ = torch.linalg.qr(torch.randn(m, k, generator=gen, device=DEV))
    v, _ = torch.linalg.qr(torch.randn(n, k, generator=gen, device=DEV))
    g = (u * torch.arange(1, k + 1, device=DEV).float().pow(-power)) @ v.t()
    for coeffs, noise in ((COEFFS, 2e-3), (FITTED, 3e-2), (((1.5, -0.5, 0.0),) * 12, 2e-3)):
        w, mom = torch.zeros(m, n, device=DEV), torch.zeros(m, n, device=DEV)
        ws = api.workspace(api.orthogonalize_workspace_size(1, m, n), DEV)
        api.muon_step(w, g, mom, lr=1.0, mu=0.0, scale=1.0, coeffs=coeffs, ws=ws)
        assert api.get_status(ws) == 0
        check_small(-w, reference(g, coeffs), noise)


def test_many_small_matrices():
    """More matrices than blocks, both chains, tall and wide."""
    for m, n in ((24, 40), (70, 33), (64, 64)):
        g = gradient((333, m, n), m)
        out = api.orthogonalize(g, out_dtype=torch.float16)
        ref = reference(g)
        rel = (out.double() - ref).flatten(1).norm(dim=1) / ref.flatten(1).norm(dim=1)
        assert float(rel.max()) <= 1e-3  # fp16's own rounding: 2^-11 / sqrt(3) / 1.4
        assert torch.equal(out[200], api.orthogonalize(g[200], out_dtype=torch.float16))


SHAPES = [(1, 1), (1, 7), (7, 1), (2, 3), (16, 16), (64, 64), (65, 63), (128, 128), (129, 127),
          (100, 1000), (1000, 100), (1, 5000), (257, 384), (333, 1000), (1000, 333), (512, 512),
          (640, 200), (1023, 1025), (40, 20_001)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n", SHAPES)
def test_orthogonalize(m, n, dtype):
    g = gradient((m, n), 1000 * m + n, dtype, 1.0 if dtype == torch.float16 else 1e-3)
    ws = api.workspace(api.orthogonalize_workspace_size(1, m, n), DEV)
    out = api.orthogonalize(g, ws=ws)
    assert api.get_status(ws) == 0
    assert out.dtype == torch.bfloat16
    check(out, reference(g))


@pytest.mark.parametrize("power", [0.0, 1.0, 2.0])
@pytest.mark.parametrize("m,n", [(384, 384), (256, 1024), (900, 300)])
def test_spectra(m, n, power):
    """A 1/i^2 spectrum leaves small singular values that the steps multiply 400 times."""
    gen = torch.Generator(device=DEV).manual_seed(m)
    k = min(m, n)
    u, _ = torch.linalg.qr(torch.randn(m, k, generator=gen, device=DEV))
    v, _ = torch.linalg.qr(torch.randn(n, k, generator=gen, device=DEV))
    g = (u * torch.arange(1, k + 1, device=DEV).float().pow(-power)) @ v.t()
    check(api.orthogonalize(g, out_dtype=torch.float16), reference(g))


@pytest.mark.parametrize("m,n", [(96, 200), (200, 96), (130, 130)])
def test_batches_strides_and_offsets(m, n):
    """Matrices that lie apart in a flat vector, at an odd offset, and a wider output."""
    batch, gap = 5, 37
    flat = torch.zeros(3 + batch * (m * n + gap), device=DEV)
    g = flat[3:].as_strided((batch, m, n), (m * n + gap, n, 1))
    g.copy_(gradient((batch, m, n), 4))
    wide = torch.full((batch, m + 2, n + 5), 9.0, device=DEV, dtype=torch.bfloat16)
    out = api.orthogonalize(g, out=wide[:, 1:m + 1, 3:n + 3])
    for b in range(batch):
        check(out[b], reference(g[b]))
    edge = wide.clone()
    edge[:, 1:m + 1, 3:n + 3] = 9.0
    assert (edge == 9).all()
    one = api.orthogonalize(g[2])
    assert torch.equal(one, out[2])
    turns = torch.empty(m, batch, n, device=DEV, dtype=torch.bfloat16).transpose(0, 1)
    assert torch.equal(api.orthogonalize(g, out=turns), out)


def test_size_does_not_matter_to_a_power_of_two():
    """|G| far outside the range in which squares of fp32 exist."""
    g = gradient((160, 96), 2, size=1.0)
    first = api.orthogonalize(g)
    for p in (2.0 ** -100, 2.0 ** -30, 2.0 ** 60, 2.0 ** 100):
        assert torch.equal(api.orthogonalize(g * p), first)
    tiny = torch.zeros(40, 50, device=DEV)
    tiny[3, 4] = 1e-44  # a subnormal
    out = api.orthogonalize(tiny)
    check(out, reference(tiny))


def test_zero_nan_and_inf_stay_in_their_matrix():
    g = gradient((4, 70, 90), 3)
    g[1] = 0
    g[2, 5, 6] = float("nan")
    g[3, 0, 0] = float("inf")
    out = api.orthogonalize(g)
    check(out[0], reference(g[0]))
    assert (out[1] == 0).all() and out[2].isnan().all() and out[3].isnan().all()


@pytest.mark.parametrize("coeffs", [FITTED, COEFFS[:1], ((1.5, -0.5, 0.0),) * 12])
def test_other_steps(coeffs):
    g = gradient((192, 320), 6, power=0.3)
    check(api.orthogonalize(g, coeffs), reference(g, coeffs))


def muon_reference(w, g, mom, lr, mu, nesterov, decay, scale, coeffs=COEFFS):
    w, g, mom = w.double(), g.double(), mom.double()
    mom = mu * mom + g
    u = g + mu * mom if nesterov else mom
    return w * (1 - lr * decay) - lr * scale * reference(u, coeffs), mom


@pytest.mark.parametrize("wt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("gt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n,nesterov", [(256, 256, True), (100, 333, False), (333, 100, True),
                                          (1, 64, True)])
def test_muon_step(m, n, nesterov, wt, gt):
    gen = torch.Generator(device=DEV).manual_seed(7)
    w = torch.randn(2, m, n, generator=gen, device=DEV).to(wt)
    mom = gradient((2, m, n), 8)
    g = gradient((2, m, n), 9, gt)
    scale = 0.2 * max(m, n) ** 0.5
    rw, rm = muon_reference(w, g, mom, 0.02, 0.9, nesterov, 0.1, scale)
    before = w.double()
    ws = api.workspace(api.orthogonalize_workspace_size(2, m, n), DEV)
    api.muon_step(w, g, mom, lr=0.02, mu=0.9, nesterov=nesterov, weight_decay=0.1, scale=scale,
                  ws=ws)
    assert api.get_status(ws) == 0
    assert ((mom.double() - rm).abs() <= 2.0 ** -22 * (mom.abs() + g.float().abs()).double()).all()
    u = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[wt]
    move = rw - before * (1 - 0.02 * 0.1)
    slack = u * rw.abs() + 3 * 2.0 ** -24 * before.abs()
    left = ((w.double() - rw).abs() - slack).clamp_min(0)
    k = min(m, n)
    assert left.norm() / move.norm() <= (5e-3 if k >= 32 else 3e-2)
    if wt == torch.float32:
        check((w.double() - before * (1 - 0.02 * 0.1)) / (-0.02 * scale),
              move / (-0.02 * scale))


def test_muon_step_on_a_slice_of_the_reduced_vector():
    """The path's own data: a dense reduced vector at an odd offset, two steps, and a
    default scale; the matrix form and the batch form agree."""
    n_all = 3 + 96 * 64 + 50
    reduced = torch.randn(n_all, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    g = reduced[3:3 + 96 * 64].view(96, 64)
    w = torch.randn(96, 64, device=DEV, generator=torch.Generator(device=DEV).manual_seed(2))
    mom = torch.zeros(96, 64, device=DEV)
    w2, mom2 = w.clone()[None], mom.clone()[None]
    rw, rm = w, mom
    for _ in range(2):
        rw, rm = muon_reference(rw, g, rm, 0.1, 0.95, True, 0.0, 1.5 ** 0.5)
        api.muon_step(w, g, mom, lr=0.1)
        api.muon_step(w2, g[None], mom2, lr=0.1)
    assert torch.equal(w, w2[0]) and torch.equal(mom, mom2[0])
    start = torch.randn(96, 64, device=DEV, generator=torch.Generator(device=DEV).manual_seed(2))
    check(w.double() - start.double(), rw - start.double())


def test_the_same_bits_again_and_on_another_stream():
    g = gradient((3, 300, 500), 12)
    first = api.orthogonalize(g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = [api.orthogonalize(g) for _ in range(3)]
    side.synchronize()
    for t in again:
        assert torch.equal(first, t)


def test_nothing_to_do_and_refusals():
    g = gradient((64, 80), 1)
    assert api.orthogonalize(g[None][:0]).shape == (0, 64, 80)
    with pytest.raises(TypeError):
        api.orthogonalize(g.double())
    with pytest.raises(TypeError):
        api.orthogonalize(g, out_dtype=torch.float32)
    with pytest.raises(ValueError):
        api.orthogonalize(g.t())
    with pytest.raises(ValueError):
        api.orthogonalize(g[0])
    with pytest.raises(ValueError):
        api.orthogonalize(g, coeffs=(1.5, -0.5, 0.0))
    with pytest.raises(api.SparcmlError):
        api.orthogonalize(g, coeffs=((float("nan"), 0.0, 0.0),))
    with pytest.raises(api.SparcmlError):
        api.orthogonalize(g, ws=api.workspace(1024, DEV))
    with pytest.raises(ValueError):
        api.orthogonalize(g[None], out=torch.zeros(64, 80, device=DEV, dtype=torch.bfloat16))
    overlap = torch.zeros(65, 80, device=DEV).as_strided((2, 64, 80), (80, 80, 1))
    mom = torch.zeros(2, 64, 80, device=DEV)
    with pytest.raises(api.SparcmlError):
        api.muon_step(overlap, mom, mom.clone(), lr=0.1)
    with pytest.raises(TypeError):
        api.muon_step(mom.clone(), mom.clone(), mom.half(), lr=0.1)
    with pytest.raises(api.SparcmlError):
        api.muon_step(mom.clone(), mom.clone(), mom, lr=float("inf"))
