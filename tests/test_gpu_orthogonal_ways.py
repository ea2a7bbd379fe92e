"""Every way through the orthogonalisation's products (training_cases.WAYS: tiles on one SM and
on a pair, of every width, halves of tiles, split and joined sums, one chain and two, wide and
tall) against the formula in 64 bits, on the GPU.

Tolerances: test_gpu_orthogonal.py derives 5e-3 of the result in the Frobenius norm from 32 rows
on, of which the bf16 output's rounding is 1.6e-3. The results here are read through fp32 weights
that start at zero and move by one, so 3.4e-3 is left for them. One tile of 64 x 64 that is
wrong in the largest matrix here would be 1.6e-2 of it.
"""
import pytest
import torch

from top_gradient_compression_gb300 import api

from gpu_helpers import DEV
from test_gpu_orthogonal import gradient
from training_cases import WAYS

pytestmark = pytest.mark.gpu

ROUNDING = 3.4e-3


def reference(g, coeffs=api.NEWTON_SCHULZ):
    """In 64 bits, as q(S) X with q the product of the steps' a + b S + c S^2."""
    x = g.double()
    if x.shape[-2] > x.shape[-1]:
        return reference(g.transpose(-1, -2), coeffs).transpose(-1, -2)
    x = x / torch.linalg.vector_norm(x, dim=(-2, -1), keepdim=True)
    s = x @ x.transpose(-1, -2)
    eye = torch.eye(s.shape[-1], dtype=s.dtype, device=s.device)
    q = eye
    for a, b, c in coeffs:
        p = a * eye + b * s + c * (s @ s)
        q, s = p @ q, p @ s @ p
    return q @ x


def near(out, ref, tol=ROUNDING):
    off = (out.double() - ref).flatten(-2).norm(dim=-1) / ref.flatten(-2).norm(dim=-1)
    assert float(off.max()) <= tol, off


def orthogonal(g, ws):
    """The result in fp32."""
    w = torch.zeros(g.shape, device=DEV)
    api.muon_step(w, g, torch.zeros(g.shape, device=DEV), lr=1.0, mu=0.0, scale=1.0, ws=ws)
    return -w


@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("size", WAYS, ids=lambda s: "x".join(map(str, s)))
def test_every_way(size, tall):
    batch, m, n = size
    if tall:
        m, n = n, m
    g = gradient((batch, m, n), m + n)
    ws = api.workspace(api.orthogonalize_workspace_size(batch, m, n), DEV)
    first = orthogonal(g, ws)
    assert api.get_status(ws) == 0
    near(first, reference(g))
    assert torch.equal(orthogonal(g, ws), first)  # the same workspace, and bits
    # an output of 16 bits is the same result, rounded once
    out = api.orthogonalize(g, out_dtype=torch.float16, ws=ws)
    assert api.get_status(ws) == 0
    assert torch.equal(out, first.half())


@pytest.mark.parametrize("size", [(8, 400, 400), (2, 100, 9000), (2, 4700, 700)])
def test_zero_nan_and_strides(size):
    """Pairs of SMs and joined sums: what is wrong with one matrix stays in it; rows at an odd
    offset of a flat vector, results into a wider array."""
    batch, m, n = size
    gap = 37
    flat = torch.zeros(3 + batch * (m * n + gap), device=DEV)
    g = flat[3:].as_strided((batch, m, n), (m * n + gap, n, 1))
    g.copy_(gradient((batch, m, n), 4))
    g[1] = 0
    wide = torch.full((batch, m + 2, n + 5), 9.0, device=DEV, dtype=torch.float16)
    out = wide[:, 1:m + 1, 3:n + 3]
    api.orthogonalize(g, out=out)
    near(out[0], reference(g[0]))
    assert (out[1] == 0).all()
    good = out.clone()
    edge = wide.clone()
    edge[:, 1:m + 1, 3:n + 3] = 9.0
    assert (edge == 9).all()
    g[1, m - 1, n - 1] = float("nan")
    api.orthogonalize(g, out=out)
    assert out[1].isnan().all()
    assert all(torch.equal(out[b], good[b]) for b in range(batch) if b != 1)


@pytest.mark.parametrize("size,wt,nesterov", [((8, 400, 400), torch.bfloat16, True),
                                              ((1, 2111, 2049), torch.float32, False),
                                              ((1, 300, 9000), torch.float16, True)])
def test_weight_step(size, wt, nesterov):
    batch, m, n = size
    gen = torch.Generator(device=DEV).manual_seed(7)
    w = torch.randn(batch, m, n, generator=gen, device=DEV).to(wt)
    mom, g = gradient(size, 8), gradient(size, 9, torch.bfloat16)
    scale = 0.2 * max(m, n) ** 0.5
    rm = 0.9 * mom.double() + g.double()
    move = -0.02 * scale * reference(g.double() + 0.9 * rm if nesterov else rm)
    kept = w.double() * (1 - 0.02 * 0.1)
    before = w.double()
    ws = api.workspace(api.orthogonalize_workspace_size(batch, m, n), DEV)
    api.muon_step(w, g, mom, lr=0.02, mu=0.9, nesterov=nesterov, weight_decay=0.1, scale=scale,
                  ws=ws)
    assert api.get_status(ws) == 0
    assert ((mom.double() - rm).abs() <= 2.0 ** -22 * (mom.abs() + g.float().abs()).double()).all()
    u = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[wt]
    slack = u * (kept + move).abs() + 3 * 2.0 ** -24 * before.abs()
    left = ((w.double() - kept - move).abs() - slack).clamp_min(0)
    assert float(left.norm() / move.norm()) <= ROUNDING
