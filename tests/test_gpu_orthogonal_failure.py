"""Waits of the orthogonalisation that run out, without a GPU fault: the workspace's injection
word has the first block withhold a product, every wait for it gives up within milliseconds, the
call returns with SPARCML_ERR_TIMEOUT in its status word, and the next call on the same workspace
is right."""
import time

import pytest
import torch

from top_gradient_compression_gb300 import api

from gpu_helpers import DEV
from test_gpu_orthogonal import gradient

pytestmark = pytest.mark.gpu

TIMEOUT = api.STATUS_CODE["SPARCML_ERR_TIMEOUT"]


def times_out_and_recovers(batch, m, n):
    g = gradient((batch, m, n), 3)
    want = api.orthogonalize(g)
    ws = api.workspace(api.orthogonalize_workspace_size(batch, m, n), DEV)
    for _ in range(2):
        api.set_fault_injection(ws, api.INJECT_WITHHOLD_FIRST)
        torch.cuda.synchronize()
        start = time.perf_counter()
        api.orthogonalize(g, ws=ws)
        assert api.get_status(ws) == TIMEOUT
        assert time.perf_counter() - start < 1.0
        api.set_fault_injection(ws, 0)
        out = api.orthogonalize(g, ws=ws)
        assert api.get_status(ws) == 0
        assert torch.equal(out, want)


# one SM per tile: few tiles and many, a split sum, two chains; then pairs of SMs
@pytest.mark.parametrize("batch,m,n", [(1, 100, 100), (1, 700, 900), (1, 300, 9000),
                                       (2, 100, 9000), (8, 400, 513), (1, 1300, 1300),
                                       (1, 4700, 777), (8, 400, 400), (1, 2049, 2111)])
def test_a_withheld_product(batch, m, n):
    times_out_and_recovers(batch, m, n)


# one matrix, more matrices than blocks, two chains whose solves and products alternate
@pytest.mark.parametrize("batch,m,n", [(1, 48, 300), (1, 64, 16384), (1, 20_001, 40),
                                       (2, 64, 9000), (7, 33, 2000), (333, 24, 40)])
def test_a_withheld_product_of_a_small_side(batch, m, n):
    times_out_and_recovers(batch, m, n)


def test_a_weight_step_and_a_fresh_workspace():
    g, w, mom = (gradient((200, 300), s) for s in (1, 2, 3))
    size = api.orthogonalize_workspace_size(1, 200, 300)
    armed, clean = api.workspace(size, DEV), api.workspace(size, DEV)
    api.set_fault_injection(armed, api.INJECT_WITHHOLD_FIRST)
    api.muon_step(w.clone(), g, mom.clone(), lr=0.1, ws=armed)
    assert api.get_status(armed) == TIMEOUT
    api.muon_step(w, g, mom, lr=0.1, ws=clean)
    assert api.get_status(clean) == 0 and w.isfinite().all()
