"""A weight gradient over more rows than the waits' limit alone would allow for: a tile of 2^24 blocks
of 64 rows takes 4 seconds, and the warps that wait for its end or for the next one go on waiting."""
import pytest
import torch

from top_gradient_compression_gb300 import api

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

EXPERTS, SIDE = 76, 8  # as many tiles as pairs of SMs, so that none is taken in parts


def test_a_tile_that_takes_seconds():
    rows = 2 ** 30
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 36 GB")
    x, dy = (torch.ones(rows, SIDE, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    w = torch.zeros(EXPERTS, SIDE, SIDE, dtype=torch.bfloat16, device=DEV)
    off = torch.arange(EXPERTS + 1, dtype=torch.int32, device=DEV) + (rows - EXPERTS)
    off[0] = 0
    ws = api.workspace(64 << 20, DEV)  # no operand is copied
    _, dw = api.expert_linear_backward(dy, x, w, off, need_dx=False, ws=ws)
    assert api.get_status(ws) == 0
    # whole numbers, of which each sum of 512 is exact, and the last one rounded
    assert bool((dw[0] == float(rows - EXPERTS + 1)).all()) and bool((dw[1:] == 1.0).all())
