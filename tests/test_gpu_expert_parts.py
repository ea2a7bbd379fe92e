"""Weight gradients of more experts than are sorted by their rows: the tiles that no whole round of
the pairs is left for are taken in parts by the deepest of them, wherever it stands."""
import pytest
import torch

from top_gradient_compression_gb300 import api

from test_gpu_experts import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("last", [[1, 0, 3, 16384], [0, 16384, 64, 1], [16384, 5, 0, 0]])
def test_the_deepest_of_the_rest_is_taken_in_parts(last):
    """308 tiles on 76 pairs leave 4, which are summed as they are alone: the same parts in the same
    order give the same bits."""
    few = Case(torch.bfloat16, last, 64, 64)
    alone = api.expert_linear_backward(few.dy, few.x, few.w, few.offsets, need_dx=False)[1]
    few.check(dw=alone)
    more = 4 * 76
    c = Case(torch.bfloat16, [1] * more + last, 64, 64)
    c.x[more:], c.dy[more:], c.w[more:] = few.x, few.dy, few.w
    dw = api.expert_linear_backward(c.dy, c.x, c.w, c.offsets, need_dx=False)[1]
    c.check(dw=dw)
    assert torch.equal(dw[more:], alone)
