"""Experts' linear layers with many more tiles than pairs of SMs, which are handed out one by one:
each has to be done once, by all warps of a pair, and the workspace's count has to be back at zero
for the next call."""
import pytest
import torch

from top_gradient_compression_gb300 import api

from test_gpu_experts import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes,n,k", [([1] * 900, 40, 24), ([64, 0, 65, 1] * 60, 264, 520),
                                       ([300] * 20, 520, 513)], ids=["tiny", "short", "many"])
def test_short_tiles_one_after_the_other(sizes, n, k):
    """900 tiles of one block each and the like, so that the words that tell pairs their next tile
    follow one another as fast as they can."""
    c = Case(torch.bfloat16, sizes, n, k)
    ws = api.workspace(api.expert_linear_workspace_size(c.rows, len(sizes), n, k), c.x.device)
    kept = api.checkpoint8(c.x)
    c.x = api.restore8(kept)
    want = c.want()
    first = None
    for turn in range(20):
        y = api.expert_linear(c.x, c.w, c.offsets, ws=ws)
        got = y, *api.expert_linear_backward(c.dy, kept if turn % 2 else c.x, c.w, c.offsets, ws=ws)
        if first is None:
            first = got
            c.check(*got, want=want)
        assert all(torch.equal(a, b) for a, b in zip(first, got))
        assert int(ws[48:52].view(torch.int32)) == 0
    assert api.get_status(ws) == 0


@pytest.mark.parametrize("n,k", [(520, 520), (264, 2304)])
def test_tiles_that_are_handed_out_after_a_wait_ran_out(n, k):
    """With a fault injected the first pair withholds its products while there are tiles to hand out:
    it draws the rest without doing them, the call says so, and the workspace's count is at zero
    again, so that the next call leaves no tile out."""
    c = Case(torch.bfloat16, [300] * 20, n, k)
    ws = api.workspace(api.expert_linear_workspace_size(c.rows, 20, n, k), c.x.device)
    kept = api.checkpoint8(c.x)
    c.x = api.restore8(kept)

    def back(x, **which):
        return api.expert_linear_backward(c.dy, x, c.w, c.offsets, ws=ws, **which)
    calls = [lambda: (api.expert_linear(c.x, c.w, c.offsets, ws=ws),)]
    for x in (c.x, kept):
        calls += [lambda x=x: back(x), lambda x=x: back(x, need_dweight=False)[:1],
                  lambda x=x: back(x, need_dx=False)[1:]]
    want = [call() for call in calls]
    assert api.get_status(ws) == 0
    for call, right in zip(calls, want):
        api.set_fault_injection(ws, api.INJECT_WITHHOLD_FIRST)
        call()
        assert api.STATUS[api.get_status(ws)] == "SPARCML_ERR_TIMEOUT"
        assert int(ws[48:52].view(torch.int32)) == 0
        api.set_fault_injection(ws, 0)
        for a, b in zip(call(), right):
            assert torch.equal(a, b)
        assert api.get_status(ws) == 0
    c.check(want[0][0], *want[1])
