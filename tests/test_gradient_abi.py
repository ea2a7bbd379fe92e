"""Host-side validation of the entry points that make a node's gradient: 8-bit activations, linear
layers of experts, norm and rotation of queries and keys. Nothing here reaches a GPU."""
import pytest

from top_gradient_compression_gb300 import _lib, api

FAKE = 1 << 20  # non-null, aligned, never dereferenced
OK, BAD, WORKSPACE = 0, 1, 2


def caller(f, good):
    """f with some of its good arguments changed, by their places."""
    def call(changes=()):
        a = list(good)
        for i, v in dict(changes).items():
            a[i] = v
        return f(*a)
    return call


def test_checkpoint8_arguments():
    # x, type, x_stride, rows, dim, codes, codes_stride, exponents, exponents_stride, stream
    call = caller(_lib.load().sparcml_checkpoint8,
                  [FAKE, 1, 300, 4, 300, FAKE, 304, FAKE, 3, None])
    for i in (0, 5, 7):
        assert call({i: None}) == BAD
    assert call({1: 3}) == BAD and call({1: -1}) == BAD
    assert call({2: -1}) == BAD and call({3: 1 << 31}) == BAD
    assert call({4: 0}) == BAD and call({4: 1 << 31}) == BAD
    assert call({0: FAKE + 1}) == BAD and call({5: FAKE + 8}) == BAD
    assert call({6: 288}) == BAD and call({6: 308}) == BAD and call({8: 2}) == BAD
    assert call({3: 0}) == OK  # no rows: nothing is enqueued


def test_restore8_arguments():
    # codes, codes_stride, exponents, exponents_stride, rows, dim, y, type, y_stride, stream
    call = caller(_lib.load().sparcml_restore8,
                  [FAKE, 304, FAKE, 3, 4, 300, FAKE, 1, 300, None])
    for i in (0, 2, 6):
        assert call({i: None}) == BAD
    assert call({1: 296}) == BAD and call({3: 2}) == BAD and call({7: 3}) == BAD
    assert call({6: FAKE + 1}) == BAD and call({8: 299}) == BAD
    assert call({4: 0}) == OK


def test_layer_norm_backward8_arguments():
    lib = _lib.load()
    ws = lib.sparcml_layer_norm_backward_workspace_size(1000, 4096)
    # dy, dy_stride, type, codes, codes_stride, exponents, exponents_stride, weight, weight_type,
    # mean, rstd, rows, dim, dx, dx_stride, dweight, dbias, accumulate, ws, ws_bytes, stream
    call = caller(lib.sparcml_layer_norm_backward8,
                  [FAKE, 4096, 1, FAKE, 4096, FAKE, 32, FAKE, 1, FAKE, FAKE, 1000, 4096, FAKE,
                   4096, FAKE, FAKE, 0, FAKE, ws, None])
    for i in (0, 3, 5, 9, 10, 13, 18):
        assert call({i: None}) == BAD
    assert call({2: 3}) == BAD and call({8: 3}) == BAD and call({1: -1}) == BAD
    assert call({4: 4080}) == BAD and call({6: 31}) == BAD and call({14: 4095}) == BAD
    assert call({9: FAKE + 2}) == BAD and call({15: FAKE + 2}) == BAD
    assert call({18: FAKE + 64}) == BAD and call({19: ws - 1}) == WORKSPACE
    assert call({11: 0, 15: None, 16: None}) == OK


def test_expert_linear_workspace():
    size = _lib.load().sparcml_expert_linear_workspace_size
    for bad in ((1 << 31, 1, 8, 8), (4, 0, 8, 8), (4, 1025, 8, 8), (4, 1, 0, 8), (4, 1, 8, 0),
                (4, 1, (1 << 24) + 1, 8), (4, 1, 8, (1 << 24) + 1), (1 << 30, 1, 1 << 24, 1 << 24)):
        assert size(*bad, 1) == 0
    plain = size(1000, 8, 512, 256, 1)
    assert plain % 256 == 0 and plain >= 256 + 1000 * 256 * 2  # x, where it is kept in 8 bits
    # copies of what is not aligned: x and dy, and the matrices
    assert size(1000, 8, 512, 256, 0) >= plain + 1000 * 512 * 2 + 8 * 512 * 256 * 2
    assert size(1000, 8, 511, 256, 1) >= 1000 * (256 + 512) * 2
    assert size(1000, 8, 512, 255, 1) >= 1000 * 256 * 2 + 8 * 512 * 256 * 2
    assert size(0, 4, 8, 8, 1) >= 256


def forward_call():
    lib = _lib.load()
    ws = lib.sparcml_expert_linear_workspace_size(100, 4, 64, 32, 1)
    # x, x_stride, weight, batch, stride, type, offsets, experts, rows, n, k, y, y_stride, ws,
    # ws_bytes, stream
    return caller(lib.sparcml_expert_linear,
                  [FAKE, 32, FAKE, 2048, 32, 1, FAKE, 4, 100, 64, 32, FAKE, 64, FAKE, ws, None]), ws


def test_expert_linear_arguments():
    call, ws = forward_call()
    for i in (0, 2, 6, 11, 13):
        assert call({i: None}) == BAD
    assert call({5: 0}) == BAD and call({5: 3}) == BAD  # the tensor cores have no fp32 product
    assert call({1: -1}) == BAD and call({3: -1}) == BAD and call({4: -1}) == BAD
    assert call({12: 63}) == BAD and call({0: FAKE + 1}) == BAD and call({6: FAKE + 2}) == BAD
    assert call({7: 0}) == BAD and call({7: 1025}) == BAD and call({9: 0}) == BAD
    assert call({13: FAKE + 128}) == BAD and call({14: 200}) == WORKSPACE
    # an operand that has to be copied, and no room for it
    assert call({2: FAKE + 2, 14: 256}) == WORKSPACE
    assert call({8: 0}) == OK  # no rows: nothing is enqueued


@pytest.mark.parametrize("stored", [False, True])
def test_expert_linear_backward_arguments(stored):
    lib = _lib.load()
    ws = lib.sparcml_expert_linear_workspace_size(100, 4, 64, 32, 1)
    x = [FAKE, 32, FAKE, 1] if stored else [FAKE, 32]
    o = len(x) - 2  # how far the arguments behind x have moved
    f = lib.sparcml_expert_linear_backward8 if stored else lib.sparcml_expert_linear_backward
    # dy, dy_stride, x..., weight, batch, stride, type, offsets, experts, rows, n, k, dx, dx_stride,
    # dweight, batch, stride, accumulate, ws, ws_bytes, stream
    call = caller(f, [FAKE, 64, *x, FAKE, 2048, 32, 1, FAKE, 4, 100, 64, 32, FAKE, 32, FAKE, 2048,
                      32, 0, FAKE, ws, None])
    for i in (0, 2, 4 + o, 8 + o, 19 + o):
        assert call({i: None}) == BAD
    if stored:
        assert call({4: None}) == BAD and call({2: FAKE + 8}) == BAD
        assert call({3: 16}) == BAD and call({5: 0}) == BAD
    assert call({7 + o: 0}) == BAD and call({14 + o: 31}) == BAD
    # dW's rows or matrices over one another
    assert call({17 + o: 31}) == BAD and call({16 + o: 2047}) == BAD and call({16 + o: 31}) == BAD
    assert call({15 + o: FAKE + 2}) == BAD
    assert call({20 + o: 255}) == WORKSPACE and call({19 + o: FAKE + 4}) == BAD
    assert call({13 + o: None, 15 + o: None}) == OK  # neither is wanted
    assert call({13 + o: None, 15 + o: None, 2: None, 4 + o: None}) == OK
    assert call({10 + o: 0, 15 + o: None}) == OK


def test_head_norm_rotary_arguments():
    lib = _lib.load()
    # q, token, head, heads, k, token, head, heads, type, tokens, dim, positions, int64, freqs,
    # turned, interleaved, q_weight, k_weight, weight_type, eps, q_out, t, h, k_out, t, h, stream
    good = [FAKE, 512, 64, 8, FAKE, 128, 64, 2, 1, 10, 64, FAKE, 0, FAKE, 64, 0, FAKE, FAKE, 1, 1e-6,
            FAKE, 512, 64, FAKE, 128, 64, None]
    call = caller(lib.sparcml_head_norm_rotary, good)
    for i in (0, 4, 11, 13, 20, 23):
        assert call({i: None}) == BAD
    assert call({8: 3}) == BAD and call({18: 3}) == BAD and call({19: -1.0}) == BAD
    assert call({19: float("nan")}) == BAD and call({9: 1 << 31}) == BAD
    assert call({10: 0}) == BAD and call({10: 513}) == BAD
    assert call({14: 66}) == BAD and call({14: 63}) == BAD
    assert call({1: -1}) == BAD and call({6: -1}) == BAD and call({3: 65536}) == BAD
    assert call({0: FAKE + 1}) == BAD and call({16: FAKE + 1}) == BAD and call({11: FAKE + 2}) == BAD
    assert call({11: FAKE + 4, 12: 1}) == BAD
    # results over one another
    assert call({21: 511}) == BAD and call({22: 63}) == BAD and call({24: -1}) == BAD
    assert call({9: 0}) == OK
    assert call({3: 0, 7: 0, 0: None, 4: None, 20: None, 23: None}) == OK  # no heads at all

    size = lib.sparcml_head_norm_rotary_backward_workspace_size
    assert size(10, 8, 2, 0) == 0 and size(10, 8, 2, 513) == 0 and size(1 << 31, 8, 2, 64) == 0
    ws = size(10, 8, 2, 64)
    assert 256 < ws and ws % 256 == 0 and size(16384, 32, 8, 512) < 4 << 20
    # dq, token, head, dk, token, head, then as above up to eps and the outputs, q_dweight,
    # k_dweight, accumulate, ws, ws_bytes, stream
    call = caller(lib.sparcml_head_norm_rotary_backward,
                  [FAKE, 512, 64, FAKE, 128, 64, *good[:26], FAKE, FAKE, 0, FAKE, ws, None])
    for i in (0, 3, 6, 10, 17, 19, 26, 29, 35):
        assert call({i: None}) == BAD
    assert call({1: -1}) == BAD and call({32: FAKE + 2}) == BAD and call({33: FAKE + 2}) == BAD
    assert call({35: FAKE + 128}) == BAD and call({36: ws - 1}) == WORKSPACE
    assert call({15: 0, 32: None, 33: None}) == OK


def test_group_size_is_the_headers():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "sparcml.h")).read()
    assert int(re.search(r"#define SPARCML_GROUP8 (\d+)", text)[1]) == api.GROUP8
