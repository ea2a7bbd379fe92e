"""Host-side validation of the entry points that make a node's gradient: 8-bit activations, linear
layers of experts, norm and rotation of queries and keys. Nothing here reaches a GPU."""
import os
import re

import pytest

from top_gradient_compression_gb300 import _lib, api

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sparcml.h")
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


HEADS = dict(q=FAKE, q_token_stride=512, q_head_stride=64, q_heads=8, k=FAKE, k_token_stride=128,
             k_head_stride=64, k_heads=2, type=1, tokens=10, dim=64, positions=FAKE,
             positions_int64=0, freqs=FAKE, turned=64, interleaved=0, q_weight=FAKE, k_weight=FAKE,
             weight_type=1, eps=1e-6, q_out=FAKE, q_out_token_stride=512, q_out_head_stride=64,
             k_out=FAKE, k_out_token_stride=128, k_out_head_stride=64, dq=FAKE,
             dq_token_stride=512, dq_head_stride=64, dk=FAKE, dk_token_stride=128,
             dk_head_stride=64, q_dweight=FAKE, k_dweight=FAKE, accumulate=0, ws=FAKE)


def test_head_args_are_the_headers():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    members = re.search(r"struct sparcml_head_args \{(.*?)\};", text, re.S)[1]
    names = [re.sub(r".*[ *]", "", m.strip()) for m in re.split(r"[;,]", members) if m.strip()]
    assert names == _lib.HEAD_ARGS
    kinds = {m.strip().split()[0] if "*" not in m else "pointer"
             for m in members.split(";") if m.strip()}
    assert kinds == {"pointer", "int64_t", "double"}


@pytest.mark.parametrize("back", [False, True])
def test_head_norm_rotary_arguments(back):
    lib = _lib.load()
    size = lib.sparcml_head_norm_rotary_backward_workspace_size
    assert size(10, 8, 2, 0) == 0 and size(10, 8, 2, 513) == 0 and size(1 << 31, 8, 2, 64) == 0
    ws = size(10, 8, 2, 64)
    assert 256 < ws and ws % 256 == 0 and size(16384, 32, 8, 512) < 4 << 20
    f = lib.sparcml_head_norm_rotary_backward if back else lib.sparcml_head_norm_rotary

    def call(**change):
        args = {**HEADS, "ws_bytes": ws, **change}
        return f(_lib.pack_head_args(*(args[m] for m in _lib.HEAD_ARGS)), None)
    assert f(None, None) == BAD
    for name in ("q", "k", "positions", "freqs", "q_out", "k_out") + \
            (("dq", "dk", "ws") if back else ()):
        assert call(**{name: 0}) == BAD, name
    for name in ("q_token_stride", "q_head_stride", "k_token_stride", "k_head_stride") + \
            (("dq_token_stride", "dk_head_stride") if back else ()):
        assert call(**{name: -1}) == BAD, name
    for name, bad in (("type", 3), ("type", -1), ("type", 1 << 32), ("weight_type", 3),
                      ("eps", -1.0), ("eps", float("nan")), ("tokens", 1 << 31), ("tokens", -1),
                      ("dim", 0), ("dim", 513), ("dim", (1 << 32) + 64), ("turned", 66),
                      ("turned", 63), ("turned", -2), ("q_heads", 65536), ("k_heads", -1),
                      ("q", FAKE + 1), ("q_weight", FAKE + 1), ("positions", FAKE + 2),
                      # results over one another
                      ("q_out_token_stride", 511), ("q_out_head_stride", 63),
                      ("k_out_token_stride", -1)):
        assert call(**{name: bad}) == BAD, (name, bad)
    assert call(positions=FAKE + 4, positions_int64=1) == BAD
    none = dict(q_heads=0, k_heads=0, q=0, k=0, q_out=0, k_out=0, q_dweight=0, k_dweight=0)
    assert call(tokens=0, q_dweight=0, k_dweight=0) == OK and call(**none) == OK
    if back:
        assert call(q_dweight=FAKE + 2) == BAD and call(ws=FAKE + 128) == BAD
        assert call(ws_bytes=ws - 1) == WORKSPACE and call(ws_bytes=-1) == WORKSPACE


def test_group_size_is_the_headers():
    text = open(HEADER).read()
    assert int(re.search(r"#define SPARCML_GROUP8 (\d+)", text)[1]) == api.GROUP8
