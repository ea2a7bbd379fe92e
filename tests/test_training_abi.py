"""Host-side validation of the training-step entry points: nothing here reaches a GPU."""
import numpy as np
import pytest

from top_gradient_compression_gb300 import _lib, api

FAKE = 1 << 20  # non-null, aligned, never dereferenced
BAD, WORKSPACE = 1, 2


def test_layer_norm_arguments():
    f = _lib.load().sparcml_layer_norm
    good = [FAKE, 0, 16, FAKE, FAKE, 0, 4, 16, 1e-5, FAKE, 16, FAKE, FAKE, None]

    def call(**change):
        a = list(good)
        for i, v in change.items():
            a[int(i[1:])] = v
        return f(*a)
    assert call(_0=None) == BAD and call(_9=None) == BAD and call(_11=None) == BAD
    assert call(_12=None) == BAD
    assert call(_1=3) == BAD and call(_5=-1) == BAD
    assert call(_2=-1) == BAD and call(_10=15) == BAD
    assert call(_7=0) == BAD and call(_6=1 << 31) == BAD and call(_7=1 << 31) == BAD
    assert call(_8=-1.0) == BAD and call(_8=float("nan")) == BAD
    assert call(_0=FAKE + 2) == BAD and call(_3=FAKE + 1) == BAD
    assert call(_6=0) == 0  # no rows: nothing is enqueued


def test_layer_norm_backward_arguments():
    lib = _lib.load()
    size = lib.sparcml_layer_norm_backward_workspace_size
    assert size(4, 0) == 0 and size(1 << 31, 4) == 0
    ws = size(1000, 4096)
    assert 2 * 4 * 4096 < ws < 64 << 20
    f = lib.sparcml_layer_norm_backward
    good = [FAKE, 4096, FAKE, 4096, 1, FAKE, 0, FAKE, FAKE, 1000, 4096, FAKE, 4096, FAKE, FAKE, 0,
            FAKE, ws, None]

    def call(**change):
        a = list(good)
        for i, v in change.items():
            a[int(i[1:])] = v
        return f(*a)
    for i in (0, 2, 7, 8, 11, 16):
        assert call(**{f"_{i}": None}) == BAD
    assert call(_4=7) == BAD and call(_6=7) == BAD
    assert call(_12=4095) == BAD and call(_1=-1) == BAD and call(_3=-1) == BAD
    assert call(_16=FAKE + 128) == BAD and call(_13=FAKE + 2) == BAD
    assert call(_17=ws - 1) == WORKSPACE


def test_orthogonalize_arguments():
    lib = _lib.load()
    size = lib.sparcml_orthogonalize_workspace_size
    assert size(-1, 4, 4) == 0 and size(1, 0, 4) == 0 and size(65536, 4, 4) == 0
    assert size(1, 32769, 32769) == 0 and size(1, (1 << 24) + 1, 4) == 0
    ws = size(2, 100, 300)
    assert ws >= 2 * (3 * 100 * 300 * 2 + 2 * 100 * 100 * 2)
    c = np.array(api.NEWTON_SCHULZ, np.float32)
    f = lib.sparcml_orthogonalize
    good = [FAKE, 0, 30000, 300, FAKE, 1, 30000, 300, 2, 100, 300, c.ctypes.data, 5, FAKE, ws, None]

    def call(**change):
        a = list(good)
        for i, v in change.items():
            a[int(i[1:])] = v
        return f(*a)
    for i in (0, 4, 11, 13):
        assert call(**{f"_{i}": None}) == BAD
    assert call(_1=3) == BAD and call(_5=0) == BAD  # the result is 16 bits wide
    assert call(_2=-1) == BAD and call(_3=-1) == BAD and call(_7=299) == BAD
    assert call(_8=-1) == BAD and call(_9=0) == BAD
    assert call(_12=0) == BAD and call(_12=65) == BAD
    assert call(_13=FAKE + 64) == BAD and call(_14=ws - 1) == WORKSPACE
    assert call(_8=0) == 0
    bad = c.copy()
    bad[2, 1] = np.inf
    assert call(_11=bad.ctypes.data) == BAD


def test_muon_step_arguments():
    lib = _lib.load()
    ws = lib.sparcml_orthogonalize_workspace_size(1, 64, 32)
    c = np.array(api.NEWTON_SCHULZ, np.float32)
    f = lib.sparcml_muon_step
    good = [FAKE, 1, 0, 32, FAKE, 0, 0, 32, FAKE, 0, 32, 1, 64, 32, 0.95, 1, 0.1, 0.0, 1.0,
            c.ctypes.data, 5, FAKE, ws, None]

    def call(**change):
        a = list(good)
        for i, v in change.items():
            a[int(i[1:])] = v
        return f(*a)
    for i in (0, 4, 8, 19, 21):
        assert call(**{f"_{i}": None}) == BAD
    assert call(_1=5) == BAD and call(_5=5) == BAD
    assert call(_3=31) == BAD and call(_10=31) == BAD and call(_7=-1) == BAD
    for i in (14, 16, 17, 18):
        assert call(**{f"_{i}": float("nan")}) == BAD
    assert call(_22=ws - 1) == WORKSPACE and call(_8=FAKE + 2) == BAD
    assert call(_11=0) == 0


def test_binding_refuses_host_tensors():
    import torch
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        api.layer_norm(x)
    with pytest.raises(TypeError):
        api.orthogonalize(x)
    with pytest.raises(TypeError):
        api.muon_step(x, x, x, lr=0.1)
