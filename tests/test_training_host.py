"""Host side of the training-step entry points, beyond the refusals of test_training_abi.py:
plans, empty batches and the binding's checks. Nothing here reaches a GPU."""
import subprocess
import sys

import numpy as np
import pytest
import torch

from top_gradient_compression_gb300 import _lib, api

from training_cases import TALL, WAYS

FAKE = 1 << 20  # non-null, aligned, never dereferenced
COEFFS = np.array(api.NEWTON_SCHULZ, np.float32)


@pytest.mark.parametrize("m,n", [(64, 80), (4096, 4096), (5000, 64), (64, 5000), (1, 1 << 24),
                                 (300, 9000), (32768, 32768)])
def test_an_empty_batch_of_any_size(m, n):
    """The size function in a process of its own, which a division by zero would end."""
    code = ("from top_gradient_compression_gb300 import _lib;"
            f"print(_lib.load().sparcml_orthogonalize_workspace_size(0, {m}, {n}))")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.split()[-1] == "256"
    lib = _lib.load()
    ws = lib.sparcml_orthogonalize_workspace_size(0, m, n)
    c = COEFFS.ctypes.data
    assert lib.sparcml_orthogonalize(None, 0, 0, n, None, 1, 0, n, 0, m, n, c, 5, FAKE, ws,
                                     None) == 0
    assert lib.sparcml_muon_step(None, 0, 0, n, None, 0, 0, n, None, 0, n, 0, m, n, 0.9, 1, 0.1,
                                 0.0, 1.0, c, 5, FAKE, ws, None) == 0
    # sizes out of range are refused without matrices too
    assert lib.sparcml_orthogonalize_workspace_size(0, 0, n) == 0
    assert lib.sparcml_orthogonalize_workspace_size(0, m, (1 << 24) + 1) == 0


def test_statistics_off_their_alignment_are_refused():
    """mean and rstd two bytes past a float would be misaligned accesses on the device."""
    lib = _lib.load()
    forward = [FAKE, 0, 16, FAKE, FAKE, 0, 4, 16, 1e-5, FAKE, 16, FAKE, FAKE, None]
    ws = lib.sparcml_layer_norm_backward_workspace_size(4, 16)
    backward = [FAKE, 16, FAKE, 16, 1, FAKE, 0, FAKE, FAKE, 4, 16, FAKE, 16, FAKE, FAKE, 0, FAKE,
                ws, None]
    for i in (11, 12):
        a = list(forward)
        a[i] = FAKE + 2
        assert lib.sparcml_layer_norm(*a) == 1
    for i in (7, 8):
        a = list(backward)
        a[i] = FAKE + 2
        assert lib.sparcml_layer_norm_backward(*a) == 1


class Placed(torch.Tensor):
    """A host tensor that says it lies on a GPU."""
    index = 0
    is_cuda = True

    @property
    def device(self):
        return torch.device("cuda", self.index)

    def get_device(self):
        return self.index


def placed(*shape, index=0, dtype=torch.float32):
    t = torch.Tensor._make_subclass(Placed, torch.zeros(*shape, dtype=dtype))
    t.index = index
    return t


@pytest.fixture
def calls(monkeypatch):
    """Entry points that record the current device and the stream they were given."""
    made, current = [], [0]

    class Device:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    class Library:
        def __getattr__(self, name):
            return lambda *a: made.append((name, current[0], a[-1])) or 0
    monkeypatch.setattr(api._lib, "_lib", Library())
    monkeypatch.setattr(api, "_several", None)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 1000 + d, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    return made


def operands(name):
    """Each operand of a call, as keywords."""
    f32, wide = torch.float32, {"dtype": torch.bfloat16}
    return {
        "layer_norm": {"x": placed(4, 8), "weight": placed(8), "bias": placed(8),
                       "out": placed(4, 8), "mean": placed(4), "rstd": placed(4)},
        "layer_norm_backward": {"dy": placed(4, 8), "x": placed(4, 8), "mean": placed(4),
                                "rstd": placed(4), "weight": placed(8), "dx": placed(4, 8),
                                "dweight": placed(8), "dbias": placed(8),
                                "ws": placed(4096, dtype=torch.uint8)},
        "orthogonalize": {"g": placed(4, 8), "out": placed(4, 8, **wide),
                          "ws": placed(4096, dtype=f32)},
        "muon_step": {"weight": placed(4, 8), "grad": placed(4, 8), "momentum": placed(4, 8),
                      "ws": placed(4096, dtype=torch.uint8)},
    }[name]


OPERATORS = ["layer_norm", "layer_norm_backward", "orthogonalize", "muon_step"]


@pytest.mark.parametrize("name", OPERATORS)
def test_operands_on_two_devices_are_refused(name, calls):
    extra = {"lr": 0.1} if name == "muon_step" else {}
    for odd in operands(name):
        args = operands(name)
        args[odd].index = 1
        with pytest.raises(ValueError, match="one device"):
            getattr(api, name)(**args, **extra)
    assert calls == []


@pytest.mark.parametrize("name", OPERATORS)
def test_the_operands_device_is_current_during_the_call(name, calls):
    extra = {"lr": 0.1} if name == "muon_step" else {}
    for index in (0, 1):
        args = operands(name)
        for t in args.values():
            t.index = index
        getattr(api, name)(**args, **extra)
    assert calls == [(f"sparcml_{name}", i, 1000 + i) for i in (0, 1)]


@pytest.mark.parametrize("name", OPERATORS)
def test_a_stream_of_another_device_is_refused(name, calls):
    class Stream:
        device = torch.device("cuda", 1)
    extra = {"lr": 0.1} if name == "muon_step" else {}
    with pytest.raises(ValueError, match="stream"):
        getattr(api, name)(**operands(name), **extra, stream=Stream())
    assert calls == []


@pytest.mark.parametrize("name", OPERATORS[1:])
def test_a_workspace_has_to_be_contiguous_device_memory(name, calls):
    extra = {"lr": 0.1} if name == "muon_step" else {}
    args = operands(name)
    args["ws"] = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(TypeError, match="ws"):
        getattr(api, name)(**args, **extra)
    args["ws"] = placed(1, dtype=torch.uint8).expand(4096)  # one byte
    with pytest.raises(ValueError, match="ws"):
        getattr(api, name)(**args, **extra)
    assert calls == []


def test_sizes_take_the_ways_that_the_gpu_tests_are_for():
    for (batch, m, n), way in WAYS.items():
        for size, want in (((batch, m, n), way),
                           ((batch, n, m), TALL.get((batch, m, n), way))):
            p = api.orthogonalize_plan(*size)
            got = (p["pair"], p["chains"], p["widths"], p["splits"] > 1, p["halves"])
            assert got == want and not p["small"], size
    assert api.orthogonalize_plan(1, 64, 4096)["small"]
    for bad in ((0, 64, 64), (1, 0, 4), (-1, 4, 4)):
        with pytest.raises(api.SparcmlError):
            api.orthogonalize_plan(*bad)
