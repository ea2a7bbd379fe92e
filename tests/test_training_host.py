"""Host side of the training-step entry points, beyond the refusals of test_training_abi.py:
plans, empty batches and the binding's checks. Nothing here reaches a GPU."""
import subprocess
import sys

import numpy as np
import pytest

from top_gradient_compression_gb300 import _lib, api

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
