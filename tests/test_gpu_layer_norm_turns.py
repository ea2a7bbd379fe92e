"""Layer norm where every group of threads walks several rows, with a ragged last turn, on the
GPU: the prefetch of the next rows, the turning slots and the running sums of the gradients,
in every variant of whole packs and of odd rows. Tolerances as in test_gpu_layer_norm.py."""
import pytest
import torch

from top_gradient_compression_gb300 import api

from gpu_helpers import DEV
from test_gpu_layer_norm import TYPES, check_backward, check_forward, make

pytestmark = pytest.mark.gpu

# (16-byte packs of a row, rows): at least four turns of the forward grid's 152 SMs x blocks x
# groups in each of its variants for many rows, by their packs per thread and lanes (1 x 8,
# 2 x 8, 4 x 8, 4 x 16, 4 x 32, 8 x 32, 16 x 32, then blocks of up to 512 and 1,024 threads);
# the backward grid is smaller and takes more turns
PACKED = [(5, 100_003), (8, 100_003), (16, 80_001), (31, 70_001), (64, 35_001), (128, 17_501),
          (256, 10_007), (512, 7_501), (1000, 1_301), (1024, 1_301), (3001, 613)]
# (columns, rows), not a whole number of packs: a row to 8, 16 and 32 lanes and to several warps
ODD = [(45, 60_001), (249, 30_001), (501, 15_001), (1023, 7_501), (4097, 1_301), (8191, 613)]


def both(x, dy, w, b):
    got = api.layer_norm(x, w, b, 1e-5)
    check_forward(x, w, b, 1e-5, got)
    back = api.layer_norm_backward(dy, x, got[1], got[2], w)
    check_backward(x, dy, w, got[1], got[2], back)
    return got, back


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("packs,rows", PACKED)
def test_whole_packs(packs, rows, dtype):
    dim = packs * (16 // torch.empty(0, dtype=dtype).element_size())
    both(*make(rows, dim, dtype, packs))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,rows", ODD)
def test_odd_rows(dim, rows, dtype):
    both(*make(rows, dim, dtype, dim))


@pytest.mark.parametrize("dim,rows", [(512, 35_001), (4096, 7_501), (8192, 1_301)])
def test_fp32_weights_of_16_bit_rows(dim, rows):
    x, dy, w, b = make(rows, dim, torch.bfloat16, 5)
    both(x, dy, w.float(), b.float())


@pytest.mark.parametrize("dim,rows,dtype", [(512, 35_001, torch.bfloat16),
                                            (2048, 5_003, torch.float32),
                                            (8192, 1_301, torch.float16),
                                            (1023, 7_501, torch.bfloat16)])
def test_in_place(dim, rows, dtype):
    """The rows ahead are on their way while these are written over."""
    x, dy, w, b = make(rows, dim, dtype, 6)
    (y, mean, rstd), want = both(x, dy, w, b)
    over = x.clone()
    again = api.layer_norm(over, w, b, 1e-5, out=over)
    assert again[0] is over
    for p, q in zip((y, mean, rstd), again):
        assert torch.equal(p, q)
    for which in ("dy", "x"):
        args = {"dy": dy.clone(), "x": x.clone()}
        got = api.layer_norm_backward(args["dy"], args["x"], mean, rstd, w, dx=args[which])
        for p, q in zip(want, got):
            assert torch.equal(p, q)


@pytest.mark.parametrize("dim,rows,pad", [(512, 20_001, 8), (512, 20_001, 3), (1023, 7_501, 2)])
def test_gradients_added_into_slices(dim, rows, pad):
    """dweight and dbias at odd offsets of a flat gradient, added to it; strided rows."""
    x, dy, w, b = make(rows, dim, torch.bfloat16, 7, pad)
    _, mean, rstd = api.layer_norm(x, w, b)
    flat = torch.randn(2 * dim + 5, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    before = flat.clone()
    dw, db = flat[1:dim + 1], flat[dim + 2:2 * dim + 2]
    got = api.layer_norm_backward(dy, x, mean, rstd, w, dweight=dw, dbias=db, accumulate=True)
    check_backward(x, dy, w, mean, rstd, got, (before[1:dim + 1], before[dim + 2:2 * dim + 2]))
    for i in (0, dim + 1, 2 * dim + 2, 2 * dim + 3, 2 * dim + 4):
        assert flat[i] == before[i]
