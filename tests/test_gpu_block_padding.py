"""An 8-bit copy holds zeros past the last column in every row, also where the row's
last block is not finite and so holds NaN up to there."""
import pytest
import torch

from block_util import fp8_64, numbers
from test_gpu_block import copy_of, place, rand, weight_of

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


BAD = (float("nan"), float("inf"), -float("inf"))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("cols,ld,shift", [(1, 1, 0), (100, 104, 0), (129, 129, 3), (250, 250, 0),
                                           (392, 392, 8), (1111, 1111, 0)])
def test_activations(dtype, fmt, cols, ld, shift):
    rows = 70
    x = rand((rows, cols), dtype, 3)
    for r in range(0, rows, 2):  # in the last block: its first column, its last, any
        x[r, max(0, (cols - 1) // 128 * 128) if r % 3 == 0 else cols - 1] = BAD[r % 3]
    x = place(x, ld, shift, dtype)
    blocks = -(-cols // 128)
    q = copy_of(x, rows, cols, ld, dtype, fmt)[:rows * blocks * 128].view(rows, blocks * 128)
    want = torch.isnan(fp8_64(x, fmt, 1)[1])
    assert torch.equal(torch.isnan(numbers(q[:, :cols].contiguous(), fmt)), want)
    assert bool((q[:, cols:] == 0).all())
    assert bool(want[0, cols - 1])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("k,n,shift", [(1, 1, 0), (130, 100, 0), (300, 1111, 3), (200, 392, 8)])
def test_weights(dtype, k, n, shift):
    w = rand((k, n), dtype, 4, 0.02)
    w[k - 1, n - 1] = float("inf")
    w[0, (n - 1) // 128 * 128] = float("nan")
    w = place(w, n, shift, dtype)
    pitch = -(-n // 128) * 128
    q = weight_of(w, k, n, dtype)[:k * pitch].view(k, pitch)
    want = torch.isnan(fp8_64(w, "e4m3", 128)[1])
    assert torch.equal(torch.isnan(numbers(q[:, :n].contiguous(), "e4m3")), want)
    assert bool((q[:, n:] == 0).all())
    assert bool(want[0, n - 1]) and bool(want[k - 1, n - 1])
