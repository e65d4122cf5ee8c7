"""Seeded random shapes, strides, alignments and options of the operators of
include/zero_block.h, each held to its own test's bounds."""
import math
import random

import pytest
import torch

import test_gpu_block as T

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def log_int(r, lo, hi):
    return int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))


@pytest.mark.parametrize("seed", range(12))
def test_random_dropout(seed):
    r = random.Random(seed)
    rows, cols = log_int(r, 1, 600), log_int(r, 1, 6000)
    T.test_dropout(r.choice(["bf16", "fp16"]), rows, cols, cols + r.choice([0, 0, 1, 8, 5]),
                   r.choice([0, 0, 1, 8, 3]), r.random() < 0.5, r.choice([0.0, 0.1, 0.5, 0.9]))


@pytest.mark.parametrize("seed", range(24))
def test_random_join(seed, monkeypatch):
    r = random.Random(seed)
    layer = r.random() < 0.5
    names = [k for k in T.NAMES if r.random() < 0.7]
    names = [k for k in names if k[0] != "b" or (layer and "w" + k[1:] in names)]
    rows, cols = log_int(r, 1, 3000), log_int(r, 1, 8192)
    rows = max(1, min(rows, 3_000_000 // cols))
    if r.random() < 0.4:
        cols = max(8, cols // 8 * 8)
    case = (rows, cols, cols + r.choice([0, 0, 8, 1, 3]), r.choice([0, 0, 8, 1, 5]), layer,
            tuple(names), r.choice([0.0, 0.1, 0.5]), r.choice([1.0, 1.5]), r.choice([1.0, 0.25]))
    monkeypatch.setattr(T, "JOINS", [case])
    T.test_join_and_its_gradient(r.choice(["bf16", "fp16"]), 0)


@pytest.mark.parametrize("seed", range(24))
def test_random_products(seed):
    r = random.Random(seed)
    rows, k, n = (log_int(r, 1, 6000) for _ in range(3))
    while rows * k * n > 10 ** 10:
        rows = max(1, rows // 2)
    T.test_fp8_products(r.choice(["bf16", "fp16"]), r.choice(["e4m3", "e5m2"]), rows, k, n,
                        r.choice([0, 0, 1, 8]), r.choice([0, 0, 8, 3]))


@pytest.mark.parametrize("rows,k,n", [(8192, 128, 4096), (8192, 64, 4096), (6000, 250, 5000),
                                      (4096, 700, 4096)])
def test_short_reductions_of_many_tiles(rows, k, n):
    """One to six blocks per tile and several tiles per pair of SMs, scales that
    differ from block to block: each tile's scales and sums follow close on
    another's."""
    for fmt in ("e4m3", "e5m2"):
        T.test_fp8_products("bf16", fmt, rows, k, n, 0, 0)
        T.test_fp8_products("fp16", fmt, n, rows, k, 0, 0)  # the other way: dy W^T over k
