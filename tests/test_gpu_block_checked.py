"""The checked build on the operators of include/zero_block.h: their own tests
record no violation; a buffer taken for an element shorter than it is gives one,
and the access to that element is left out; a wait that expires (a copy left out
on purpose, 20 ms) leaves NaN, never a part of a sum, and all else right."""
import json
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
TIMEOUT = 3  # ZERO_DEVERR_TIMEOUT


@pytest.fixture(scope="module")
def cases():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    r = subprocess.run([sys.executable, os.path.join(HERE, "block_checked_runner.py")],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    return [json.loads(x) for x in r.stdout.splitlines() if x.startswith("{")]


def test_no_violations(cases):
    got = [c for c in cases if c["kind"] == "own"]
    assert {c["case"] for c in got} == {"dropout", "join", "copy", "weight", "product", "block"}
    for c in got:
        assert c["violations"] == 0, c


def test_every_buffer_is_tested(cases):
    got = [c for c in cases if c["kind"] == "short"]
    assert {(c["case"], c["buffer"]) for c in got} == {
        *(("dropout", k) for k in range(3)), *(("join", k) for k in (*range(5), *range(10, 15))),
        *(("join_grad", k) for k in (1, 2, 4, 5, 6, 7, 8, 9)),
        ("copy", 0), ("copy", 1), ("weight", 0), ("weight", 1), ("product", 0)}
    for c in got:
        assert c["clean"] == 0 and c["violations"] > 0 and c["left_out"], c


def test_products_give_no_partial_sums(cases):
    got = [c for c in cases if c["kind"] == "expired"]
    assert len(got) == 6
    for c in got:
        assert c["finite"] and c["error"] == TIMEOUT, c
        assert 0 < c["lost"] <= c["all"] and c["others_right"] and c["after_right"], c
    # the block was one of a pair's first tile, or of a later one
    assert [c["first_lost"] for c in got] == [True, False, True, False, False, True]
