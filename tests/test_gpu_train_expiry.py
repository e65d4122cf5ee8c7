"""A pipeline wait that expires inside an operator (an arrival is left out on
purpose, with a limit of 20 ms, in the checked build): what was not finished is
NaN and never a part of a sum, the rest is right, and the next call is too."""
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
    r = subprocess.run([sys.executable, os.path.join(HERE, "train_expiry_runner.py")],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    return [json.loads(x) for x in r.stdout.splitlines() if x.startswith("{")]


def test_weight_gradient_gives_no_partial_sums(cases):
    got = [c for c in cases if c["case"] == "wgrad"]
    assert len(got) == 9
    for c in got:
        assert c["finite"] and c["error"] == TIMEOUT, c
        assert 0 < c["lost"] <= c["all"] and c["others_right"] and c["after_right"], c
    # the step was one of a pair's first tile, or of a later one
    assert [c["first_lost"] for c in got] == [
        True, False, False, False, True, True, False, True, True]


def test_policy_rows_left_are_nan(cases):
    got = [c for c in cases if c["case"] == "policy"]
    assert len(got) == 8
    for c in got:
        assert c["finite"] and c["after_right"], c
        # from the row on, the rows of its CTAs and no others; left-out rows stay 0
        assert c["at_lost"] and c["first_lost"] == c["at"] and c["off"] == 0, c
        assert 1 <= c["lost"] <= 16 and c["others_right"], c
        assert c["whole"] and c["loss_too"] and c["stats_nan"], c


def test_log_probabilities_left_are_nan(cases):
    got = [c for c in cases if c["case"] == "logp"]
    assert len(got) == 2
    for c in got:
        assert c["finite"] and c["after_right"] and c["others_right"], c
        assert c["at_lost"] and c["lost"] == 1, c
