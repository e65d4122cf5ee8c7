"""The checked build on the operators of include/zero_train.h: their results
still match the 64-bit references and no kernel records a violation."""
import json
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_operators_record_no_violation():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    r = subprocess.run([sys.executable, os.path.join(HERE, "train_checked_runner.py")],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    got = [json.loads(x) for x in r.stdout.splitlines() if x.startswith("{")]
    assert got[0]["case"] == "selftest" and got[0]["violations"] == 1
    assert {x["case"] for x in got[1:]} == {"table_grad", "lookup", "lookup_odd", "wgrad", "policy",
                                            "activation"}
    for x in got[1:]:
        assert x["violations"] == 0, x
