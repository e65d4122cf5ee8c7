"""The checked build tests the operators' loads and stores against the buffers:
one that it takes for an element shorter than it is gives a violation, and the
access to that element is left out."""
import json
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_buffer_is_tested():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    r = subprocess.run([sys.executable, os.path.join(HERE, "train_bounds_runner.py")],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    got = [json.loads(x) for x in r.stdout.splitlines() if x.startswith("{")]
    seen = {(c["case"], c["buffer"]) for c in got}
    assert seen == {("lookup", 0), ("lookup", 1), ("save", 0), ("save", 6), ("load", 3),
                    ("load", 6), ("wgrad", 0), ("wgrad", 1), ("policy", 0), ("policy", 1),
                    ("logp", 0),
                    *((n, k) for n in ("table_grad", "table_grad_clear") for k in range(4)),
                    *(("act", k) for k in (0, 1, 3, 6, 7)),
                    *(("grad", k) for k in (2, 3, 4, 5, 6, 7))}
    for c in got:
        assert c["clean"] == 0 and c["violations"] > 0 and c["left_out"], c
