"""The operators of include/zero_block.h in a second context of one device, in two in
turn, in one made after another is gone, and in the primary context before and after
its reset: what the library keeps of a device serves in all of them."""
import json
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_context_gives_the_same():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    r = subprocess.run([sys.executable, os.path.join(HERE, "block_contexts_runner.py")],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    runs = [json.loads(x) for x in r.stdout.splitlines() if x.startswith("{")]
    assert [x["run"] for x in runs] == ["first", "second", "first again", "second again", "third",
                                       "primary", "primary after a reset"]
    for x in runs[1:]:
        assert x["sums"] == runs[0]["sums"], x["run"]
    sums = runs[0]["sums"]
    assert len(set(sums.values())) == len(sums)  # none was left as it was (zeros)
