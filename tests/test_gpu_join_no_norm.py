"""The join without a norm on either side keeps no statistics: its gradient takes
none."""
import pytest
import torch

from test_gpu_block import NAMES, backward, forward, join_case, target, untouched
from train_util import within

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("names", [(), ("gate",)])
@pytest.mark.parametrize("rows,cols,shift", [(1, 8, 0), (9, 100, 0), (700, 768, 0), (333, 1111, 3)])
def test_gradient_without_statistics(layer, names, rows, cols, shift):
    c = join_case("bf16", rows, cols, cols, shift, layer, names, 0.25, 1.5, 0.5)
    whole, h_out = target(rows, cols, cols, shift, "bf16")
    forward(c, h_out, None, None)
    within(h_out, *c["ref"].h_out(c["h"].double(), c["y"].double()), "h_out")
    (wh, dh), (wy, dy) = (target(rows, cols, cols, shift, "bf16") for _ in range(2))
    grads = {k: torch.empty(cols, device="cuda", dtype=torch.bfloat16) if k in names else None
             for k in NAMES}
    backward(c, h_out, None, dh, dy, grads, dz=False)
    want = c["ref"].grads(h_out.double(), c["y"].double(), None, c["dh_out"].double())
    within(dh, *want["dh"], "dh")
    within(dy, *want["dy"], "dy")
    for k in names:
        within(grads[k], *want[k], k)
    for w, v in ((whole, h_out), (wh, dh), (wy, dy)):
        untouched(w, v)
