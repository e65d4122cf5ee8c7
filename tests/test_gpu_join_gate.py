"""A gate that is infinite in some channels: those come out infinite where dropout
keeps n (with a bias infinite or NaN: the kernel multiplies the normed y and the bias
by the gate apart, infinities whose signs may differ), the stream alone where it does
not, every other channel as it was. A bias that is not there adds nothing."""
import pytest
import torch

from block_util import Join64
from test_gpu_block import forward, join_case
from train_util import within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("names", [("gate",), ("w_post", "gate"), ("w_post", "b_post", "gate")])
@pytest.mark.parametrize("cols", [264, 263])
@pytest.mark.parametrize("p", [0.0, 0.5])
def test_infinite_gate(layer, names, cols, p):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    if not layer and "b_post" in names:
        pytest.skip("biases belong to layer norm")
    rows = 40
    c = join_case("bf16", rows, cols, cols, 0, layer, names, p, 1.0, 0.5, seed=3)
    finite = dict(c["w"], gate=c["w"]["gate"].clone())
    c["w"]["gate"][5] = float("inf")
    c["w"]["gate"][cols - 1] = -float("inf")
    h_out = torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16)
    forward(c, h_out, None, None)
    ref = Join64(layer, c["eps"], 1.0, 0.5, c["keep"], finite, "bf16")
    n = ref.branch(c["y"].double())[0]
    want, bound = ref.h_out(c["h"].double(), c["y"].double())
    for col in (5, cols - 1):
        big = 0.5 * c["w"]["gate"][col].double() * n[:, col]
        want[:, col] = torch.where(c["keep"][:, col] > 0, big, c["h"][:, col].double())
        bound[:, col] = 2.0 ** -8 * want[:, col].abs()
    if "b_post" in names:
        lost = torch.isinf(want) & torch.isnan(h_out)
        h_out = torch.where(lost, want, h_out.double())
    within(h_out, want, bound, "h_out")
