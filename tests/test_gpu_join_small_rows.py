"""The join with eps = 0: rows whose mean square is a normal fp32 number come out as
they should however small they are, those below that NaN, as rows of zeros do: never
an infinity, never a value that fp32 has lost."""
import pytest
import torch

from block_util import Join64
from test_gpu_block import NAMES, backward, forward, join_case
from train_util import within

pytestmark = pytest.mark.gpu

# row's size; squares below 2^-126 (1.2e-38) are subnormal or 0
FINE = [1.0, 1e-9, 1e-15, 1e-18]
LOST = [3e-20, 1e-21, 1e-24, 1e-30, 1e-37, 0.0]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def case(names, layer, cols):
    sizes = FINE + LOST
    c = join_case("bf16", len(sizes), cols, cols, 0, layer, names, 0.0, 1.0, 1.0, eps=0.0)
    scale = torch.tensor(sizes, device="cuda", dtype=torch.float64)[:, None]
    for name in ("h", "y"):
        c[name].copy_(c[name].double() * scale)
    return c


def buffers(c, n):
    return [torch.empty(c["rows"], c["cols"], device="cuda", dtype=torch.bfloat16) for _ in range(n)]


@pytest.mark.parametrize("cols", [96, 257, 2048])
@pytest.mark.parametrize("layer", [False, True])
def test_norm_after_the_block(layer, cols):
    c = case(("w_post", "b_post") if layer else ("w_post",), layer, cols)
    (h_out,) = buffers(c, 1)
    forward(c, h_out, None, None)
    n = len(FINE)
    ref = Join64(layer, 0.0, 1.0, 1.0, c["keep"][:n], c["w"], "bf16")
    within(h_out[:n], *ref.h_out(c["h"][:n].double(), c["y"][:n].double()), "h_out")
    assert bool(torch.isnan(h_out[n:]).all())


@pytest.mark.parametrize("cols", [96, 257, 2048])
@pytest.mark.parametrize("layer", [False, True])
def test_norm_before_the_next_block_and_its_gradient(layer, cols):
    """y is 0, so that the stored h_out is h."""
    names = ("w_pre", "b_pre") if layer else ("w_pre",)
    c = case(names, layer, cols)
    c["y"].zero_()
    h_out, z, dh, dy = buffers(c, 4)
    stats = torch.empty(c["rows"], 4, device="cuda")
    forward(c, h_out, z, stats)
    assert torch.equal(h_out, c["h"])
    n = len(FINE)
    ref = Join64(layer, 0.0, 1.0, 1.0, c["keep"][:n], c["w"], "bf16")
    within(z[:n], *ref.z(h_out[:n].double()), "z")
    assert bool(torch.isnan(z[n:]).all())
    grads = {k: torch.empty(cols, device="cuda", dtype=torch.bfloat16) if k in names else None
             for k in NAMES}
    backward(c, h_out, stats, dh, dy, grads)
    want = ref.grads(h_out[:n].double(), c["y"][:n].double(), c["dz"][:n].double(),
                     c["dh_out"][:n].double())
    within(dh[:n], *want["dh"], "dh")
    assert bool(torch.isnan(dh[n:]).all())


def test_eps_of_the_least_normal_number():
    """A row of zeros with any eps above 0 is 0; the smallest eps taken is 2^-126."""
    c = case(("w_post", "w_pre"), False, 96)
    c["eps"] = 2.0 ** -126
    c["y"].zero_()
    c["h"].zero_()
    h_out, z = buffers(c, 2)
    forward(c, h_out, z, None)
    assert bool((h_out == 0).all()) and bool((z == 0).all())


def test_eps_that_takes_the_sum_past_the_range():
    """Mean square and eps each in fp32's range, their sum not: NaN, not 0."""
    c = case(("w_post",), False, 96)
    c["eps"] = 3e38
    c["y"][0] = 1e19
    (h_out,) = buffers(c, 1)
    forward(c, h_out, None, None)
    assert bool(torch.isnan(h_out[0]).all()) and bool(torch.isfinite(h_out[1:]).all())
