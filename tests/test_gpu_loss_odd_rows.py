"""Token log-probabilities and the policy loss on rows with odd values: large
finite logits, masks among them, taken tokens of the type's lowest value, ruled-out tokens
and infinite losses in the statistics, rows of the largest length."""
import math

import pytest
import torch

import fsdp_sharded_mixed_shard_gb300 as Z
import test_gpu_train as T
from train_util import DT, TINY, U, ZT, rand, within

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def token_logp(x, act):
    lp = torch.full((x.shape[0],), 9.0, device="cuda")
    dtype = next(k for k, t in DT.items() if t == x.dtype)
    Z.zero_token_logp(x.data_ptr(), x.shape[0], x.shape[1], x.stride(0), ZT[dtype], act.data_ptr(),
                      act.element_size(), lp.data_ptr(), T.stream())
    return lp


def logp64(x, act):
    """(logp, its bound, share of every token): the maximum is subtracted first,
    so that 64 bits hold the rest beside it. The kernel holds m log2(e) to half
    an ulp, at most 2^-24 |m| 1.5 and never over 64; that enters every exponent
    and log s, which round at its size. The rest as in train_util.logp_bound."""
    d = x.double()
    v = x.shape[1]
    m = d.amax(1, keepdim=True)
    e = (d - m).exp()
    s = e.sum(1, keepdim=True)
    xa = (d - m).gather(1, act.long()[:, None]).squeeze(1)
    lp = xa - s.log().squeeze(1)
    held = (m.squeeze(1).abs() * 1.5 * 2.0 ** -24).clamp(max=64.0)
    bound = (xa.abs() + held + math.log(v) + 1) * 2.0 ** -22 + 40 * 2.0 ** -23 + 2.0 ** -21 + (
        v / 32 + 64) * 2.0 ** -24
    return lp, bound, e / s


def masked(rows, v, dtype, fill, seed):
    """Six kinds of rows by turns: the first half masked; all but three tokens;
    all; the fill beside half of it and nothing else; both in the first half;
    nothing masked."""
    x = rand((rows, v), dtype, seed, 2.0)
    at = torch.arange(v, device="cuda")
    half = at < v // 2
    few = (at != 1) & (at != v // 3) & (at != v - 2)
    third = at % 3 == 0
    for r in range(rows):
        k = r % 6
        if k in (0, 4):
            x[r, half] = fill
        if k == 1:
            x[r, few] = fill
        if k in (2, 3):
            x[r] = fill
        if k == 3:
            x[r, third] = fill / 2
        if k == 4:
            x[r, half & third] = fill / 2
    return x


FILLS = [-1e8, -1e9, -3e9, -1e10, -1e12, -1e20, -1e30, -2e30, -2.0 ** 101, "lowest", 1e9, 1e10,
         1e20, 2.0 ** 101]
# one CTA per row, a cluster per row, rows of several CTAs in several turns
SIZES = [(6, 1000), (6, 50257), (600, 1003), (12, 128256)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,v", SIZES)
@pytest.mark.parametrize("fill", FILLS)
def test_large_finite_logits(dtype, rows, v, fill):
    fill = torch.finfo(DT[dtype]).min if fill == "lowest" else fill
    x = masked(rows, v, dtype, fill, 11)
    act = x.float().topk(2, 1).indices[:, 1].to(torch.int32)
    want, bound, p = logp64(x, act)
    within(token_logp(x, act), want, bound, "token logp")
    g = torch.Generator(device="cuda")
    g.manual_seed(12)
    adv = torch.randn(rows, generator=g, device="cuda")
    w = torch.rand(rows, generator=g, device="cuda") + 0.1
    old, ref = (want - 0.1).float(), (want + 0.2).float()
    dl = torch.full_like(x, 7.0)
    hp = Z.ZeroPolicyParams(0.2, 0.3, 0.1)
    lp, loss, stats = T.run_policy(x, v, dtype, act, old, ref, adv, w, hp, None, dl)
    within(lp, want, bound, "logp")
    r, ed = (want - old.double()).exp(), (ref.double() - want).exp()
    a, ww, d = adv.double(), w.double(), ref.double() - want
    size = r * a.abs() + 0.1 * (ed + 1 + d.abs())
    err = size * 2 * (bound + 2.0 ** -21)
    wl = -r * a + 0.1 * (torch.expm1(d) - d)  # no ratio is past an edge
    within(loss, wl, err, "loss")
    sums = torch.stack([(ww * wl).sum(), (ww * (torch.expm1(d) - d)).sum(), 0 * ww.sum(), ww.sum()])
    within(stats, sums, torch.stack([(ww * err).sum(), 10 * (ww * err).sum(), 0 * ww.sum(),
                                     0 * ww.sum()]) + 1e-6 * (ww * (1 + size)).sum(), "stats")
    slope = ww * (-r * a + 0.1 * (1 - ed))
    want_g = -slope[:, None] * p
    want_g.scatter_add_(1, act.long()[:, None], slope[:, None])
    pm = p.clone()
    pm.scatter_add_(1, act.long()[:, None], torch.ones(rows, 1, dtype=torch.float64, device="cuda"))
    # exp's argument rounds at its size, at most 2 bound; next to a maximum of
    # 2^30 and more every other token's share is nothing (below 2^-60)
    bg = U[dtype] * want_g.abs() + (pm + 2.0 ** -60) * (
        ww * size * 4 * (bound + 2.0 ** -21))[:, None] + TINY[dtype]
    within(dl, want_g, bg, "dlogits")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,v", SIZES)
@pytest.mark.parametrize("fill", FILLS[:9])
def test_masked_token_taken(dtype, rows, v, fill):
    """The taken token is one of the masked: its logp is the mask's value less
    the rest, a rounding or two at its size."""
    x = masked(rows, v, dtype, fill, 13)
    act = x.float().argmin(1)
    want, bound, _ = logp64(x, act)
    within(token_logp(x, act), want, bound + want.abs() * 2.0 ** -22, "token logp")


@pytest.mark.parametrize("dtype", ["bf16", "fp32", "fp16"])
@pytest.mark.parametrize("v", [40, 50257])
def test_lowest_value_taken(dtype, v):
    """The lowest finite value less a few units is that value in fp32, so the
    ratio to a policy that says the same is 1 and its KL term 0."""
    low = torch.finfo(DT[dtype]).min
    x = rand((3, v), dtype, 14)
    x[:, 5:] = low
    x[2, 0] = -low / 2  # the sum of the two passes the type's range
    act = torch.tensor([7, v - 1, 9], device="cuda", dtype=torch.int32)
    want, _, p = logp64(x, act)
    want = want.float()
    lp = token_logp(x, act)
    assert torch.isfinite(lp[:2]).all()
    within(lp, want, want.abs().double() * 2.0 ** -22, "token logp")
    adv = torch.tensor([1.0, -2.0, 0.5], device="cuda")
    w = torch.ones(3, device="cuda")
    dl = torch.empty_like(x)
    got, loss, stats = T.run_policy(x[:2], v, dtype, act[:2], lp[:2], lp[:2], adv[:2], w[:2],
                                    Z.ZeroPolicyParams(0.2, 0.2, 0.1), None, dl[:2])
    assert torch.equal(got, lp[:2]) and torch.equal(loss, -adv[:2]) and stats[1] == 0
    want_g = adv[:2, None].double() * p[:2]
    want_g.scatter_add_(1, act[:2].long()[:, None], -adv[:2, None].double())
    within(dl[:2], want_g, U[dtype] * want_g.abs() + 2.0 ** -18 * p[:2] + TINY[dtype], "dlogits")


@pytest.mark.parametrize("rows", [5, 3000])
def test_kl_statistic_without_a_reference(rows):
    """No reference, no KL term: 0 also where the taken token is ruled out."""
    v = 33
    x = rand((rows, v), "bf16", 15)
    x[3, 4] = float("-inf")
    act = torch.full((rows,), 4, device="cuda", dtype=torch.int32)
    one = torch.ones(rows, device="cuda")
    lp, loss, stats = T.run_policy(x, v, "bf16", act, -one, None, one, one,
                                   Z.ZeroPolicyParams(0.2, 0.2, 0.5), None, None)
    assert lp[3] == float("-inf") and torch.isfinite(loss).all()
    assert stats[1] == 0 and stats[3] == rows


@pytest.mark.parametrize("rows,at", [(1, 0), (5, 3), (3000, 0), (3000, 1700), (3000, 2999)])
def test_infinite_loss_in_the_statistics(rows, at):
    """A ratio past fp32 with a negative advantage: that row's loss is +inf, and
    so is the sum; the other sums do not change."""
    v = 33
    x = rand((rows, v), "bf16", 16)
    act = torch.full((rows,), 4, device="cuda", dtype=torch.int32)
    one = torch.ones(rows, device="cuda")
    old = token_logp(x, act)
    old[at] = -1000.0
    lp, loss, stats = T.run_policy(x, v, "bf16", act, old, None, -one, one,
                                   Z.ZeroPolicyParams(0.2, 0.2, 0.0), None, None)
    assert loss[at] == math.inf and torch.isfinite(loss).sum() == rows - 1
    assert stats[0] == math.inf and stats[1] == 0 and stats[2] == 0 and stats[3] == rows
    # finite terms whose sum passes fp32, at ratios of 1: the call's own logp
    big = torch.full((rows,), 3e38, device="cuda")
    _, loss, stats = T.run_policy(x, v, "bf16", act, lp, None, -big, one,
                                  Z.ZeroPolicyParams(0.2, 0.2, 0.0), None, None)
    assert torch.equal(loss, big) and stats[0] == (math.inf if rows > 1 else 3e38)


@pytest.mark.parametrize("dtype,shift", [("bf16", 0), ("bf16", 1), ("bf16", 7), ("fp16", 3),
                                         ("fp32", 0), ("fp32", 3)])
def test_rows_of_the_largest_length(dtype, shift):
    v = Z.ZERO_MAX_LOGIT_ROW_BYTES // (4 if dtype == "fp32" else 2)
    T.test_policy_loss(2, v, v, shift, dtype)
