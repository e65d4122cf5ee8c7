"""The policy example's block in fp16 under its loss scale: the gradients in a replica
are the scale times those of the same model in 64 bits, and the sharded step takes
them: parameters move, in both working types."""
import pytest
import torch

from block_util import factors, fp8_64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


class Linear8(torch.autograd.Function):
    """x W with both in 8 bits; the input's gradient with dy (E5M2) and W in 8 bits,
    the weight's from x and dy as they are."""

    @staticmethod
    def forward(ctx, x, w):
        w8 = fp8_64(w.to(torch.float16), "e4m3", 128)[1]
        ctx.save_for_backward(x, w8)
        return fp8_64(x.to(torch.float16), "e4m3", 1)[1] @ w8

    @staticmethod
    def backward(ctx, dy):
        x, w8 = ctx.saved_tensors
        return fp8_64(dy.to(torch.float16), "e5m2", 1)[1] @ w8.t(), x.t() @ dy


def batch(m, seed):
    g = torch.Generator(device=m.group.device)
    g.manual_seed(seed)
    draw = lambda: torch.randint(0, m.vocab, (m.rows,), generator=g, device=m.group.device,  # noqa: E731
                                 dtype=torch.int32)
    tok, act = draw(), draw()
    tok[-4:] = -1
    adv = torch.randn(m.rows, generator=g, device=m.group.device)
    w = torch.rand(m.rows, generator=g, device=m.group.device) / m.rows
    w[-4:] = 0
    return tok, act, adv, w


def test_fp16_gradients_against_autograd():
    """What differs is each activation's rounding to fp16 (2^-11) and, for weight
    gradients, to 8-bit checkpoints (2^-7): ten in a row stay below 10 2^-7 of a
    gradient's norm. A value that an fp16 rounding (off by 2^-12 in the mean) moves
    over a border of E4M3 or E5M2, borders 2^-4 to 2^-3 and 2^-3 to 2^-2 apart, is off
    by that step: at most one element in 128 by 2^-3, one in 256 by 2^-2, both below
    2^-6 in the root mean square; at most eight operands in 8 bits stand between a
    gradient and the inputs, their moves independent: below sqrt(8) 2^-6 together.
    Both sides are multiplied by the loss scale, a power of two, before they round."""
    from fsdp_sharded_mixed_shard_gb300.examples.policy_finetune import BlockPolicyModel
    m = BlockPolicyModel(rows=512, n_ranks=2, fp16=True)
    try:
        dev, rows, d = m.group.device, m.rows, m.dim
        scale = m.group.read_scaler().scale
        assert scale == 65536.0
        with torch.cuda.stream(m.group.stream):
            tok, act, adv, w = batch(m, 5)
            logits = m.forward(tok)
            old = m.log_probs(logits, act, torch.empty(rows, device=dev)) + 0.05
            m.backward(1, tok, act, old, old, adv, w)
        torch.cuda.synchronize()
        p = {k: t.double().clone().requires_grad_() for k, t in m.param.items()}
        first, second = (factors(rows, d, m.drop, 1234, call, 0, dev) for call in (2, 3))
        rms = lambda t: t / ((t * t).mean(1, keepdim=True) + 1e-5).sqrt()  # noqa: E731
        x = 8.0 * p["embed"][tok.long().clamp(min=0)] * (tok >= 0)[:, None] * first
        a, u = Linear8.apply(x, p["gate"]), Linear8.apply(x, p["up"])
        y = Linear8.apply(a * torch.sigmoid(a) * u, p["down"])
        out = x + p["channel"] * (rms(y) * p["post"] * second)
        lp = torch.log_softmax(Linear8.apply(rms(out) * p["norm"], p["out"]), 1)
        lp = lp.gather(1, act.long()[:, None]).squeeze(1)
        r, od = (lp - old.double()).exp(), old.double() - lp
        gain = torch.minimum(r * adv, r.clamp(0.8, 1.28) * adv)
        (scale * ((-gain + 0.02 * (od.exp() - od - 1)) * w).sum()).backward()
        rep = m.group.replicas[1].view(torch.float16)
        bound = 10 * 2.0 ** -7 + 8 ** 0.5 * 2.0 ** -6
        for k, t in p.items():
            got = rep[m.offset[k]:m.offset[k] + t.numel()].view(t.shape).double()
            assert bool(torch.isfinite(got).all()), k
            assert t.grad.norm() > 0
            assert (got - t.grad).norm() <= bound * t.grad.norm(), k
        assert m.group.read_scaler().error == 0
    finally:
        m.close()


@pytest.mark.parametrize("fp16", [False, True])
def test_steps_are_taken(fp16):
    """Every step is applied or (fp16) skipped for an overflow that halves the scale;
    one that is applied moves every tensor by about the learning rate."""
    from fsdp_sharded_mixed_shard_gb300.examples.policy_finetune import BlockPolicyModel
    m, steps, lr = BlockPolicyModel(rows=512, n_ranks=2, fp16=fp16, lr=2.0 ** -6), 5, 2.0 ** -6
    try:
        before = {k: t.double().clone() for k, t in m.param.items()}
        for step in range(steps):
            with torch.cuda.stream(m.group.stream):
                for rank in range(2):
                    tok, act, adv, w = batch(m, 10 * step + rank)
                    logits = m.forward(tok)
                    old = m.log_probs(logits, act, torch.empty(m.rows, device=m.group.device))
                    m.backward(rank, tok, act, old, old, adv, w)
                m.group.step()
            if step == 0:
                torch.cuda.synchronize()
                first, s = {k: t.double().clone() for k, t in m.param.items()}, m.group.read_scaler()
        torch.cuda.synchronize()
        end = m.group.read_scaler()
        assert end.error == 0 and end.t + end.n_skipped == steps and end.t > 0
        if not fp16:
            assert end.t == steps and end.scale == 1.0
        else:
            assert end.scale == 65536.0 / 2 ** end.n_skipped
        for k, t in m.param.items():
            assert bool(torch.isfinite(t).all()), k
            moved = (t.double() - before[k]).abs()
            assert bool((moved > 0).any()), k
            if s.t == 1:  # Adam's first step is lr where there is a gradient; one rounding to bf16
                delta = (first[k] - before[k]).abs()
                assert delta.max() <= lr + 2.0 ** -8 * (first[k].abs().max() + lr), k
                assert delta.max() >= lr / 2, k
    finally:
        m.close()
