"""The policy example with its block of 8-bit float linear layers, dropout and the
residual join: it runs under the sharded step in both working types, and the
gradients that it writes into a replica are those of the same model in 64 bits."""
import pytest
import torch

from block_util import factors, fp8_64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.mark.parametrize("fp16", [False, True])
def test_block_example_runs(fp16):
    from fsdp_sharded_mixed_shard_gb300.examples.policy_finetune import finetune
    r = finetune(steps=6, fp16=fp16, block=True)
    assert len(r) == 6 and all(0.0 <= x <= 1.0 for x in r)


class Linear8(torch.autograd.Function):
    """x W with both in 8 bits; the input's gradient with dy (E5M2) and W in 8
    bits, the weight's from x and dy as they are."""

    @staticmethod
    def forward(ctx, x, w):
        w8 = fp8_64(w.to(torch.bfloat16), "e4m3", 128)[1]
        ctx.save_for_backward(x, w8)
        return fp8_64(x.to(torch.bfloat16), "e4m3", 1)[1] @ w8

    @staticmethod
    def backward(ctx, dy):
        x, w8 = ctx.saved_tensors
        return fp8_64(dy.to(torch.bfloat16), "e5m2", 1)[1] @ w8.t(), x.t() @ dy


def test_block_example_gradients_against_autograd():
    """One micro-batch's replica against autograd in 64 bits over the same 16-bit
    parameters, masks and 8-bit roundings. What differs is each activation's
    rounding to bf16 (2^-8) and, for weight gradients, to 8-bit checkpoints (2^-7):
    ten in a row stay below 10 2^-7 of a gradient's norm. A value that a bf16
    rounding (off by 2^-9 in the mean) moves over a border of E4M3 or E5M2, borders
    2^-4 to 2^-3 and 2^-3 to 2^-2 apart, is off by that step: at most one element
    in 16 by 2^-3, one in 32 by 2^-2, both 2^-5 in the root mean square; at most
    eight operands in 8 bits stand between a gradient and the inputs, their moves
    independent: below sqrt(8) 2^-5 together."""
    from fsdp_sharded_mixed_shard_gb300.examples.policy_finetune import BlockPolicyModel
    m = BlockPolicyModel(rows=512, n_ranks=2)
    try:
        dev, rows, v, d = m.group.device, m.rows, m.vocab, m.dim
        g = torch.Generator(device=dev)
        g.manual_seed(5)
        with torch.cuda.stream(m.group.stream):
            tok = torch.randint(0, v, (rows,), generator=g, device=dev, dtype=torch.int32)
            tok[-4:] = -1
            act = torch.randint(0, v, (rows,), generator=g, device=dev, dtype=torch.int32)
            adv = torch.randn(rows, generator=g, device=dev)
            w = torch.rand(rows, generator=g, device=dev)
            w[-4:] = 0
            logits = m.forward(tok)
            old = m.log_probs(logits, act, torch.empty(rows, device=dev)) + 0.05
            m.backward(1, tok, act, old, old, adv, w)
        torch.cuda.synchronize()
        p = {k: t.double().clone().requires_grad_() for k, t in m.param.items()}
        assert all(bool((p[k] == 1).all()) for k in ("post", "channel", "norm"))
        first, second = (factors(rows, d, m.drop, 1234, call, 0, dev) for call in (2, 3))
        rms = lambda t: t / ((t * t).mean(1, keepdim=True) + 1e-5).sqrt()  # noqa: E731
        x = 8.0 * p["embed"][tok.long().clamp(min=0)] * (tok >= 0)[:, None] * first
        a, u = Linear8.apply(x, p["gate"]), Linear8.apply(x, p["up"])
        y = Linear8.apply(a * torch.sigmoid(a) * u, p["down"])
        out = x + p["channel"] * (rms(y) * p["post"] * second)
        z = rms(out) * p["norm"]
        lp = torch.log_softmax(Linear8.apply(z, p["out"]), 1)
        lp = lp.gather(1, act.long()[:, None]).squeeze(1)
        r, od = (lp - old.double()).exp(), old.double() - lp
        gain = torch.minimum(r * adv, r.clamp(0.8, 1.28) * adv)
        ((-gain + 0.02 * (od.exp() - od - 1)) * w).sum().backward()
        rep = m.group.replicas[1].view(torch.bfloat16)
        for k, t in p.items():
            got = rep[m.offset[k]:m.offset[k] + t.numel()].view(t.shape).double()
            bound = 10 * 2.0 ** -7 + 8 ** 0.5 * 2.0 ** -5
            assert (got - t.grad).norm() <= bound * t.grad.norm(), k
        assert m.group.read_scaler().error == 0
    finally:
        m.close()
