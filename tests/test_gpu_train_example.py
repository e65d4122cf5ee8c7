"""The policy fine-tuning example learns its task through the operators and the
sharded step, in both working types, and the gradients it writes into a replica
are those of the same loss differentiated in 64 bits."""
import pytest
import torch

import fsdp_sharded_mixed_shard_gb300 as Z

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.mark.parametrize("fp16", [False, True])
def test_policy_example_learns(fp16):
    """31 answers: chance is 0.032; the reward after training is over 0.5."""
    from fsdp_sharded_mixed_shard_gb300.examples.policy_finetune import finetune
    r = finetune(steps=80, fp16=fp16)
    assert sum(r[:5]) / 5 < 0.1
    assert sum(r[-5:]) / 5 > 0.5


def test_example_gradients_against_autograd():
    """One micro-batch's replica against autograd in 64 bits on the same 16-bit
    parameters. The path rounds each activation to bf16 (2^-8) and keeps some
    in 8 bits (2^-7 of a block's largest): ten such roundings in a row, their
    errors independent, stay below 10 * 2^-7 of each gradient's norm."""
    from fsdp_sharded_mixed_shard_gb300.examples.policy_finetune import PolicyModel
    m = PolicyModel(rows=512, n_ranks=2)
    try:
        dev, rows, v = m.group.device, m.rows, m.vocab
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
        ok = (tok >= 0)[:, None]
        x = 8.0 * p["embed"][tok.long().clamp(min=0)] * ok
        a, u = x @ p["gate"], x @ p["up"]
        y = x + (a * torch.sigmoid(a) * u) @ p["down"]
        lp = torch.log_softmax(y @ p["out"], 1).gather(1, act.long()[:, None]).squeeze(1)
        r, od = (lp - old.double()).exp(), old.double() - lp
        gain = torch.minimum(r * adv, r.clamp(0.8, 1.28) * adv)
        ((-gain + 0.02 * (od.exp() - od - 1)) * w).sum().backward()
        rep = m.group.replicas[1].view(torch.bfloat16)
        for k, t in p.items():
            got = rep[m.offset[k]:m.offset[k] + t.numel()].view(t.shape).double()
            assert (got - t.grad).norm() <= 10 * 2.0 ** -7 * t.grad.norm(), k
        assert m.group.read_scaler().error == 0
    finally:
        m.close()
    assert Z.zero_version() >= 100
