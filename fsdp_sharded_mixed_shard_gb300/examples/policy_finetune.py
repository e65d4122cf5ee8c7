"""Fine-tunes a small token policy with a clipped policy loss under the sharded
step: every operator of include/zero_train.h on its way from the flat working
parameters to a gradient replica, then zero_step.

    python -m fsdp_sharded_mixed_shard_gb300.examples.policy_finetune [--steps 60] [--fp16] [--block]

The model (embedding, a gated MLP with a residual, an output layer) lives in
one flat parameter vector. N ranks are N gradient replicas on one GPU; each
takes its own micro-batch:

  forward    zero_embedding; the MLP's input kept as an 8-bit checkpoint
             (zero_ckpt_save); zero_ckpt_act for SwiGLU and the checkpoints of
             its two inputs; the output layer's input kept as a checkpoint
  loss       zero_token_logp before the update gives the old log-probabilities,
             zero_policy_loss the loss and the gradient of the logits under the
             scaler's loss scale
  backward   zero_ckpt_act_grad from the checkpoints; zero_ckpt_wgrad for every
             weight, zero_embedding_grad for the table, each written at its
             tensor's offset in the rank's replica
  step       Group.step: reduce-scatter, AdamW, cast (and, in fp16, the skip
             of a step whose gradients overflowed)

Forward products and the gradients of activations are library GEMMs, or, with
--block, the operators of include/zero_block.h: linear layers in 8-bit floats
(zero_fp8_linear, zero_fp8_linear_dgrad), dropout on the embedding (zero_dropout),
and the MLP's output joined to the residual stream between two norms, with a
gate and dropout (zero_block_join, zero_block_join_grad). The task:
answer token t with (3 t + 1) mod vocab; the reward is 1 for that and 0 else.
"""
import argparse

import torch

from .. import (ZERO_ACT_SWIGLU, ZERO_BF16, ZERO_E4M3, ZERO_E5M2, ZERO_FP16, ZERO_NORM_RMS,
                ZeroDropoutParams, ZeroJoinParams, ZeroJoinWeights, ZeroPolicyParams,
                ZeroScaler, zero_block_join, zero_block_join_grad,
                zero_block_join_workspace_bytes, zero_cast_params, zero_ckpt_act,
                zero_ckpt_act_grad, zero_ckpt_bytes, zero_ckpt_save, zero_ckpt_wgrad,
                zero_dropout, zero_embedding, zero_embedding_grad,
                zero_embedding_workspace_bytes, zero_fp8_bytes, zero_fp8_linear,
                zero_fp8_linear_dgrad, zero_fp8_quant, zero_fp8_quant_weight,
                zero_fp8_weight_bytes, zero_plan_tensor_offsets, zero_policy_loss,
                zero_token_logp)
from .. import harness, workloads


class PolicyModel:
    """The model's views of one Group's flat parameters and the buffers of one
    micro-batch of `rows` tokens."""

    def __init__(self, vocab=31, dim=64, hidden=128, rows=512, n_ranks=4, fp16=False, lr=1e-2):
        self.vocab, self.dim, self.hidden, self.rows = vocab, dim, hidden, rows
        shapes = self.shapes()
        numels = [a * b for a, b in shapes.values()]
        wl = workloads.Workload("policy_example", numels, n_ranks, 0, not fp16, 3, lr=lr,
                                weight_decay=0.0, init_scale=65536.0 if fp16 else 1.0,
                                dynamic_scale=fp16, steps=1)
        self.group = harness.Group(wl)
        self.group.init_state()
        self.stream = self.group.sptr
        self.dtype = torch.float16 if fp16 else torch.bfloat16
        self.zt = ZERO_FP16 if fp16 else ZERO_BF16
        self.offset = dict(zip(shapes, zero_plan_tensor_offsets(self.group.plan)))
        flat = self.group.flat.view(self.dtype)
        self.param = {k: flat[o:o + a * b].view(a, b) for (k, (a, b)), o in
                      zip(shapes.items(), self.offset.values())}
        dev = self.group.device
        act = lambda *s: torch.empty(*s, dtype=self.dtype, device=dev)  # noqa: E731
        f32 = lambda *s: torch.empty(*s, device=dev)  # noqa: E731
        ckpt = lambda cols: torch.empty(zero_ckpt_bytes(rows, cols), dtype=torch.uint8,  # noqa: E731
                                        device=dev)
        self.x, self.h = act(rows, dim), act(rows, hidden)
        self.dg, self.du = act(rows, hidden), act(rows, hidden)
        self.logits, self.logp, self.loss, self.stats = act(rows, vocab), f32(rows), f32(rows), f32(4)
        self.cx, self.cg, self.cu = ckpt(dim), ckpt(hidden), ckpt(hidden)
        self.ch, self.cy = ckpt(hidden), ckpt(dim)
        self.work = torch.empty(zero_embedding_workspace_bytes(rows, vocab, dim),
                                dtype=torch.uint8, device=dev)
        self.hp = ZeroPolicyParams(0.2, 0.28, 0.02)

    def shapes(self):
        """The tensors of the flat parameter vector, in order."""
        return dict(embed=(self.vocab, self.dim), gate=(self.dim, self.hidden),
                    up=(self.dim, self.hidden), down=(self.hidden, self.dim),
                    out=(self.dim, self.vocab))

    def close(self):
        self.group.close()

    def forward(self, tokens):
        """Logits of a micro-batch; the checkpoints stay for backward()."""
        m, st, rows, p = self, self.stream, self.rows, self.param
        zero_embedding(tokens.data_ptr(), 4, rows, p["embed"].data_ptr(), m.vocab, m.dim, 8.0, m.zt,
                       m.x.data_ptr(), st)
        zero_ckpt_save(m.x.data_ptr(), rows, m.dim, m.dim, m.zt, m.cx.data_ptr(), st)
        gate, up = m.x @ p["gate"], m.x @ p["up"]
        zero_ckpt_act(ZERO_ACT_SWIGLU, gate.data_ptr(), up.data_ptr(), rows, m.hidden, m.hidden,
                      m.zt, m.h.data_ptr(), m.hidden, m.cg.data_ptr(), m.cu.data_ptr(), st)
        y = m.x + m.h @ p["down"]
        zero_ckpt_save(y.data_ptr(), rows, m.dim, m.dim, m.zt, m.cy.data_ptr(), st)
        torch.matmul(y, p["out"], out=m.logits)
        return m.logits

    def log_probs(self, logits, actions, out):
        zero_token_logp(logits.data_ptr(), self.rows, self.vocab, self.vocab, self.zt,
                        actions.data_ptr(), 4, out.data_ptr(), self.stream)
        return out

    def backward(self, rank, tokens, actions, old, ref, advantage, weight):
        """Loss of the last forward() and every parameter's gradient, written
        into rank's replica; the logits become their own gradient."""
        m, st, rows, p = self, self.stream, self.rows, self.param
        replica = m.group.rep_ptrs()[rank]
        at = lambda name: replica + 2 * m.offset[name]  # noqa: E731
        scaler = m.group.scaler.data_ptr()
        zero_policy_loss(m.logits.data_ptr(), rows, m.vocab, m.vocab, m.zt, actions.data_ptr(), 4,
                         old.data_ptr(), ref.data_ptr(), advantage.data_ptr(), weight.data_ptr(),
                         m.hp, scaler, m.logp.data_ptr(), m.loss.data_ptr(), m.stats.data_ptr(),
                         m.logits.data_ptr(), st)
        wgrad = lambda c, cols, dy, n, name: zero_ckpt_wgrad(  # noqa: E731
            c.data_ptr(), rows, cols, dy.data_ptr(), n, n, m.zt, at(name), scaler, st)
        dlogits = m.logits
        wgrad(m.cy, m.dim, dlogits, m.vocab, "out")
        dy = dlogits @ p["out"].t()
        dh = dy @ p["down"].t()
        zero_ckpt_act_grad(ZERO_ACT_SWIGLU, m.cg.data_ptr(), m.cu.data_ptr(), dh.data_ptr(), rows,
                           m.hidden, m.hidden, m.zt, m.dg.data_ptr(), m.du.data_ptr(),
                           m.h.data_ptr(), m.hidden, st)
        zero_ckpt_save(m.h.data_ptr(), rows, m.hidden, m.hidden, m.zt, m.ch.data_ptr(), st)
        wgrad(m.ch, m.hidden, dy, m.dim, "down")
        wgrad(m.cx, m.dim, m.dg, m.hidden, "gate")
        wgrad(m.cx, m.dim, m.du, m.hidden, "up")
        dx = dy + m.dg @ p["gate"].t() + m.du @ p["up"].t()
        zero_embedding_grad(tokens.data_ptr(), 4, rows, dx.data_ptr(), m.vocab, m.dim, 8.0, m.zt,
                            0, at("embed"), m.work.data_ptr(), st)


class BlockPolicyModel(PolicyModel):
    """The same policy with its MLP as a block of a larger model has it: linear
    layers in 8-bit floats, dropout, and the output joined to the residual stream
    between two norms, with a gate per channel."""

    def __init__(self, *args, drop=0.1, **kw):
        super().__init__(*args, **kw)
        m, rows, dev = self, self.rows, self.group.device
        g = self.group
        with torch.cuda.stream(g.stream):
            for name in ("post", "channel", "norm"):  # in the ranks' master shards
                at = torch.arange(m.offset[name], m.offset[name] + m.dim, device=dev)
                g.state[0, 0, at // g.S, at % g.S] = 1.0
            ptrs = [g.state[0, 0, r].data_ptr() for r in range(g.N)]
            zero_cast_params(g.plan, 0, g.N, ptrs, g.flat.data_ptr(), 0, g.sptr)
        raw = lambda n: torch.empty(n, dtype=torch.uint8, device=dev)  # noqa: E731
        self.w8 = {k: raw(zero_fp8_weight_bytes(*m.param[k].shape))
                   for k in ("gate", "up", "down", "out")}
        # 8-bit copies of a layer's input or its output's gradient, by width
        self.a8 = {n: raw(zero_fp8_bytes(rows, n)) for n in {m.dim, m.hidden, m.vocab}}
        act = lambda *s: torch.empty(*s, dtype=self.dtype, device=dev)  # noqa: E731
        self.y, self.stream_out, self.z = act(rows, m.dim), act(rows, m.dim), act(rows, m.dim)
        self.dz, self.dx, self.dy = act(rows, m.dim), act(rows, m.dim), act(rows, m.dim)
        self.g, self.u, self.dh = act(rows, m.hidden), act(rows, m.hidden), act(rows, m.hidden)
        self.stats = torch.empty(rows, 4, device=dev)
        self.join_work = raw(zero_block_join_workspace_bytes(rows, m.dim))
        self.loss_stats = torch.empty(4, device=dev)
        self.drop, self.calls = drop, 0

    def shapes(self):
        vector = (1, self.dim)
        return dict(super().shapes(), post=vector, channel=vector, norm=vector)

    def dropout(self, place):
        """Dropout `place` of this micro-batch; the device's step count (the
        scaler's t) is part of the draw."""
        t = self.group.scaler.data_ptr() + ZeroScaler.t.offset
        return ZeroDropoutParams(self.drop, 1234, 2 * self.calls + place, t)

    def join_params(self):
        return ZeroJoinParams(ZERO_NORM_RMS, 1e-5, 1.0, 1.0, self.dropout(1))

    def vectors(self, at):
        return ZeroJoinWeights(at("post"), 0, at("channel"), at("norm"), 0)

    def linear(self, x, name, out):
        """out = x W, x by its 8-bit copy."""
        k, n = self.param[name].shape
        x8, st = self.a8[k].data_ptr(), self.stream
        zero_fp8_quant(x.data_ptr(), self.rows, k, k, self.zt, ZERO_E4M3, x8, st)
        zero_fp8_linear(x8, ZERO_E4M3, self.rows, self.w8[name].data_ptr(), k, n, self.zt,
                        out.data_ptr(), n, self.group.scaler.data_ptr(), st)
        return out

    def input_gradient(self, dy, name, out):
        """out = dy W^T, dy by its 8-bit copy."""
        k, n = self.param[name].shape
        dy8, st = self.a8[n].data_ptr(), self.stream
        zero_fp8_quant(dy.data_ptr(), self.rows, n, n, self.zt, ZERO_E5M2, dy8, st)
        zero_fp8_linear_dgrad(dy8, ZERO_E5M2, self.rows, self.w8[name].data_ptr(), k, n, self.zt,
                              out.data_ptr(), k, self.group.scaler.data_ptr(), st)
        return out

    def forward(self, tokens):
        m, st, rows, p = self, self.stream, self.rows, self.param
        self.calls += 1
        for name, copy in m.w8.items():  # the step before has changed them
            zero_fp8_quant_weight(p[name].data_ptr(), *p[name].shape, m.zt, copy.data_ptr(), st)
        zero_embedding(tokens.data_ptr(), 4, rows, p["embed"].data_ptr(), m.vocab, m.dim, 8.0, m.zt,
                       m.x.data_ptr(), st)
        zero_dropout(m.dropout(0), m.x.data_ptr(), 0, rows, m.dim, m.dim, m.zt, m.x.data_ptr(),
                     m.dim, st)
        zero_ckpt_save(m.x.data_ptr(), rows, m.dim, m.dim, m.zt, m.cx.data_ptr(), st)
        m.linear(m.x, "gate", m.g)
        m.linear(m.x, "up", m.u)
        zero_ckpt_act(ZERO_ACT_SWIGLU, m.g.data_ptr(), m.u.data_ptr(), rows, m.hidden, m.hidden,
                      m.zt, m.h.data_ptr(), m.hidden, m.cg.data_ptr(), m.cu.data_ptr(), st)
        m.linear(m.h, "down", m.y)
        zero_block_join(m.join_params(), m.vectors(lambda k: p[k].data_ptr()), m.x.data_ptr(),
                        m.y.data_ptr(), rows, m.dim, m.dim, m.zt, m.stream_out.data_ptr(),
                        m.z.data_ptr(), m.stats.data_ptr(), st)
        zero_ckpt_save(m.z.data_ptr(), rows, m.dim, m.dim, m.zt, m.cy.data_ptr(), st)
        return m.linear(m.z, "out", m.logits)

    def backward(self, rank, tokens, actions, old, ref, advantage, weight):
        m, st, rows, p = self, self.stream, self.rows, self.param
        replica = m.group.rep_ptrs()[rank]
        at = lambda name: replica + 2 * m.offset[name]  # noqa: E731
        scaler = m.group.scaler.data_ptr()
        zero_policy_loss(m.logits.data_ptr(), rows, m.vocab, m.vocab, m.zt, actions.data_ptr(), 4,
                         old.data_ptr(), ref.data_ptr(), advantage.data_ptr(), weight.data_ptr(),
                         m.hp, scaler, m.logp.data_ptr(), m.loss.data_ptr(),
                         m.loss_stats.data_ptr(), m.logits.data_ptr(), st)
        wgrad = lambda c, cols, dy, n, name: zero_ckpt_wgrad(  # noqa: E731
            c.data_ptr(), rows, cols, dy.data_ptr(), n, n, m.zt, at(name), scaler, st)
        wgrad(m.cy, m.dim, m.logits, m.vocab, "out")
        m.input_gradient(m.logits, "out", m.dz)
        zero_block_join_grad(m.join_params(), m.vectors(lambda k: p[k].data_ptr()),
                             m.stream_out.data_ptr(), m.y.data_ptr(), m.stats.data_ptr(),
                             m.dz.data_ptr(), 0, rows, m.dim, m.dim, m.zt, m.dx.data_ptr(),
                             m.dy.data_ptr(), m.vectors(at), m.join_work.data_ptr(), st)
        m.input_gradient(m.dy, "down", m.dh)
        zero_ckpt_act_grad(ZERO_ACT_SWIGLU, m.cg.data_ptr(), m.cu.data_ptr(), m.dh.data_ptr(), rows,
                           m.hidden, m.hidden, m.zt, m.dg.data_ptr(), m.du.data_ptr(),
                           m.h.data_ptr(), m.hidden, st)
        zero_ckpt_save(m.h.data_ptr(), rows, m.hidden, m.hidden, m.zt, m.ch.data_ptr(), st)
        wgrad(m.ch, m.hidden, m.dy, m.dim, "down")
        wgrad(m.cx, m.dim, m.dg, m.hidden, "gate")
        wgrad(m.cx, m.dim, m.du, m.hidden, "up")
        m.dx += m.input_gradient(m.dg, "gate", m.dz)
        m.dx += m.input_gradient(m.du, "up", m.dz)
        zero_dropout(m.dropout(0), m.dx.data_ptr(), 0, rows, m.dim, m.dim, m.zt, m.dx.data_ptr(),
                     m.dim, st)
        zero_embedding_grad(tokens.data_ptr(), 4, rows, m.dx.data_ptr(), m.vocab, m.dim, 8.0, m.zt,
                            0, at("embed"), m.work.data_ptr(), st)


def finetune(steps=60, fp16=False, seed=0, n_ranks=4, report=None, block=False):
    """Trains for `steps` steps; returns the mean reward of each."""
    model = (BlockPolicyModel if block else PolicyModel)(n_ranks=n_ranks, fp16=fp16)
    dev, rows, vocab = model.group.device, model.rows, model.vocab
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rewards = []
    try:
        with torch.cuda.stream(model.group.stream):
            weight = torch.full((rows,), 1.0 / (rows - 8), device=dev)
            weight[rows - 8:] = 0  # a ragged batch: the last rows are padding
            for step in range(steps):
                total = 0.0
                for rank in range(n_ranks):
                    tokens = torch.randint(0, vocab, (rows,), generator=g, device=dev,
                                           dtype=torch.int32)
                    tokens[rows - 8:] = -1
                    logits = model.forward(tokens)
                    actions = torch.multinomial(logits.float().softmax(1), 1, generator=g)
                    actions = actions.squeeze(1).to(torch.int32)
                    old = model.log_probs(logits, actions, torch.empty(rows, device=dev))
                    hit = (actions == (3 * tokens + 1) % vocab).float()
                    hit[rows - 8:] = 0
                    mean = (hit * weight).sum()
                    advantage = (hit - mean) / (hit.std() + 1e-3)
                    # the policy a step ago is the reference here: old serves as both
                    model.backward(rank, tokens, actions, old, old, advantage, weight)
                    total += mean.item()
                model.group.step()
                rewards.append(total / n_ranks)
                if report and step % 10 == 9:
                    report("step %3d  mean reward %.3f  scale %g" % (
                        step + 1, rewards[-1], model.group.read_scaler().scale))
        error = model.group.read_scaler().error
        if error:
            raise RuntimeError("device error word %d" % error)
    finally:
        torch.cuda.synchronize()
        model.close()
    return rewards


def main():
    ap = argparse.ArgumentParser(description="policy fine-tuning with the sharded step")
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--fp16", action="store_true", help="fp16 with a dynamic loss scale")
    ap.add_argument("--block", action="store_true",
                    help="8-bit float linear layers, dropout, and norms around the residual join")
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args()
    finetune(a.steps, a.fp16, a.seed, report=print, block=a.block)


if __name__ == "__main__":
    main()
