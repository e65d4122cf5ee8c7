"""64-bit references and derived error bounds for the operators of
include/zero_train.h (used by tests/test_gpu_train.py).

u: unit roundoff of the 16-bit type; an operator computes in fp32 and rounds
once, so every bound is u |want| + half the smallest subnormal + what fp32 can
lose on the way, stated at each function."""
import math

import torch

import fsdp_sharded_mixed_shard_gb300 as Z

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ZT = {"bf16": Z.ZERO_BF16, "fp16": Z.ZERO_FP16, "fp32": Z.ZERO_FP32}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -24, "fp32": 2.0 ** -149}


def rand(shape, dtype, seed, sd=1.0, dev="cuda"):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float64) * sd).to(DT[dtype])


def offset_rows(rows, cols, ld, dtype, shift=0, fill=None):
    """A [rows, cols] view with row distance ld whose first element sits
    `shift` elements into its allocation; the rest of the allocation holds a
    pattern (returned whole, to check that nothing else is written)."""
    whole = torch.full((shift + max(rows, 1) * ld + 8,), 7.0 if fill is None else fill,
                       device="cuda", dtype=DT[dtype])
    return whole, whole[shift:shift + max(rows, 1) * ld].view(-1, ld)[:rows, :cols]


def within(got, want, bound, what=""):
    """Every element within its bound; NaN and infinities must agree."""
    got, want = got.double(), want.double()
    bad = torch.isnan(got) != torch.isnan(want)
    inf = torch.isinf(want)
    bad |= inf & (got != want)
    fine = torch.isfinite(want)
    bad |= fine & ~((got - want).abs() <= bound)
    if bool(bad.any()):
        i = bad.flatten().nonzero()[0].item()
        b = bound.flatten()[i].item() if torch.is_tensor(bound) and bound.numel() > 1 else bound
        raise AssertionError("%s: %d of %d out of bounds; element %d: got %r want %r bound %r" % (
            what, int(bad.sum()), bad.numel(), i, got.flatten()[i].item(),
            want.flatten()[i].item(), b))


# ------------------------------------------------------------- checkpoints ----

def ckpt64(x):
    """(q, scale byte, values) of the checkpoint of x, block by block in 64 bits."""
    low = -24 if x.dtype == torch.float16 else -126
    rows, cols = x.shape
    pitch = -(-cols // 128) * 128
    b = torch.zeros(rows, pitch, dtype=torch.float64, device=x.device)
    b[:, :cols] = x.double()
    b = b.view(rows, -1, 32)
    fine = torch.isfinite(b).all(2, keepdim=True)
    top = torch.where(fine, b, torch.zeros_like(b)).abs().amax(2, keepdim=True)
    k = torch.where(top > 0, torch.frexp(top).exponent - 7, torch.full_like(top, low).int())
    k = k.clamp(min=low)
    step = ((k.long() + 1023) << 52).view(torch.float64)  # 2^k from its bits: exact
    q = (torch.where(fine, b, torch.zeros_like(b)) / step).round().clamp(-127, 127)
    val = torch.where(fine, q * step, torch.full_like(b, math.nan))
    scale = torch.where(fine, k + 127, torch.full_like(k, 255))
    return (q.view(rows, pitch).to(torch.int8), scale.view(rows, -1).to(torch.uint8),
            val.view(rows, pitch)[:, :cols])


def split_ckpt(buf, rows, cols):
    pitch = -(-cols // 128) * 128
    return (buf[:rows * pitch].view(torch.int8).view(rows, pitch),
            buf[rows * pitch:rows * pitch * 33 // 32].view(rows, pitch // 32))


def gate64(act, x):
    """(z, p, z'): the activation is x p(z) (times u)."""
    if act == Z.ZERO_ACT_SWIGLU:
        return x, torch.sigmoid(x), torch.ones_like(x)
    c, a = 2 * math.sqrt(2 / math.pi), 0.044715
    z = c * (x + a * x ** 3)
    return z, torch.sigmoid(z), c * (1 + 3 * a * x ** 2)


def act64(act, x, u):
    _, p, _ = gate64(act, x)
    return x * p * (u if u is not None else 1.0)


def act_bound(act, x, u, dtype):
    """fp32: z carries 4 roundings (relative 2^-22), exp's argument one more,
    ex2 and the reciprocal 2 ulp each: relative error of p at most
    (|z| + 4) 2^-21; three products after it."""
    y = act64(act, x, u)
    z, _, _ = gate64(act, x)
    return U[dtype] * y.abs() + (z.abs() + 6) * 2.0 ** -21 * y.abs() + TINY[dtype]


def act_grad64(act, x, u, dy):
    _, p, z1 = gate64(act, x)
    dx = dy * (u if u is not None else 1.0) * (p + x * p * (1 - p) * z1)
    return dx, (dy * x * p if u is not None else None)


def act_grad_bounds(act, x, u, dy, dtype):
    """dx = dy u (p + x p (1 - p) z'): the two terms may cancel, so the fp32
    part is relative to their magnitudes, and 1 - p is off by p's own error."""
    z, p, z1 = gate64(act, x)
    rel = (z.abs() + 8) * 2.0 ** -20
    mag = (dy * (u if u is not None else 1.0)).abs() * p * (1 + (x * z1).abs())
    dx, du = act_grad64(act, x, u, dy)
    bx = U[dtype] * dx.abs() + rel * mag + TINY[dtype]
    bu = None if u is None else U[dtype] * du.abs() + rel * du.abs() + TINY[dtype]
    return bx, bu


# ------------------------------------------------------------------ policy ----

def policy64(x, act, old, ref, adv, w, lo, hi, beta, scale):
    """logp, loss, stats and dlogits of the clipped policy loss in 64 bits."""
    x, old, adv, w = (t.double() for t in (x, old, adv, w))
    v = x.shape[1]
    on = (w != 0) & (act >= 0) & (act < v)
    a = act.long().clamp(0, v - 1)[:, None]
    m = x.amax(1, keepdim=True)
    lse = (m + (x - m).exp().sum(1, keepdim=True).log())
    lp = (x.gather(1, a) - lse).squeeze(1)
    r = (lp - old).exp()
    held = r.clamp(1 - lo, 1 + hi)
    cut = held * adv < r * adv
    loss = -torch.where(cut, held, r) * adv
    slope = torch.where(cut, torch.zeros_like(r), -r * adv)
    kl = torch.zeros_like(r)
    if ref is not None:
        d = ref.double() - lp
        kl = torch.expm1(d) - d
        if beta:
            loss = loss + beta * kl
            slope = slope - beta * torch.expm1(d)
    slope = slope * w * scale
    p = (x - lse).exp()
    g = -slope[:, None] * p
    g.scatter_add_(1, a, slope[:, None])
    zero = torch.zeros_like(lp)
    stats = torch.stack([torch.where(on, t, zero).sum() for t in (w * loss, w * kl, w * cut, w)])
    return (torch.where(on, lp, zero), torch.where(on, loss, zero), stats,
            torch.where(on[:, None], g, torch.zeros_like(g)), lse.squeeze(1), p, on)


def logp_bound(x, act, lse):
    """fp32: x_a - m - log s rounds three times at most at |x_a| + |m| + |lse|;
    s: each exp's argument is off by |x - m| 2^-23 (taken at the spread of the
    values that matter, 40) and ex2 by 2 ulp, and at most vocab / 32 + 64
    additions follow one another."""
    x = x.double()
    v = x.shape[1]
    xa = x.gather(1, act.long().clamp(0, v - 1)[:, None]).squeeze(1).abs()
    m = x.amax(1).abs()
    return (xa + m + lse.abs()) * 2.0 ** -23 + 40 * 2.0 ** -23 + 2.0 ** -21 + (
        v / 32 + 64) * 2.0 ** -24
