"""Cases that time the operators of a micro-batch's forward and backward pass:
the embedding and its table gradient, 8-bit activation checkpoints and their
use in the backward pass, and the clipped policy loss with its gradient.

`run` computes them in plain torch (32 bits, rounded once at the end), or,
with `own` set, through the library's entry points. `exact` is the same from
the definitions in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 32           # elements that share one checkpoint scale
CLIP_LO, CLIP_HI, KL = 0.2, 0.28, 0.04


# ------------------------------------------------------------------- cases ----

def listed():
    return [
        # one 1024-token sequence through the token embedding of the GPT-2-sized list
        dict(name="lookup_1k_768_fp16", kind="lookup", dtype="fp16", rows=1024, vocab=50257, dim=768, scale=1.0),
        # a micro-batch of four 8k sequences, Llama-style table, outputs scaled by sqrt(dim)
        dict(name="lookup_32k_2048_bf16", kind="lookup", dtype="bf16", rows=32768, vocab=128256, dim=2048, scale=45.254834),
        # the table's gradient for eight 1024-token sequences, GPT-2-sized table
        dict(name="table_grad_8k_768_fp16", kind="table_grad", dtype="fp16", rows=8192, vocab=50257, dim=768, scale=1.0),
        # the same for a Llama-style micro-batch: the dense 0.5 GB table gradient
        dict(name="table_grad_16k_2048_bf16", kind="table_grad", dtype="bf16", rows=16384, vocab=128256, dim=2048, scale=45.254834),
        # a short ragged batch through GELU: odd rows, a row length off every vector size
        dict(name="gelu_1003x2050_fp16", kind="gelu", dtype="fp16", rows=1003, cols=2050),
        # the gated MLP of one Llama-style block for 8k tokens
        dict(name="swiglu_8192x8192_bf16", kind="swiglu", dtype="bf16", rows=8192, cols=8192),
        # qkv weight gradient of the GPT-2-sized block for one sequence
        dict(name="wgrad_1024_768x2304_fp16", kind="wgrad", dtype="fp16", rows=1024, cols=768, n=2304),
        # gate/up weight gradient of the Llama-style block for 8k tokens
        dict(name="wgrad_8192_2048x8192_bf16", kind="wgrad", dtype="bf16", rows=8192, cols=2048, n=8192),
        # the last few tokens of one answer: latency
        dict(name="policy_16x50257_fp16", kind="policy", dtype="fp16", rows=16, vocab=50257),
        # two 1024-token answers, odd vocabulary: every second row starts off the 4-byte grid
        dict(name="policy_2048x50257_bf16", kind="policy", dtype="bf16", rows=2048, vocab=50257),
        # a policy micro-batch over the large vocabulary
        dict(name="policy_4096x128256_bf16", kind="policy", dtype="bf16", rows=4096, vocab=128256),
        # the reference policy's log-probabilities from fp32 logits
        dict(name="logp_2048x128256_fp32", kind="logp", dtype="fp32", rows=2048, vocab=128256),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["lookup", "table_grad", "gelu", "swiglu", "wgrad", "policy", "logp"])
    dtype = rng.choice(["bf16", "fp16"])
    # half of the row lengths are whole numbers of 64, the others anything
    def width(lo, hi):
        w = _log_int(rng, lo, hi)
        return max(64, w // 64 * 64) if rng.random() < 0.5 else w
    if kind in ("lookup", "table_grad"):
        return dict(kind=kind, dtype=dtype, rows=_log_int(rng, 1, 16384), vocab=_log_int(rng, 1000, 128256),
                    dim=width(64, 2048), scale=rng.choice([1.0, 45.254834]))
    if kind in ("gelu", "swiglu"):
        return dict(kind=kind, dtype=dtype, rows=_log_int(rng, 1, 8192), cols=width(64, 8192))
    if kind == "wgrad":
        return dict(kind=kind, dtype=dtype, rows=_log_int(rng, 1, 8192), cols=width(64, 2048), n=width(64, 8192))
    if kind == "logp":
        return dict(kind=kind, dtype=rng.choice(["bf16", "fp16", "fp32"]), rows=_log_int(rng, 1, 2048),
                    vocab=_log_int(rng, 1000, 128256))
    return dict(kind=kind, dtype=dtype, rows=_log_int(rng, 1, 4096), vocab=_log_int(rng, 1000, 128256))


# ------------------------------------------------------------------ inputs ----

def _tokens(g, rows, vocab, dev):
    """Token ids with the rank-frequency law of text (p ~ 1/rank, ids spread
    over the table) and the last sixteenth padding (-1), as a ragged batch has."""
    u = torch.rand(rows, generator=g, device=dev, dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab)) - 1.0).to(torch.int64).clamp_(0, vocab - 1)
    tok = (rank * 7919) % vocab
    tok[rows - rows // 16:] = -1
    return tok.to(torch.int32)


def _weights(rows, dev):
    """Prompt tokens carry no loss: 16 of every 64 rows (their last one is
    kept where the batch is shorter than that)."""
    w = (torch.arange(rows, device=dev) % 64 >= 16).to(torch.float32)
    if rows <= 16:
        w[rows - 1] = 1.0
    return w / w.sum()


def _active(rows):
    return 1 if rows <= 16 else rows - (rows // 64) * 16 - min(16, rows % 64)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c, dt = dict(case), DT[case["dtype"]]
    kind, rows = c["kind"], c["rows"]
    # the loss scale an fp16 run multiplies its root gradient by
    scale = 1024.0 if dt == torch.float16 else 1.0
    s = {"case": c, "dt": dt, "loss_scale": scale, "stream": torch.cuda.current_stream().cuda_stream}

    def normal(*shape, sd=1.0, dtype=dt):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).mul_(sd).to(dtype)

    if kind in ("lookup", "table_grad"):
        s["tokens"] = _tokens(g, rows, c["vocab"], dev)
        if kind == "lookup":
            s["table"] = normal(c["vocab"], c["dim"], sd=0.02)
            s["out"] = torch.empty(rows, c["dim"], device=dev, dtype=dt)
        else:
            s["dy"] = normal(rows, c["dim"], sd=1e-3 * scale)
            s["out"] = torch.empty(c["vocab"], c["dim"], device=dev, dtype=dt)
            # enough for any row count and width of this file's range
            s["work"] = None
    elif kind in ("gelu", "swiglu"):
        # pre-activations: each channel has a spread of its own, a few are outliers
        spread = torch.exp(0.5 * torch.randn(c["cols"], generator=g, device=dev))
        for name in ("x",) if kind == "gelu" else ("x", "u"):
            s[name] = (torch.randn(rows, c["cols"], generator=g, device=dev) * spread).to(dt)
        s["dy"] = normal(rows, c["cols"], sd=1e-3 * scale)
        for name in ("y", "dx", "h") if kind == "gelu" else ("y", "dx", "du", "h"):
            s[name] = torch.empty(rows, c["cols"], device=dev, dtype=dt)
        s["ckpt"] = None
    elif kind == "wgrad":
        s["x"] = normal(rows, c["cols"])
        s["dy"] = normal(rows, c["n"], sd=1e-3 * scale)
        s["dw"] = torch.empty(c["cols"], c["n"], device=dev, dtype=dt)
        s["ckpt"] = None
    else:
        v = c["vocab"]
        x = torch.randn(rows, v, generator=g, device=dev, dtype=torch.float32).mul_(2.5)
        # the taken token is a likely one
        pick = torch.randint(0, v, (rows, 16), generator=g, device=dev)
        act = pick.gather(1, x.gather(1, pick).argmax(1, keepdim=True)).squeeze(1)
        s["logits"] = x.to(dt)
        s["actions"] = act.to(torch.int32)
        s["logp"] = torch.empty(rows, device=dev, dtype=torch.float32)
        if kind == "policy":
            x = s["logits"]
            lp = torch.empty(rows, device=dev)
            for i in range(0, rows, 512):
                xi = x[i:i + 512].float()
                lp[i:i + 512] = xi.gather(1, act[i:i + 512, None]).squeeze(1) - xi.logsumexp(1)
            # ratios of a policy a few updates old, some past the clip edges; one that
            # would sit on an edge is moved off it (which side it falls on is rounding)
            d = 0.15 * torch.randn(rows, generator=g, device=dev)
            for edge in (math.log(1 - CLIP_LO), math.log(1 + CLIP_HI)):
                d = torch.where((d - edge).abs() < 1e-3, torch.full_like(d, edge + 2e-3), d)
            s["old"] = lp - d
            s["ref"] = lp + 0.3 * torch.randn(rows, generator=g, device=dev)
            s["adv"] = torch.randn(rows, generator=g, device=dev)
            s["w"] = _weights(rows, dev)
            s["loss"] = torch.empty(rows, device=dev)
            s["stats"] = torch.empty(4, device=dev)
            s["dlogits"] = torch.empty(rows, v, device=dev, dtype=dt)
    # the device scaler the optimizer step keeps (loss scale first, then its counters)
    s["scaler"] = torch.zeros(20, device=dev, dtype=torch.float32)
    s["scaler"][0] = scale
    return s


# ------------------------------------------------------------- plain forms ----

def _k_min(dt):
    return -24 if dt == torch.float16 else -126


def _round_trip(x):
    """x in 32 bits -> the values its 8-bit checkpoint stands for."""
    dt, x = x.dtype, x.float()
    rows, cols = x.shape
    pad = -cols % BLOCK
    if pad:
        x = torch.cat([x, x.new_zeros(rows, pad)], 1)
    b = x.view(rows, -1, BLOCK)
    top = b.abs().amax(2, keepdim=True)
    k = ((top.view(torch.int32) >> 23) - 127 - 6).clamp(min=_k_min(dt))
    step = ((k + 127) << 23).view(torch.float32)
    q = torch.clamp(torch.round(b / step), -127, 127)
    return (q * step).view(rows, -1)[:, :cols]


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


_C, _A = math.sqrt(2.0 / math.pi), 0.044715


def _plain(s):
    c, dt, kind = s["case"], s["dt"], s["case"]["kind"]
    if kind == "lookup":
        tok = s["tokens"].long()
        ok = (tok >= 0) & (tok < c["vocab"])
        rows = s["table"][tok.clamp(0, c["vocab"] - 1)].float() * c["scale"]
        return (rows * ok[:, None]).to(dt)
    if kind == "table_grad":
        tok = s["tokens"].long()
        ok = (tok >= 0) & (tok < c["vocab"])
        g = torch.zeros(c["vocab"], c["dim"], device=tok.device)
        g.index_add_(0, tok.clamp(0, c["vocab"] - 1), s["dy"].float() * ok[:, None])
        return (g * c["scale"]).to(dt)
    if kind == "gelu":
        x, dy = s["x"].float(), s["dy"].float()
        y = 0.5 * x * (1 + torch.tanh(_C * (x + _A * x * x * x)))
        x = _round_trip(s["x"])
        t = torch.tanh(_C * (x + _A * x * x * x))
        h = 0.5 * x * (1 + t)
        dx = dy * (0.5 * (1 + t) + 0.5 * x * (1 - t * t) * _C * (1 + 3 * _A * x * x))
        return y.to(dt), dx.to(dt), h.to(dt)
    if kind == "swiglu":
        x, u, dy = s["x"].float(), s["u"].float(), s["dy"].float()
        y = x * _sigmoid(x) * u
        x, u = _round_trip(s["x"]), _round_trip(s["u"])
        p = _sigmoid(x)
        h = x * p * u
        dx = dy * u * p * (1 + x * (1 - p))
        du = dy * x * p
        return y.to(dt), dx.to(dt), du.to(dt), h.to(dt)
    if kind == "wgrad":
        return (_round_trip(s["x"]).t() @ s["dy"].float()).to(dt)
    x = s["logits"].float()
    a = s["actions"].long()[:, None]
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    z = e.sum(1, keepdim=True)
    lp = (x.gather(1, a) - top - torch.log(z)).squeeze(1)
    if kind == "logp":
        return lp
    w, adv = s["w"], s["adv"]
    on = w > 0
    r = torch.exp(lp - s["old"])
    rc = r.clamp(1 - CLIP_LO, 1 + CLIP_HI)
    cut = (rc * adv < r * adv) & on
    d = s["ref"] - lp
    kl = torch.exp(d) - d - 1
    loss = torch.where(on, -torch.minimum(r * adv, rc * adv) + KL * kl, torch.zeros_like(lp))
    gl = torch.where(cut, torch.zeros_like(r), -r * adv) + KL * (1 - torch.exp(d))
    gl = torch.where(on, s["loss_scale"] * w * gl, torch.zeros_like(gl))
    dx = e / z * -gl[:, None]
    dx.scatter_add_(1, a, gl[:, None])
    stats = torch.stack([(w * loss).sum(), (w * torch.where(on, kl, torch.zeros_like(kl))).sum(),
                         (w * cut).sum(), w.sum()])
    return torch.where(on, lp, torch.zeros_like(lp)), loss, stats, dx.to(dt)


# ------------------------------------------------------ the library's calls ----

def _own(s):
    import fsdp_sharded_mixed_shard_gb300 as Z
    c, kind, st, rows = s["case"], s["case"]["kind"], s["stream"], s["case"]["rows"]
    zt = {"bf16": Z.ZERO_BF16, "fp16": Z.ZERO_FP16, "fp32": Z.ZERO_FP32}[c["dtype"]]
    if kind == "lookup":
        Z.zero_embedding(s["tokens"].data_ptr(), 4, rows, s["table"].data_ptr(), c["vocab"], c["dim"], c["scale"],
                         zt, s["out"].data_ptr(), st)
        return s["out"]
    if kind == "table_grad":
        if s["work"] is None:  # a program keeps one workspace for all its calls
            s["work"] = torch.empty(Z.zero_embedding_workspace_bytes(rows, c["vocab"], c["dim"]), device="cuda",
                                    dtype=torch.uint8)
        Z.zero_embedding_grad(s["tokens"].data_ptr(), 4, rows, s["dy"].data_ptr(), c["vocab"], c["dim"], c["scale"],
                              zt, 0, s["out"].data_ptr(), s["work"].data_ptr(), st)
        return s["out"]
    if kind in ("gelu", "swiglu"):
        cols, gated = c["cols"], kind == "swiglu"
        act = Z.ZERO_ACT_SWIGLU if gated else Z.ZERO_ACT_GELU
        if s["ckpt"] is None:
            n = Z.zero_ckpt_bytes(rows, cols)
            s["ckpt"] = [torch.empty(n, device="cuda", dtype=torch.uint8) for _ in range(2 if gated else 1)]
        ck = [t.data_ptr() for t in s["ckpt"]] + [0]
        Z.zero_ckpt_act(act, s["x"].data_ptr(), s["u"].data_ptr() if gated else 0, rows, cols, cols, zt,
                        s["y"].data_ptr(), cols, ck[0], ck[1], st)
        Z.zero_ckpt_act_grad(act, ck[0], ck[1], s["dy"].data_ptr(), rows, cols, cols, zt, s["dx"].data_ptr(),
                             s["du"].data_ptr() if gated else 0, s["h"].data_ptr(), cols, st)
        return (s["y"], s["dx"], s["du"], s["h"]) if gated else (s["y"], s["dx"], s["h"])
    if kind == "wgrad":
        cols, n = c["cols"], c["n"]
        if s["ckpt"] is None:
            s["ckpt"] = torch.empty(Z.zero_ckpt_bytes(rows, cols), device="cuda", dtype=torch.uint8)
        Z.zero_ckpt_save(s["x"].data_ptr(), rows, cols, cols, zt, s["ckpt"].data_ptr(), st)
        Z.zero_ckpt_wgrad(s["ckpt"].data_ptr(), rows, cols, s["dy"].data_ptr(), n, n, zt, s["dw"].data_ptr(),
                          s["scaler"].data_ptr(), st)
        return s["dw"]
    v = c["vocab"]
    if kind == "logp":
        Z.zero_token_logp(s["logits"].data_ptr(), rows, v, v, zt, s["actions"].data_ptr(), 4, s["logp"].data_ptr(), st)
        return s["logp"]
    hp = Z.ZeroPolicyParams(CLIP_LO, CLIP_HI, KL)
    Z.zero_policy_loss(s["logits"].data_ptr(), rows, v, v, zt, s["actions"].data_ptr(), 4, s["old"].data_ptr(),
                       s["ref"].data_ptr(), s["adv"].data_ptr(), s["w"].data_ptr(), hp, s["scaler"].data_ptr(),
                       s["logp"].data_ptr(), s["loss"].data_ptr(), s["stats"].data_ptr(), s["dlogits"].data_ptr(), st)
    return s["logp"], s["loss"], s["stats"], s["dlogits"]


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work ----

def work(case):
    c = case
    rows, b = c["rows"], 4 if c["dtype"] == "fp32" else 2
    if c["kind"] == "lookup":
        return {"bytes": rows * (4 + 2 * b * c["dim"]), "flops": rows * c["dim"]}
    if c["kind"] == "table_grad":
        return {"bytes": rows * (4 + b * c["dim"]) + b * c["vocab"] * c["dim"], "flops": (rows + c["vocab"]) * c["dim"]}
    if c["kind"] in ("gelu", "swiglu"):
        n, q = rows * c["cols"], 1 + 1 / BLOCK
        # forward: x in, y and checkpoint out; backward: checkpoint and dy in, gradients and the activation out
        per = (2 * b + q) + (q + b + 2 * b) if c["kind"] == "gelu" else (3 * b + 2 * q) + (2 * q + b + 3 * b)
        return {"bytes": int(n * per), "flops": 30 * n}
    if c["kind"] == "wgrad":
        q = 1 + 1 / BLOCK
        return {"bytes": int(rows * c["cols"] * (b + 2 * q) + b * rows * c["n"] + b * c["cols"] * c["n"]),
                "flops": 2 * rows * c["cols"] * c["n"]}
    if c["kind"] == "logp":
        return {"bytes": rows * (b * c["vocab"] + 8), "flops": 3 * rows * c["vocab"]}
    on = _active(rows)
    return {"bytes": b * c["vocab"] * (on + rows) + rows * 28, "flops": 6 * on * c["vocab"]}


# ------------------------------------------------------------------ 64 bits ----

def _stored64(x):
    """The values of the checkpoint, from its definition, in 64 bits."""
    low, x = _k_min(x.dtype), x.double()
    out = torch.empty_like(x)
    for i in range(0, x.shape[1], BLOCK):
        b = x[:, i:i + BLOCK]
        top = b.abs().max(1, keepdim=True).values
        k = torch.where(top > 0, torch.frexp(top).exponent - 1 - 6, torch.full_like(top, low).int()).clamp(min=low)
        unit = torch.ldexp(torch.ones_like(top), k)
        out[:, i:i + BLOCK] = (b / unit).round().clamp(-127, 127) * unit
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c, kind = case, case["kind"]
    if kind in ("lookup", "table_grad"):
        tok = s["tokens"].long()
        at = ((tok >= 0) & (tok < c["vocab"])).nonzero().squeeze(1)
        if kind == "lookup":
            out = torch.zeros(c["rows"], c["dim"], device="cuda", dtype=torch.float64)
            out[at] = c["scale"] * s["table"][tok[at]].double()
            return out
        g = torch.zeros(c["vocab"], c["dim"], device="cuda", dtype=torch.float64)
        return g.index_put_((tok[at],), c["scale"] * s["dy"][at].double(), accumulate=True)
    if kind == "wgrad":
        return torch.einsum("tk,tn->kn", _stored64(s["x"]), s["dy"].double())
    if kind in ("gelu", "swiglu"):
        x, dy = s["x"].double(), s["dy"].double()
        k, a = (2 / math.pi) ** 0.5, 0.044715
        if kind == "gelu":
            # x * sigmoid(2 z) is the same function as x/2 (1 + tanh z)
            gate = lambda v: torch.sigmoid(2 * k * (v + a * v ** 3))  # noqa: E731
            v = _stored64(s["x"])
            p = gate(v)
            return x * gate(x), dy * (p + v * p * (1 - p) * 2 * k * (1 + 3 * a * v ** 2)), v * p
        v, u = _stored64(s["x"]), _stored64(s["u"])
        p = torch.sigmoid(v)
        return x * torch.sigmoid(x) * s["u"].double(), dy * u * (p + v * p * (1 - p)), dy * v * p, v * p * u
    x, a = s["logits"].double(), s["actions"].long()
    lp_all = torch.log_softmax(x, 1)
    del x
    lp = lp_all[torch.arange(c["rows"], device="cuda"), a]
    if kind == "logp":
        return lp
    w, adv, old, ref = (s[n].double() for n in ("w", "adv", "old", "ref"))
    on = w > 0
    r = (lp - old).exp()
    inside = torch.where(adv >= 0, r <= 1 + CLIP_HI, r >= 1 - CLIP_LO)
    gain = torch.where(inside, r, torch.where(adv >= 0, 1.0 + CLIP_HI, 1.0 - CLIP_LO)) * adv
    kl = torch.expm1(ref - lp) - (ref - lp)
    loss = (KL * kl - gain) * on
    slope = (-(r * adv * inside) - KL * torch.expm1(ref - lp)) * on * w * s["loss_scale"]
    grad = lp_all.exp_().mul_(-slope[:, None])
    grad[torch.arange(c["rows"], device="cuda"), a] += slope
    stats = torch.stack([(w * loss).sum(), (w * kl * on).sum(), (w * ~inside * on).sum(), w.sum()])
    return lp * on, loss, stats, grad
