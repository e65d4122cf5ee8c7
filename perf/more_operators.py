"""Cases that time the operators at a block's edge and in its linear layers:
dropout from a counter, the join of a block to the residual stream (norms, gate
and residual scale), and linear layers in 8-bit floating point.

`run` computes them in plain torch (32 bits, rounded once at the end), or,
with `own` set, through the library's entry points. `exact` is the same from
the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
BLOCK = 128          # elements that share one scale of the 8-bit floats
EPS = 1e-5


# ------------------------------------------------------------------- cases ----

def listed():
    return [
        # the last tokens of one answer through the embedding's dropout: latency
        dict(name="dropout_16x768_fp16", kind="dropout", dtype="fp16", rows=16, cols=768, p=0.1),
        # a short ragged batch, a row length off every vector size
        dict(name="dropout_1003x2049_fp16", kind="dropout", dtype="fp16", rows=1003, cols=2049, p=0.1),
        # a gated MLP's inner activations for 8k tokens
        dict(name="dropout_8192x8192_bf16", kind="dropout", dtype="bf16", rows=8192, cols=8192, p=0.25),
        # a few tokens through the edge of a GPT-2-sized block: latency
        dict(name="join_16x768_fp16", kind="join", dtype="fp16", rows=16, cols=768, norm="layer", post=False,
             gate=False, p=0.1, a=1.0, s=1.0),
        # one 1024-token sequence, GPT-2-sized: h + dropout(y), then the next layer norm
        dict(name="join_1024x768_fp16", kind="join", dtype="fp16", rows=1024, cols=768, norm="layer", post=False,
             gate=False, p=0.1, a=1.0, s=1.0),
        # a ragged batch at an odd width, everything in use
        dict(name="join_1003x1111_bf16", kind="join", dtype="bf16", rows=1003, cols=1111, norm="layer", post=True,
             gate=True, p=0.1, a=1.0, s=0.5),
        # a Llama-style block with norms on both sides, a gate and a residual scale, 8k tokens
        dict(name="join_8192x2048_bf16", kind="join", dtype="bf16", rows=8192, cols=2048, norm="rms", post=True,
             gate=True, p=0.0, a=1.0, s=0.25),
        # the same at the width of the largest rows taken
        dict(name="join_4096x8192_bf16", kind="join", dtype="bf16", rows=4096, cols=8192, norm="rms", post=True,
             gate=True, p=0.0, a=1.0, s=0.25),
        # a few tokens through a GPT-2-sized qkv layer: latency, one weight read
        dict(name="linear_16_768x2304_fp16", kind="linear", dtype="fp16", rows=16, k=768, n=2304, fmt="e4m3"),
        # odd everything
        dict(name="linear_1003_1111x2222_bf16", kind="linear", dtype="bf16", rows=1003, k=1111, n=2222, fmt="e4m3"),
        # down projection of a Llama-style block for one 2048-token sequence
        dict(name="linear_2048_8192x2048_bf16", kind="linear", dtype="bf16", rows=2048, k=8192, n=2048, fmt="e5m2"),
        # gate or up projection of the same for 8k tokens
        dict(name="linear_8192_2048x8192_bf16", kind="linear", dtype="bf16", rows=8192, k=2048, n=8192, fmt="e4m3"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["dropout", "join", "linear"])
    dtype = rng.choice(["bf16", "fp16"])
    # half of the row lengths are whole numbers of 64, the others anything
    def width(lo, hi):
        w = _log_int(rng, lo, hi)
        return max(64, w // 64 * 64) if rng.random() < 0.5 else w
    if kind == "dropout":
        return dict(kind=kind, dtype=dtype, rows=_log_int(rng, 1, 8192), cols=width(64, 8192),
                    p=rng.choice([0.05, 0.1, 0.25, 0.5]))
    if kind == "join":
        post = rng.random() < 0.6
        return dict(kind=kind, dtype=dtype, rows=_log_int(rng, 1, 4096), cols=width(64, 8192),
                    norm=rng.choice(["rms", "layer"]), post=post, gate=post and rng.random() < 0.7,
                    p=rng.choice([0.0, 0.0, 0.1]), a=rng.choice([1.0, 1.0, 1.4142135]),
                    s=rng.choice([1.0, 0.5, 0.25]))
    return dict(kind=kind, dtype=dtype, rows=_log_int(rng, 1, 8192), k=width(64, 2048), n=width(64, 8192),
                fmt=rng.choice(["e4m3", "e5m2"]))


# ------------------------------------------------------------------ inputs ----

def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c, dt = dict(case), DT[case["dtype"]]
    kind, rows = c["kind"], c["rows"]
    # the loss scale an fp16 run multiplies its root gradient by
    scale = 1024.0 if dt == torch.float16 else 1.0
    s = {"case": c, "dt": dt, "stream": torch.cuda.current_stream().cuda_stream, "work": None}

    def normal(*shape, sd=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).mul_(sd).add_(mean).to(dt)

    def channels(r, n, sd=1.0):
        # each channel has a spread of its own, a few are outliers
        spread = torch.exp(0.5 * torch.randn(n, generator=g, device=dev)).mul_(sd)
        return torch.randn(r, n, generator=g, device=dev).mul_(spread).to(dt)

    if kind in ("dropout", "join"):
        # the run's seed, which dropout of the step this is, and the step the device counts
        s["seed"] = (0x9E3779B97F4A7C15 * (seed + 1)) % (1 << 64)
        s["call"] = 1 + seed % 97
        s["step"] = torch.full((1,), 1000 + seed % 1009, device=dev, dtype=torch.int64)
    if kind == "dropout":
        s["x"], s["res"] = channels(rows, c["cols"]), channels(rows, c["cols"], 2.0)
        s["dy"] = normal(rows, c["cols"], sd=1e-3 * scale)
        s["out"], s["dx"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
    elif kind == "join":
        n = c["cols"]
        s["h"], s["y"] = channels(rows, n, 3.0), channels(rows, n)
        s["dz"], s["dh_out"] = normal(rows, n, sd=1e-3 * scale), normal(rows, n, sd=1e-3 * scale)
        layer = c["norm"] == "layer"
        s["w_pre"], s["b_pre"] = normal(n, sd=0.1, mean=1.0), normal(n, sd=0.05) if layer else None
        s["w_post"] = normal(n, sd=0.1, mean=1.0) if c["post"] else None
        s["b_post"] = normal(n, sd=0.05) if c["post"] and layer else None
        s["gate"] = normal(n, sd=0.1, mean=0.5) if c["gate"] else None
        for name in ("h_out", "z", "dh", "dy"):
            s[name] = torch.empty(rows, n, device=dev, dtype=dt)
        s["stats"] = torch.empty(rows, 4, device=dev, dtype=torch.float32)
        for name in ("w_post", "b_post", "gate", "w_pre", "b_pre"):
            s["d" + name] = None if s[name] is None else torch.empty(n, device=dev, dtype=dt)
    else:
        k, n = c["k"], c["n"]
        s["x"], s["w"] = channels(rows, k), normal(k, n, sd=0.02)
        s["dy"] = normal(rows, n, sd=1e-3 * scale)
        s["y"] = torch.empty(rows, n, device=dev, dtype=dt)
        s["dx"] = torch.empty(rows, k, device=dev, dtype=dt)
    # the device scaler the optimizer step keeps (loss scale first, then its counters)
    s["scaler"] = torch.zeros(20, device=dev, dtype=torch.float32)
    s["scaler"][0] = scale
    return s


# ------------------------------------------------------------- plain forms ----

def _threshold(p):
    return min(int(p * 65536 + 0.5), 65535)


def _mul32(m, x):
    """High and low word of m x for 32-bit words held in int64: a 64-bit
    product does not fit, so by halves of m."""
    lo, hi = (m & 0xFFFF) * x, (m >> 16) * x  # 48 bits each
    mid = hi + (lo >> 16)
    return mid >> 16, (mid & 0xFFFF) << 16 | lo & 0xFFFF


def _draws(s, rows, cols):
    """The generator's 16 bits for each element: Philox 4x32 with 7 rounds,
    key = seed, counter = (column / 8, row, call, step), two columns a word."""
    dev = s["step"].device
    groups = (cols + 7) // 8
    c0 = torch.arange(groups, device=dev)[None, :].expand(rows, groups)
    c1 = torch.arange(rows, device=dev)[:, None].expand(rows, groups)
    c2 = torch.full_like(c0, s["call"])
    c3 = (s["step"] & 0xFFFFFFFF).view(1, 1).expand(rows, groups)
    k0, k1 = s["seed"] & 0xFFFFFFFF, s["seed"] >> 32
    for _ in range(7):
        h0, l0 = _mul32(0xD2511F53, c0)
        h1, l1 = _mul32(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16,
                         c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16], 2)
    return words.view(rows, groups * 8)[:, :cols]


def _drop(s, x, p):
    if p == 0:
        return x
    t = _threshold(p)
    keep = _draws(s, *x.shape) >= t
    return torch.where(keep, x * (65536.0 / (65536 - t)), torch.zeros_like(x))


def _normed(x, layer):
    """x centred (layer) and divided by its root mean square, and 1 / that."""
    if layer:
        x = x - x.mean(1, keepdim=True)
    r = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    return x * r, r


def _norm_back(g, xhat, r, layer):
    out = g - xhat * (g * xhat).mean(1, keepdim=True)
    if layer:
        out = out - g.mean(1, keepdim=True)
    return out * r


def _round8(x, fmt, blocks):
    """x as its 8-bit floats with one power-of-two scale per block stand for it;
    blocks: rows and columns of one."""
    x = x.float()
    (rows, cols), (br, bc) = x.shape, blocks
    b = torch.nn.functional.pad(x, (0, -cols % bc, 0, -rows % br))
    b = b.view(b.shape[0] // br, br, b.shape[1] // bc, bc)
    bits = b.abs().amax((1, 3), keepdim=True).view(torch.int32)
    top = 8 if fmt == "e4m3" else 15  # the largest number is 1.75 2^top
    k = (bits >> 23) - 127 - top + ((bits & 0x7FFFFF) > 0x600000).int()
    k = torch.where(bits == 0, torch.zeros_like(k), k.clamp(min=-126))
    inv, step = ((127 - k) << 23).view(torch.float32), ((k + 127) << 23).view(torch.float32)
    t = torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2
    q = (b * inv).to(t).float() * step
    return q.reshape(q.shape[0] * br, -1)[:rows, :cols]


def _plain(s):
    c, dt, kind = s["case"], s["dt"], s["case"]["kind"]
    if kind == "dropout":
        out = s["res"].float() + _drop(s, s["x"].float(), c["p"])
        return out.to(dt), _drop(s, s["dy"].float(), c["p"]).to(dt)
    if kind == "linear":
        x, w = _round8(s["x"], "e4m3", (1, BLOCK)), _round8(s["w"], "e4m3", (BLOCK, BLOCK))
        dy = _round8(s["dy"], c["fmt"], (1, BLOCK))
        return (x @ w).to(dt), (dy @ w.t()).to(dt)
    layer, p = c["norm"] == "layer", c["p"]
    f = {n: None if s[n] is None else s[n].float() for n in ("w_post", "b_post", "gate", "w_pre", "b_pre")}
    # forward
    n = s["y"].float()
    if c["post"]:
        yhat, ry = _normed(n, layer)
        n = yhat * f["w_post"]
        if layer:
            n = n + f["b_post"]
    b = _drop(s, n, p)
    gb = b * f["gate"] if c["gate"] else b
    h_out = (c["a"] * s["h"].float() + c["s"] * gb).to(dt)
    hhat, rh = _normed(h_out.float(), layer)
    z = hhat * f["w_pre"]
    if layer:
        z = z + f["b_pre"]
    # backward
    dz = s["dz"].float()
    dw_pre = (dz * hhat).sum(0)
    d = s["dh_out"].float() + _norm_back(dz * f["w_pre"], hhat, rh, layer)
    dh = c["a"] * d
    out = [h_out, z.to(dt), dh.to(dt)]
    grads = [dw_pre.to(dt)]
    if layer:
        grads.append(dz.sum(0).to(dt))
    d = c["s"] * d
    if c["gate"]:
        grads.append((d * b).sum(0).to(dt))
        d = d * f["gate"]
    d = _drop(s, d, p)
    if c["post"]:
        grads.append((d * yhat).sum(0).to(dt))
        if layer:
            grads.append(d.sum(0).to(dt))
        d = _norm_back(d * f["w_post"], yhat, ry, layer)
    return out + [d.to(dt)] + grads


# ------------------------------------------------------ the library's calls ----

def _own(s):
    import fsdp_sharded_mixed_shard_gb300 as Z
    c, kind, st, rows = s["case"], s["case"]["kind"], s["stream"], s["case"]["rows"]
    zt = {"bf16": Z.ZERO_BF16, "fp16": Z.ZERO_FP16}[c["dtype"]]
    at = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
    if kind == "dropout":
        n = c["cols"]
        drop = Z.ZeroDropoutParams(c["p"], s["seed"], s["call"], at(s["step"]))
        Z.zero_dropout(drop, at(s["x"]), at(s["res"]), rows, n, n, zt, at(s["out"]), n, st)
        Z.zero_dropout(drop, at(s["dy"]), 0, rows, n, n, zt, at(s["dx"]), n, st)
        return s["out"], s["dx"]
    if kind == "join":
        n, layer = c["cols"], c["norm"] == "layer"
        drop = Z.ZeroDropoutParams(c["p"], s["seed"], s["call"], at(s["step"]))
        hp = Z.ZeroJoinParams(Z.ZERO_NORM_LAYER if layer else Z.ZERO_NORM_RMS, EPS, c["a"], c["s"], drop)
        names = ("w_post", "b_post", "gate", "w_pre", "b_pre")
        w = Z.ZeroJoinWeights(*[at(s[k]) for k in names])
        dw = Z.ZeroJoinWeights(*[at(s["d" + k]) for k in names])
        if s["work"] is None:  # a program keeps one workspace for all its calls
            s["work"] = torch.empty(Z.zero_block_join_workspace_bytes(rows, n), device="cuda", dtype=torch.uint8)
        Z.zero_block_join(hp, w, at(s["h"]), at(s["y"]), rows, n, n, zt, at(s["h_out"]), at(s["z"]),
                          at(s["stats"]), st)
        Z.zero_block_join_grad(hp, w, at(s["h_out"]), at(s["y"]), at(s["stats"]), at(s["dz"]), at(s["dh_out"]),
                               rows, n, n, zt, at(s["dh"]), at(s["dy"]), dw, at(s["work"]), st)
        out = [s[k] for k in ("h_out", "z", "dh", "dy", "dw_pre")]
        return out + [s["d" + k] for k in ("b_pre", "gate", "w_post", "b_post") if s["d" + k] is not None]
    k, n = c["k"], c["n"]
    fmt = Z.ZERO_E4M3 if c["fmt"] == "e4m3" else Z.ZERO_E5M2
    if s["work"] is None:  # 8-bit copies of the input, the weight and the gradient
        s["work"] = [torch.empty(b, device="cuda", dtype=torch.uint8) for b in (
            Z.zero_fp8_bytes(rows, k), Z.zero_fp8_weight_bytes(k, n), Z.zero_fp8_bytes(rows, n))]
    x8, w8, dy8 = (at(t) for t in s["work"])
    Z.zero_fp8_quant_weight(at(s["w"]), k, n, zt, w8, st)
    Z.zero_fp8_quant(at(s["x"]), rows, k, k, zt, Z.ZERO_E4M3, x8, st)
    Z.zero_fp8_linear(x8, Z.ZERO_E4M3, rows, w8, k, n, zt, at(s["y"]), n, at(s["scaler"]), st)
    Z.zero_fp8_quant(at(s["dy"]), rows, n, n, zt, fmt, dy8, st)
    Z.zero_fp8_linear_dgrad(dy8, fmt, rows, w8, k, n, zt, at(s["dx"]), k, at(s["scaler"]), st)
    return s["y"], s["dx"]


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work ----

def work(case):
    c, rows = case, case["rows"]
    if c["kind"] == "dropout":
        # forward: x and residual in, their sum out; backward: dy in, dx out
        return {"bytes": rows * c["cols"] * 10, "flops": 3 * rows * c["cols"]}
    if c["kind"] == "join":
        # forward: h and y in, h' and z out; backward: h', y, dz and dh' in, dh and dy out
        vectors = 2 * (1 + c["gate"] + c["post"] + (c["norm"] == "layer") * (1 + c["post"]))
        return {"bytes": 2 * c["cols"] * (10 * rows + vectors), "flops": 40 * rows * c["cols"]}
    k, n = c["k"], c["n"]
    return {"bytes": 2 * (k * n + 2 * rows * k + 2 * rows * n), "flops": 4 * rows * k * n}


# ------------------------------------------------------------------ 64 bits ----

def _keep64(s, rows, cols, p):
    """Which elements stay, from the generator's definition in numpy."""
    groups = (cols + 7) // 8
    word = np.uint64(0xFFFFFFFF)
    c = [np.broadcast_to(np.arange(groups, dtype=np.uint64), (rows, groups)),
         np.broadcast_to(np.arange(rows, dtype=np.uint64)[:, None], (rows, groups)),
         np.full((rows, groups), s["call"], np.uint64),
         np.full((rows, groups), int(s["step"].item()) % (1 << 32), np.uint64)]
    key = [s["seed"] % (1 << 32), s["seed"] >> 32]
    for _ in range(7):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [b >> np.uint64(32) ^ c[1] ^ np.uint64(key[0]), b & word,
             a >> np.uint64(32) ^ c[3] ^ np.uint64(key[1]), a & word]
        key = [(key[0] + 0x9E3779B9) % (1 << 32), (key[1] + 0xBB67AE85) % (1 << 32)]
    draws = np.stack(c, 2).astype("<u4").view("<u2").reshape(rows, groups * 8)[:, :cols]
    return torch.from_numpy(draws >= _threshold(p)).cuda()


def _norm64(x, layer, w, b):
    if layer:
        v = x.var(1, unbiased=False, keepdim=True)
        return (x - x.mean(1, keepdim=True)) / (v + EPS).sqrt() * w + b
    return x / ((x ** 2).sum(1, keepdim=True) / x.shape[1] + EPS).sqrt() * w


def _values8(x, fmt, br, bc):
    """The values of the 8-bit floats in 64 bits: each block's scale from
    frexp, each element to the nearest number of the format."""
    x = x.double()
    out = torch.empty_like(x)
    bits, low, most = (3, -6, 448.0) if fmt == "e4m3" else (2, -14, 57344.0)
    two_to = lambda e: ((e.long() + 1023) << 52).view(torch.float64)  # noqa: E731  (exact, from its bits)
    for i in range(0, x.shape[1], bc):
        b = x[:, i:i + bc]
        top = b.abs().amax(1)
        if br > 1:
            pad = -top.shape[0] % br
            top = torch.cat([top, top.new_zeros(pad)]).view(-1, br).amax(1).repeat_interleave(br)[:x.shape[0]]
        m, e = torch.frexp(top / most)  # the least k with top <= most 2^k
        k = torch.where(m == 0.5, e - 1, e).clamp(min=-126)
        k = torch.where(top == 0, torch.zeros_like(k), k)
        unit = two_to(k)[:, None]
        v = b / unit
        step = two_to((torch.frexp(v).exponent - 1).clamp(min=low) - bits)
        out[:, i:i + bc] = (v / step).round() * step * unit
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c, dt, rows = case, s["dt"], case["rows"]
    if c["kind"] == "dropout":
        keep = _keep64(s, rows, c["cols"], c["p"]) * (65536.0 / (65536 - _threshold(c["p"])))
        return s["res"].double() + s["x"].double() * keep, s["dy"].double() * keep
    if c["kind"] == "linear":
        x, w = _values8(s["x"], "e4m3", 1, BLOCK), _values8(s["w"], "e4m3", BLOCK, BLOCK)
        dy = _values8(s["dy"], c["fmt"], 1, BLOCK)
        return torch.einsum("tk,kn->tn", x, w), torch.einsum("tn,kn->tk", dy, w)
    layer = c["norm"] == "layer"
    names = [n for n in ("h", "y", "w_post", "b_post", "gate", "w_pre", "b_pre") if s[n] is not None]
    v = {n: s[n].double().requires_grad_() for n in names}
    keep = 1.0
    if c["p"] > 0:
        keep = _keep64(s, rows, c["cols"], c["p"]) * (65536.0 / (65536 - _threshold(c["p"])))
    b = (_norm64(v["y"], layer, v["w_post"], v.get("b_post")) if c["post"] else v["y"]) * keep
    h_out = c["a"] * v["h"] + c["s"] * (b * v["gate"] if c["gate"] else b)
    stored = h_out.detach().to(dt).double().requires_grad_()  # what the next block reads is 16 bits
    z = _norm64(stored, layer, v["w_pre"], v.get("b_pre"))
    pre = [n for n in ("w_pre", "b_pre") if n in v]
    got = torch.autograd.grad(z, [stored] + [v[n] for n in pre], s["dz"].double())
    total = got[0] + s["dh_out"].double()
    rest = [n for n in ("gate", "w_post", "b_post") if n in v]
    back = torch.autograd.grad(h_out, [v["h"], v["y"]] + [v[n] for n in rest], total)
    return [h_out.detach(), z.detach(), back[0], back[1]] + list(got[1:]) + list(back[2:])
