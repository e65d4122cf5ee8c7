"""Runs the operators of include/zero_block.h through libzero_checked.so in its
own process and prints one JSON line per case: the tests' own cases with the
violations recorded, each buffer taken for an element shorter than it is, and
waits made to expire (zero_selftest_plant). Used by
tests/test_gpu_block_checked.py."""
import json
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import fsdp_sharded_mixed_shard_gb300 as Z  # noqa: E402

Z.use_checked_library()

import torch  # noqa: E402

import test_gpu_block as T  # noqa: E402
from test_gpu_block import NAMES, at, stream  # noqa: E402
from train_util import DT, offset_rows, rand  # noqa: E402

BF = Z.ZERO_BF16


def status():
    torch.cuda.synchronize()
    return Z.zero_checked_status()[0]


def own_cases():
    for c in T.DROPS:
        yield "dropout", lambda c=c: T.test_dropout("bf16", *c)
    for k in range(len(T.JOINS)):
        yield "join", lambda k=k: T.test_join_and_its_gradient("fp16", k)
    for c in T.COPIES:
        yield "copy", lambda c=c: T.test_fp8_copy("bf16", "e4m3", *c)
    for c in ((1, 1, 0), (100, 300, 1), (1111, 2222, 3), (768, 2304, 8)):
        yield "weight", lambda c=c: T.test_fp8_weight_copy("bf16", *c)
    for c in T.PRODUCTS:
        yield "product", lambda c=c: T.test_fp8_products("bf16", "e4m3", *c)
    yield "block", T.test_block_captured_and_replayed


# --------------------------------------------------------- a buffer too short ----

def array(rows, cols, shift, seed=None):
    _, v = offset_rows(rows, cols, cols, "bf16", shift)
    return v if seed is None else v.copy_(rand((rows, cols), "bf16", seed))


def dropout(cols, shift):
    rows = 9
    x, r, out = array(rows, cols, shift, 1), array(rows, cols, shift, 2), array(rows, cols, shift)
    p = Z.ZeroDropoutParams(0.25, 3, 4, 0)
    return (lambda: Z.zero_dropout(p, at(x), at(r), rows, cols, cols, BF, at(out), cols, stream()),
            {0: None, 1: None, 2: out})


def join(cols, shift, layer, back):
    rows = 9
    h, y, dz, up = (array(rows, cols, shift, k) for k in range(4))
    w = {k: None if k[0] == "b" and not layer else rand((1, cols), "bf16", 9)[0] for k in NAMES}
    g = {k: None if v is None else torch.empty_like(v) for k, v in w.items()}
    h_out, z, dh, dy = (array(rows, cols, shift) for _ in range(4))
    stats = torch.zeros(rows, 4, device="cuda")
    work = torch.empty(Z.zero_block_join_workspace_bytes(rows, cols), dtype=torch.uint8,
                       device="cuda")
    p = Z.ZeroJoinParams(int(layer), 1e-5, 1.0, 0.5, Z.ZeroDropoutParams(0.25, 3, 4, 0))
    fwd = lambda: Z.zero_block_join(p, T.weights_of(w), at(h), at(y), rows, cols, cols, BF,  # noqa: E731
                                    at(h_out), at(z), at(stats), stream())
    if not back:
        # the parameters come in whole blocks: seen where the last element is alone in one
        last = {10 + k: None for k, name in enumerate(NAMES) if w[name] is not None and cols % 8 == 1}
        return fwd, {0: None, 1: None, 2: h_out, 3: z, 4: stats, **last}
    fwd()
    run = lambda: Z.zero_block_join_grad(  # noqa: E731
        p, T.weights_of(w), at(h_out), at(y), at(stats), at(dz), at(up), rows, cols, cols, BF,
        at(dh), at(dy), T.weights_of(g), at(work), stream())
    return run, {1: None, 2: None, 4: None, 5: None, 6: None, 7: dh, 8: dy, 9: None}


def copy(cols, shift):
    rows = 128
    x = array(rows, cols, shift, 5)
    buf = torch.empty(Z.zero_fp8_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    return (lambda: Z.zero_fp8_quant(at(x), rows, cols, cols, BF, 0, at(buf), stream()),
            {0: None, 1: None})


def weight(shift):
    k, n = 128, 512
    w = array(k, n, shift, 6)
    buf = torch.empty(Z.zero_fp8_weight_bytes(k, n), dtype=torch.uint8, device="cuda")
    return (lambda: Z.zero_fp8_quant_weight(at(w), k, n, BF, at(buf), stream()),
            {0: None, 1: None})


def product(rows, k, n):
    x, w = rand((rows, k), "bf16", 1), rand((k, n), "bf16", 2)
    x8 = T.copy_of(x, rows, k, k, "bf16", "e4m3")
    w8 = T.weight_of(w, k, n, "bf16")
    y = array(rows, n, 0)
    return (lambda: Z.zero_fp8_linear(at(x8), 0, rows, at(w8), k, n, BF, at(y), n, 0, stream()),
            {0: y})


def short_cases():
    for cols, shift in ((264, 0), (257, 0)):  # on the grid; off it, the last element in a block
        yield "dropout", dropout(cols, shift)
        for layer in (False, True):
            yield "join", join(cols, shift, layer, False)
            yield "join_grad", join(cols, shift, layer, True)
    yield "copy", copy(512, 0)
    yield "copy", copy(509, 1)  # the last element in a block of its own, as at weight's
    yield "weight", weight(0)
    yield "weight", weight(1)
    yield "product", product(300, 200, 257)    # off the grid
    yield "product", product(16, 8192, 256)    # a split reduction


def short(name, run, buffers):
    run()
    clean = status()
    for k, out in buffers.items():
        if out is not None:
            out[-1, -1] = 7
        Z.zero_selftest_plant(Z.ZERO_PLANT_SHORT, k)
        run()
        n = status()
        Z.zero_selftest_plant(Z.ZERO_PLANT_NOTHING)
        left_out = out is None or out[-1, -1].item() == 7
        run()  # what a run with a short buffer left behind goes
        status()
        yield dict(kind="short", case=name, buffer=k, clean=clean, violations=n, left_out=left_out)


# ---------------------------------------------------------- waits that expire ----

# rows, k, n, direction, block whose copy is left out
EXPIRED = [
    (8192, 640, 2048, "x W", 0),      # several tiles of five blocks per pair: the first
    (8192, 640, 2048, "x W", 7),      # the second, whose sums share columns with the first's
    (8192, 640, 2048, "dy W^T", 13),  # tiles of sixteen blocks: the first
    (8192, 2048, 640, "dy W^T", 8),   # several tiles of five blocks: the second
    (8192, 640, 2047, "x W", 6),      # rows off the 16-byte grid
    (16, 8192, 256, "x W", 3),        # a split reduction
]


def expired(rows, k, n, way, where):
    x, w, dy = rand((rows, k), "bf16", 1), rand((k, n), "bf16", 2), rand((rows, n), "bf16", 3)
    w8 = T.weight_of(w, k, n, "bf16")
    if way == "x W":
        a8, fn, cols = T.copy_of(x, rows, k, k, "bf16", "e4m3"), Z.zero_fp8_linear, n
    else:
        a8, fn, cols = T.copy_of(dy, rows, n, n, "bf16", "e4m3"), Z.zero_fp8_linear_dgrad, k
    out = [torch.empty(rows, cols, device="cuda", dtype=DT["bf16"]) for _ in range(3)]
    scaler = torch.zeros(20, device="cuda")

    def run(o, s):
        fn(at(a8), 0, rows, at(w8), k, n, BF, at(o), cols, at(s), stream())
        torch.cuda.synchronize()

    run(out[0], None)
    Z.zero_selftest_plant(Z.ZERO_PLANT_NO_COPY, where)
    run(out[1], scaler)
    Z.zero_selftest_plant(Z.ZERO_PLANT_NOTHING)
    run(out[2], None)
    want, got, after = out
    lost = torch.isnan(got)
    error = Z.ZeroScaler.from_buffer_copy(scaler.cpu().numpy().tobytes()).error
    return dict(kind="expired", error=error, lost=int(lost.sum()), all=got.numel(),
                first_lost=bool(lost[0, 0]), others_right=bool(((got == want) | lost).all()),
                after_right=torch.equal(after, want), finite=bool(torch.isfinite(want).all()))


def main():
    for name, fn in own_cases():
        fn()
        print(json.dumps(dict(kind="own", case=name, violations=status())), flush=True)
    for name, (run, buffers) in short_cases():
        for line in short(name, run, buffers):
            print(json.dumps(line), flush=True)
    for c in EXPIRED:
        print(json.dumps(expired(*c)), flush=True)


if __name__ == "__main__":
    main()
