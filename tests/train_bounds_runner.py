"""Takes each buffer of each operator for one element shorter than it is
(zero_selftest_plant, checked build) in its own process and prints one JSON line
per case. Used by tests/test_gpu_train_bounds.py."""
import json
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import fsdp_sharded_mixed_shard_gb300 as Z  # noqa: E402

Z.use_checked_library()

import torch  # noqa: E402

import test_gpu_train as T  # noqa: E402
from train_util import offset_rows, rand  # noqa: E402

BF = Z.ZERO_BF16


def place(t, ld, shift):
    _, v = offset_rows(*t.shape, ld, "bf16", shift)
    return v.copy_(t)


def lookup(dim, shift):
    vocab, rows = 50, 21
    table = place(rand((vocab, dim), "bf16", 1), dim, shift)
    tok = torch.arange(rows, device="cuda", dtype=torch.int32) + vocab - rows
    _, out = offset_rows(rows, dim, dim, "bf16", shift)
    yield lambda: Z.zero_embedding(tok.data_ptr(), 4, rows, table.data_ptr(), vocab, dim, 1.0, BF,
                                   out.data_ptr(), T.stream())
    yield {0: None, 1: out}


def table_grad(dim, shift, accumulate, named):
    """named: whether a token names the table's last row; 99 tokens one row, which spans runs."""
    vocab, rows = 200, 130
    tok = torch.full((rows,), 7, device="cuda", dtype=torch.int32)
    tok[99:] = torch.arange(rows - 99, device="cuda", dtype=torch.int32) + (169 if named else 100)
    dy = place(rand((rows, dim), "bf16", 2), dim, shift)
    _, grad = offset_rows(vocab, dim, dim, "bf16", shift)
    yield lambda: T.run_grad(tok, dy, vocab, dim, 1.0, "bf16", accumulate, grad)
    yield {0: None, 1: grad, 2: None, 3: None}


def ckpt(op, gated, cols, ld, shift):
    rows = 13
    x, u, dy = (place(rand((rows, cols), "bf16", k), ld, shift) for k in (3, 4, 5))
    n = Z.zero_ckpt_bytes(rows, cols)
    kx, ku = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    y, dx, du = (offset_rows(rows, cols, ld, "bf16", shift)[1] for _ in range(3))
    act = Z.ZERO_ACT_SWIGLU if gated else Z.ZERO_ACT_GELU
    g = lambda t: t.data_ptr() if gated else 0  # noqa: E731
    st = T.stream()
    if op == "save":
        yield lambda: Z.zero_ckpt_save(x.data_ptr(), rows, cols, ld, BF, kx.data_ptr(), st)
        yield {0: None, 6: None}
    elif op == "load":
        yield lambda: Z.zero_ckpt_load(kx.data_ptr(), rows, cols, BF, y.data_ptr(), ld, st)
        yield {3: y, 6: None}
    elif op == "act":
        yield lambda: Z.zero_ckpt_act(act, x.data_ptr(), g(u), rows, cols, ld, BF, y.data_ptr(),
                                      ld, kx.data_ptr(), g(ku), st)
        yield {0: None, 3: y, 6: None, **({1: None, 7: None} if gated else {})}
    else:
        yield lambda: Z.zero_ckpt_act_grad(act, kx.data_ptr(), g(ku), dy.data_ptr(), rows, cols, ld,
                                           BF, dx.data_ptr(), g(du), y.data_ptr(), ld, st)
        yield {2: None, 3: y, 4: dx, 6: None, **({5: du, 7: None} if gated else {})}


def wgrad(rows, cols, n, shift):
    x, dy = rand((rows, cols), "bf16", 6), place(rand((rows, n), "bf16", 7), n, shift)
    ck = torch.empty(Z.zero_ckpt_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    Z.zero_ckpt_save(x.data_ptr(), rows, cols, cols, BF, ck.data_ptr(), T.stream())
    torch.cuda.synchronize()
    _, dw = offset_rows(cols, n, n, "bf16", shift)
    yield lambda: Z.zero_ckpt_wgrad(ck.data_ptr(), rows, cols, dy.data_ptr(), n, n, BF,
                                    dw.data_ptr(), 0, T.stream())
    yield {0: None, 1: dw}


def policy(rows, v, shift, shift_out, last, dtype):
    """Rows and a length that leave the last element alone in its block; last:
    the last row's weight."""
    _, x, act, old, ref, adv, w = T.policy_inputs(rows, v, v, dtype, shift, 8)
    w[rows - 1] = last
    _, dl = offset_rows(rows, v, v, dtype, shift_out)
    hp = Z.ZeroPolicyParams(0.2, 0.2, 0.1)
    yield lambda: T.run_policy(x, v, dtype, act, old, ref, adv, w, hp, None, dl)
    yield {1: dl, **({0: None} if last and (shift + rows * v) % (8 if dtype == "bf16" else 4) == 1
                     else {})}


def logp(rows, v):
    x = rand((rows, v), "bf16", 9)
    act = torch.full((rows,), v - 1, device="cuda", dtype=torch.int32)
    lp = torch.empty(rows, device="cuda")
    yield lambda: Z.zero_token_logp(x.data_ptr(), rows, v, v, BF, act.data_ptr(), 4, lp.data_ptr(),
                                    T.stream())
    yield {0: None}


def cases():
    for dim, shift in ((264, 0), (257, 0), (257, 3)):
        yield "lookup", lookup(dim, shift)
        for accumulate in (0, 1):
            yield "table_grad", table_grad(dim, shift, accumulate, True)
        yield "table_grad_clear", table_grad(dim, shift, 0, False)
    for cols, ld, shift in ((264, 264, 0), (257, 300, 1), (130, 136, 0), (1000, 1000, 0)):
        for op in ("save", "load", "act", "grad"):
            for gated in (False, True)[:1 if op in ("save", "load") else 2]:
                yield op, ckpt(op, gated, cols, ld, shift)
    for c in ((65, 130, 264, 0), (300, 130, 777, 0), (300, 130, 264, 1),   # one part
              (2048, 128, 256, 0), (2048, 128, 255, 1), (2000, 200, 104, 0)):  # split
        yield "wgrad", wgrad(*c)
    for dtype in ("bf16", "fp32"):
        for c in ((9, 257, 0, 0, 0.5), (9, 257, 0, 0, 0.0), (9, 257, 0, 3, 0.5),
                  (3, 50257, 1, 1, 0.5),
                  (4, 264, 0, 0, 0.5), (4, 5000, 0, 0, 0.0), (700, 264, 0, 0, 0.5)):
            yield "policy", policy(*c, dtype)
    yield "logp", logp(9, 257)
    yield "logp", logp(17, 50257)


def main():
    for name, case in cases():
        run, buffers = case
        run()
        torch.cuda.synchronize()
        clean, _ = Z.zero_checked_status()
        for k, out in buffers.items():
            if out is not None:
                out[-1, -1] = 7
            Z.zero_selftest_plant(Z.ZERO_PLANT_SHORT, k)
            run()
            torch.cuda.synchronize()
            n, _ = Z.zero_checked_status()
            Z.zero_selftest_plant(Z.ZERO_PLANT_NOTHING)
            print(json.dumps(dict(case=name, buffer=k, clean=clean, violations=n,
                                  left_out=out is None or out[-1, -1].item() == 7)), flush=True)


if __name__ == "__main__":
    main()
