"""Makes pipeline waits of the operators expire (zero_selftest_plant, checked
build) in its own process and prints one JSON line per case. Used by
tests/test_gpu_train_expiry.py."""
import json
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import fsdp_sharded_mixed_shard_gb300 as Z  # noqa: E402

Z.use_checked_library()

import torch  # noqa: E402

import test_gpu_train as T  # noqa: E402
from train_util import DT, offset_rows, rand  # noqa: E402


def error_of(scaler):
    return Z.ZeroScaler.from_buffer_copy(scaler.cpu().numpy().tobytes()).error


# rows, cols, n, ld, type, step whose copy is left out
WGRAD = [
    (320, 2048, 8192, 8192, "bf16", 0),     # four tiles of five steps per pair: the first
    (320, 2048, 8192, 8192, "bf16", 7),     # the second: its output warps wait by then
    (320, 4096, 4096, 4096, "fp16", 13),    # the third
    (2048, 2048, 8192, 8192, "bf16", 40),   # two column groups, the second of two tiles
    (2048, 128, 256, 256, "bf16", 3),       # tokens split over a cluster
    (8192, 100, 104, 104, "bf16", 5),       # over eight pairs
    (320, 2048, 8191, 8191, "bf16", 6),     # dy off the 16-byte grid
    (2000, 2048, 8191, 8191, "bf16", 1),    # two column groups
    (2048, 128, 255, 255, "fp16", 2),       # split
]


def wgrad(rows, cols, n, ld, dtype, at):
    x = rand((rows, cols), dtype, 1)
    _, dy = offset_rows(rows, n, ld, dtype)
    dy.copy_(rand((rows, n), dtype, 2, 0.1))
    want, got, after = (torch.empty(cols, n, dtype=DT[dtype], device="cuda") for _ in range(3))
    scaler = torch.zeros(20, device="cuda")
    T.run_wgrad(x, dy, ld, dtype, want)
    torch.cuda.synchronize()
    Z.zero_selftest_plant(Z.ZERO_PLANT_NO_COPY, at)
    T.run_wgrad(x, dy, ld, dtype, got, scaler.data_ptr())
    torch.cuda.synchronize()
    Z.zero_selftest_plant(Z.ZERO_PLANT_NOTHING)
    T.run_wgrad(x, dy, ld, dtype, after)
    torch.cuda.synchronize()
    lost = torch.isnan(got)
    same = (got == want) | lost
    return dict(case="wgrad", error=error_of(scaler), lost=int(lost.sum()), all=got.numel(),
                others_right=bool(same.all()), first_lost=bool(lost[0, 0]),
                after_right=torch.equal(after, want), finite=bool(torch.isfinite(want).all()))


# rows, vocab, type, what is left out, row
POLICY = [
    (700, 257, "bf16", Z.ZERO_PLANT_NO_COPY, 4),       # a CTA per row
    (6000, 257, "bf16", Z.ZERO_PLANT_NO_COPY, 10),     # several rows per CTA
    (2048, 50257, "bf16", Z.ZERO_PLANT_NO_COPY, 0),    # pairs of CTAs, several rows each
    (2048, 50257, "bf16", Z.ZERO_PLANT_NO_COPY, 901),  # copied while another row's gradient leaves
    (16, 50257, "fp16", Z.ZERO_PLANT_NO_COPY, 7),      # few rows
    (2048, 50257, "bf16", Z.ZERO_PLANT_NO_SEND, 500),
    (16, 50257, "fp16", Z.ZERO_PLANT_NO_SEND, 3),
    (400, 128256, "fp32", Z.ZERO_PLANT_NO_SEND, 100),
]


def policy(rows, v, dtype, what, at):
    _, x, act, old, ref, adv, w = T.policy_inputs(rows, v, v, dtype, 0, 3)
    w[at] = 0.5
    hp = Z.ZeroPolicyParams(0.2, 0.25, 0.1)

    def run():
        dl = torch.full((rows, v), 7.0, dtype=DT[dtype], device="cuda")
        lp, loss, stats = T.run_policy(x, v, dtype, act, old, ref, adv, w, hp, None, dl)
        torch.cuda.synchronize()
        return lp, loss, stats, dl

    want = run()
    Z.zero_selftest_plant(what, at)
    got = run()
    Z.zero_selftest_plant(Z.ZERO_PLANT_NOTHING)
    after = run()
    lost = torch.isnan(got[0])
    none = torch.isnan(got[3]).all(1)
    right = all(torch.equal(g[~lost], a[~lost]) for g, a in zip((got[0], got[1], got[3]),
                                                                 (want[0], want[1], want[3])))
    return dict(case="policy", at_lost=bool(lost[at]), lost=int(lost.sum()), rows=rows,
                off=int(w[lost].eq(0).sum()), whole=bool((none == lost).all()),
                loss_too=torch.equal(torch.isnan(got[1]), lost), others_right=right,
                first_lost=int(lost.nonzero()[0]) if bool(lost.any()) else -1, at=at,
                stats_nan=bool(torch.isnan(got[2][0])),
                after_right=all(torch.equal(a, b) for a, b in zip(after, want)),
                finite=all(bool(torch.isfinite(t).all()) for t in want))


def logp(rows, v, dtype, at):
    x = rand((rows, v), dtype, 5, 2.0)
    act = torch.randint(0, v, (rows,), device="cuda", dtype=torch.int32)

    def run():
        lp = torch.full((rows,), 9.0, device="cuda")
        Z.zero_token_logp(x.data_ptr(), rows, v, v, T.ZT[dtype], act.data_ptr(), 4, lp.data_ptr(),
                          T.stream())
        torch.cuda.synchronize()
        return lp

    want = run()
    Z.zero_selftest_plant(Z.ZERO_PLANT_NO_SEND, at)
    got = run()
    Z.zero_selftest_plant(Z.ZERO_PLANT_NOTHING)
    lost = torch.isnan(got)
    return dict(case="logp", at_lost=bool(lost[at]), lost=int(lost.sum()), rows=rows,
                others_right=torch.equal(got[~lost], want[~lost]),
                after_right=torch.equal(run(), want), finite=bool(torch.isfinite(want).all()))


def main():
    for c in WGRAD:
        print(json.dumps(wgrad(*c)), flush=True)
    for c in POLICY:
        print(json.dumps(policy(*c)), flush=True)
    for c in ((16, 50257, "bf16", 5), (40, 128256, "fp32", 11)):
        print(json.dumps(logp(*c)), flush=True)


if __name__ == "__main__":
    main()
