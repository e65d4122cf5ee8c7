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


def main():
    for c in WGRAD:
        print(json.dumps(wgrad(*c)), flush=True)


if __name__ == "__main__":
    main()
