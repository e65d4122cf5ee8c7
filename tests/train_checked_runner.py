"""Runs the operators of include/zero_train.h through libzero_checked.so in its
own process and prints one JSON line per case with the violations recorded.
Used by tests/test_gpu_train_checked.py."""
import json
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import fsdp_sharded_mixed_shard_gb300 as Z  # noqa: E402

Z.use_checked_library()

import torch  # noqa: E402

import test_gpu_train as T  # noqa: E402


def cases():
    for c in T.GRAD_CASES[:9]:
        yield "table_grad", lambda c=c: T.test_table_grad("bf16", 0, *c)
    yield "lookup", lambda: T.test_lookup("fp16", 1023, 503, 768, 0, 45.25, "skewed", torch.int32)
    yield "lookup_odd", lambda: T.test_lookup("bf16", 5, 1000, 257, 3, 3.0, "outside", torch.int64)
    for c in T.WGRAD:
        yield "wgrad", lambda c=c: T.test_weight_gradient("bf16", *c)
    for c in T.POLICY[:9]:
        yield "policy", lambda c=c: T.test_policy_loss(*c)
    for c in T.CKPT_SIZES:
        yield "activation", lambda c=c: T.test_activation_and_its_gradient("fp16", True, *c)


def main():
    Z.zero_selftest_check()
    torch.cuda.synchronize()
    n, first = Z.zero_checked_status()
    print(json.dumps(dict(case="selftest", violations=n, first=first)), flush=True)
    for name, fn in cases():
        fn()
        torch.cuda.synchronize()
        n, first = Z.zero_checked_status()
        print(json.dumps(dict(case=name, violations=n, first=first)), flush=True)


if __name__ == "__main__":
    main()
