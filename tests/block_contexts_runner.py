"""Runs the operators of include/zero_block.h in two contexts of one device, one
after the other and then in turn, in a third, and in the device's primary context
before and after a reset of it; prints one JSON line per run: each output's checksum.
Driver calls only (no torch), so that nothing else makes a context or lives in one.
Used by tests/test_gpu_block_contexts.py."""
import ctypes as C
import hashlib
import json
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fsdp_sharded_mixed_shard_gb300 as Z  # noqa: E402

cuda = C.CDLL("libcuda.so.1")
BF = Z.ZERO_BF16


def ok(status):
    if status:
        raise RuntimeError("driver error %d" % status)


class Context:
    def __init__(self, device):
        self.h = C.c_void_p()
        ok(cuda.cuCtxCreate_v2(C.byref(self.h), 0, device))  # and makes it current
        self.mem = []

    def enter(self):
        ok(cuda.cuCtxSetCurrent(self.h))

    def buffer(self, n, host=None):
        p = C.c_uint64()
        ok(cuda.cuMemAlloc_v2(C.byref(p), C.c_size_t(n)))
        ok(cuda.cuMemsetD8_v2(p, C.c_ubyte(0), C.c_size_t(n)))
        if host is not None:
            assert host.nbytes <= n
            ok(cuda.cuMemcpyHtoD_v2(p, host.ctypes.data_as(C.c_void_p), C.c_size_t(host.nbytes)))
        self.mem.append(p)
        return p.value

    def read(self, p, n):
        out = np.empty(n, np.uint8)
        ok(cuda.cuMemcpyDtoH_v2(out.ctypes.data_as(C.c_void_p), C.c_uint64(p), C.c_size_t(n)))
        return out

    def free(self):
        for p in self.mem:
            ok(cuda.cuMemFree_v2(p))
        self.mem = []

    def close(self):
        self.free()
        ok(cuda.cuCtxDestroy_v2(self.h))


class Primary(Context):
    """The device's own context, as the CUDA runtime uses it."""

    def __init__(self, device):
        self.h, self.device, self.mem = C.c_void_p(), device, []
        ok(cuda.cuDevicePrimaryCtxRetain(C.byref(self.h), device))

    def reset(self):
        self.free()
        ok(cuda.cuDevicePrimaryCtxReset_v2(self.device))
        ok(cuda.cuDevicePrimaryCtxRetain(C.byref(self.h), self.device))


def bf16(rng, n, sd=1.0):
    """n normal numbers' upper 16 bits"""
    x = (rng.standard_normal(n) * sd).astype(np.float32)
    return (x.view(np.uint32) >> 16).astype(np.uint16)


def run(ctx):
    ctx.enter()
    rng = np.random.default_rng(5)
    sums = {}

    def keep(name, p, n):
        ok(cuda.cuCtxSynchronize())
        sums[name] = hashlib.sha1(ctx.read(p, n).tobytes()).hexdigest()

    # many tiles, and a reduction split over a cluster of 16 CTAs
    for rows, k, n in ((600, 512, 640), (16, 8192, 256)):
        x = ctx.buffer(2 * rows * k, bf16(rng, rows * k))
        w = ctx.buffer(2 * k * n, bf16(rng, k * n, 0.02))
        dy = ctx.buffer(2 * rows * n, bf16(rng, rows * n))
        x8, w8, dy8 = (ctx.buffer(b) for b in (
            Z.zero_fp8_bytes(rows, k), Z.zero_fp8_weight_bytes(k, n), Z.zero_fp8_bytes(rows, n)))
        y, dx = ctx.buffer(2 * rows * n), ctx.buffer(2 * rows * k)
        Z.zero_fp8_quant_weight(w, k, n, BF, w8)
        Z.zero_fp8_quant(x, rows, k, k, BF, 0, x8)
        Z.zero_fp8_linear(x8, 0, rows, w8, k, n, BF, y, n)
        Z.zero_fp8_quant(dy, rows, n, n, BF, 1, dy8)
        Z.zero_fp8_linear_dgrad(dy8, 1, rows, w8, k, n, BF, dx, k)
        keep("y %d" % rows, y, 2 * rows * n)
        keep("dx %d" % rows, dx, 2 * rows * k)
    for rows, cols in ((50, 768), (700, 8192)):
        h, y, dz, up = (ctx.buffer(2 * rows * cols, bf16(rng, rows * cols)) for _ in range(4))
        h_out, z, dh, dv = (ctx.buffer(2 * rows * cols) for _ in range(4))
        w = Z.ZeroJoinWeights(*[ctx.buffer(2 * cols, bf16(rng, cols)) for _ in range(5)])
        g = [ctx.buffer(2 * cols) for _ in range(5)]
        stats = ctx.buffer(16 * rows)
        work = ctx.buffer(Z.zero_block_join_workspace_bytes(rows, cols))
        p = Z.ZeroJoinParams(Z.ZERO_NORM_LAYER, 1e-5, 1.0, 0.5, Z.ZeroDropoutParams(0.1, 1, 2, 0))
        Z.zero_block_join(p, w, h, y, rows, cols, cols, BF, h_out, z, stats)
        Z.zero_block_join_grad(p, w, h_out, y, stats, dz, up, rows, cols, cols, BF, dh, dv,
                               Z.ZeroJoinWeights(*g), work)
        for name, t in (("h_out", h_out), ("z", z), ("dh", dh), ("dy", dv)):
            keep("%s %d" % (name, cols), t, 2 * rows * cols)
        for k in range(5):
            keep("gradient %d %d" % (k, cols), g[k], 2 * cols)
        Z.zero_dropout(p.drop, h, y, rows, cols, cols, BF, z, cols)
        keep("dropout %d" % cols, z, 2 * rows * cols)
    ctx.free()
    return sums


def main():
    ok(cuda.cuInit(0))
    device = C.c_int()
    ok(cuda.cuDeviceGet(C.byref(device), 0))
    first = Context(device)
    line = lambda what, sums: print(json.dumps(dict(run=what, sums=sums)), flush=True)  # noqa: E731
    line("first", run(first))
    second = Context(device)
    line("second", run(second))
    line("first again", run(first))
    first.enter()
    first.close()
    line("second again", run(second))
    second.close()
    third = Context(device)
    line("third", run(third))
    third.close()
    primary = Primary(device)
    line("primary", run(primary))
    primary.reset()
    line("primary after a reset", run(primary))


if __name__ == "__main__":
    main()
