"""Refusals of the operators in include/zero_block.h: every argument check runs
before any CUDA call, so it works on a host without a GPU. The addresses are
never read."""
import ctypes as C

import pytest

import fsdp_sharded_mixed_shard_gb300 as Z
from test_train_abi import EALIGN, EINVAL, ERANGE, changed, refused

BF, P = Z.ZERO_BF16, 4096
NAN, INF = float("nan"), float("inf")


def test_struct_sizes():
    assert C.sizeof(Z.ZeroDropoutParams) == 32
    assert C.sizeof(Z.ZeroJoinParams) == 64
    assert C.sizeof(Z.ZeroJoinWeights) == 40


def drop(p=0.1, step=0):
    return Z.ZeroDropoutParams(p, 1, 2, step)


def test_dropout():
    ok = [drop(), P, 0, 4, 100, 104, BF, 2 * P, 104]
    f = Z.zero_dropout
    for p in (-0.1, 1.0, 1.5, NAN):
        refused(EINVAL, f, *changed(ok, i0=drop(p)))
    for bad in (dict(i1=0), dict(i7=0), dict(i3=-1), dict(i4=-1), dict(i5=99), dict(i8=99),
                dict(i6=Z.ZERO_FP32), dict(i7=P, i8=112)):
        refused(EINVAL, f, *changed(ok, **bad))
    for bad in (dict(i1=P + 1), dict(i2=P + 1), dict(i7=P + 1), dict(i0=drop(step=P + 2))):
        refused(EALIGN, f, *changed(ok, **bad))
    for bad in (dict(i3=1 << 31), dict(i4=1 << 31, i5=1 << 31, i8=1 << 31),
                dict(i3=1 << 24, i4=1 << 16, i5=1 << 16, i8=1 << 16),
                dict(i4=1 << 62, i5=1 << 62, i8=1 << 62)):
        refused(ERANGE, f, *changed(ok, **bad))
    f(*changed(ok, i3=0, i1=0, i7=0))
    f(*changed(ok, i4=0))


def join(norm=Z.ZERO_NORM_LAYER, eps=1e-5, a=1.0, s=1.0, d=None):
    return Z.ZeroJoinParams(norm, eps, a, s, d or drop())


ALL = Z.ZeroJoinWeights(P, P, P, P, P)


def test_join():
    ok = [join(), ALL, P, 2 * P, 4, 100, 104, BF, 3 * P, 4 * P, 5 * P]
    f = Z.zero_block_join
    for j in (join(norm=2), join(norm=-1), join(eps=-1e-9), join(eps=NAN), join(eps=INF),
              join(a=NAN), join(a=INF), join(s=NAN), join(s=-INF), join(d=drop(1.0))):
        refused(EINVAL, f, *changed(ok, i0=j))
    rms = join(norm=Z.ZERO_NORM_RMS)
    for w in (Z.ZeroJoinWeights(0, P, P, P, P), Z.ZeroJoinWeights(P, P, P, 0, P)):
        refused(EINVAL, f, *changed(ok, i1=w))
    for w in (Z.ZeroJoinWeights(P, P, 0, P, 0), Z.ZeroJoinWeights(P, 0, 0, P, P)):
        refused(EINVAL, f, *changed(ok, i0=rms, i1=w))
    for bad in (dict(i2=0), dict(i3=0), dict(i8=0), dict(i9=0), dict(i4=-1), dict(i5=-1),
                dict(i6=99), dict(i7=2), dict(i9=3 * P),
                dict(i1=Z.ZeroJoinWeights(P, P, P, 0, 0))):  # z without its norm
        refused(EINVAL, f, *changed(ok, **bad))
    for i in (2, 3, 8, 9):
        refused(EALIGN, f, *changed(ok, **{"i%d" % i: 7 * P + 1}))
    refused(EALIGN, f, *changed(ok, i10=P + 8))
    refused(EALIGN, f, *changed(ok, i0=join(d=drop(step=P + 1))))
    for k in range(5):
        refused(EALIGN, f, *changed(ok, i1=Z.ZeroJoinWeights(*[P + (j == k) for j in range(5)])))
    refused(ERANGE, f, *changed(ok, i4=1 << 31))
    refused(ERANGE, f, *changed(ok, i5=Z.ZERO_MAX_JOIN_COLS + 1, i6=Z.ZERO_MAX_JOIN_COLS + 1))
    f(*changed(ok, i4=0, i2=0, i3=0, i8=0))
    f(*changed(ok, i5=0))


def test_join_grad():
    ok = [join(), ALL, P, 2 * P, 3 * P, 4 * P, 5 * P, 4, 100, 104, BF, 6 * P, 7 * P, ALL, 8 * P]
    f = Z.zero_block_join_grad
    for bad in (dict(i2=0), dict(i3=0), dict(i4=0), dict(i5=0), dict(i11=0), dict(i12=0),
                dict(i14=0), dict(i7=-1), dict(i8=-1), dict(i9=99), dict(i10=2),
                dict(i0=join(norm=7)), dict(i12=6 * P)):
        refused(EINVAL, f, *changed(ok, **bad))
    for k in range(5):  # a gradient that is asked for and has no place, or the other way round
        one_less = Z.ZeroJoinWeights(*[0 if j == k else P for j in range(5)])
        refused(EINVAL, f, *changed(ok, i13=one_less))
        if k in (1, 2, 4):
            refused(EINVAL, f, *changed(ok, i1=one_less))
    no_pre = Z.ZeroJoinWeights(P, P, P, 0, 0)
    refused(EINVAL, f, *changed(ok, i1=no_pre, i13=no_pre))  # dz without w_pre
    for i in (2, 3, 5, 6, 11, 12):
        refused(EALIGN, f, *changed(ok, **{"i%d" % i: 9 * P + 1}))
    for i in (4, 14):
        refused(EALIGN, f, *changed(ok, **{"i%d" % i: P + 8}))
    for k in range(5):
        refused(EALIGN, f, *changed(ok, i13=Z.ZeroJoinWeights(*[P + (j == k) for j in range(5)])))
    refused(ERANGE, f, *changed(ok, i7=1 << 31))
    refused(ERANGE, f, *changed(ok, i8=Z.ZERO_MAX_JOIN_COLS + 1, i9=1 << 20))
    f(*changed(ok, i8=0))
    w = Z.zero_block_join_workspace_bytes
    assert w(0, 100) == 0 and w(-1, 100) == 0 and w(5, -1) == 0
    assert w(5, Z.ZERO_MAX_JOIN_COLS + 1) == 0 and w(1 << 31, 8) == 0
    assert w(1, 1) == 4 * 8 * 4 and w(1 << 30, 768) == 152 * 4 * 768 * 4


def test_fp8_sizes():
    assert Z.zero_fp8_bytes(3, 100) == 3 * 128 + 512
    assert Z.zero_fp8_bytes(129, 513) == 129 * 640 + 2 * 2 * 512
    assert Z.zero_fp8_weight_bytes(100, 600) == 100 * 640 + (5 * 1 + 1 * 2) * 512
    for f in (Z.zero_fp8_bytes, Z.zero_fp8_weight_bytes):
        assert f(0, 100) == 0 and f(-1, 5) == 0 and f(5, -1) == 0 and f(1 << 31, 5) == 0


def test_fp8_copies():
    f, ok = Z.zero_fp8_quant, [P, 4, 100, 104, BF, Z.ZERO_E5M2, 2 * P]
    for bad in (dict(i0=0), dict(i6=0), dict(i1=-1), dict(i2=-1), dict(i3=99), dict(i4=2),
                dict(i5=2), dict(i5=-1)):
        refused(EINVAL, f, *changed(ok, **bad))
    for bad in (dict(i0=P + 1), dict(i6=P + 8)):
        refused(EALIGN, f, *changed(ok, **bad))
    for bad in (dict(i1=1 << 31), dict(i2=1 << 31, i3=1 << 31),
                dict(i1=1 << 24, i2=1 << 16, i3=1 << 16)):
        refused(ERANGE, f, *changed(ok, **bad))
    f(*changed(ok, i1=0, i0=0))
    f, ok = Z.zero_fp8_quant_weight, [P, 40, 100, BF, 2 * P]
    for bad in (dict(i0=0), dict(i4=0), dict(i1=-1), dict(i2=-1), dict(i3=2)):
        refused(EINVAL, f, *changed(ok, **bad))
    for bad in (dict(i0=P + 1), dict(i4=P + 8)):
        refused(EALIGN, f, *changed(ok, **bad))
    for bad in (dict(i1=1 << 31), dict(i2=1 << 31), dict(i1=1 << 30, i2=1 << 30)):
        refused(ERANGE, f, *changed(ok, **bad))
    f(*changed(ok, i1=0, i0=0, i4=0))


@pytest.mark.parametrize("f,n", [(Z.zero_fp8_linear, 100), (Z.zero_fp8_linear_dgrad, 40)])
def test_fp8_products(f, n):
    ok = [P, Z.ZERO_E4M3, 4, 2 * P, 40, 100, BF, 3 * P, 104, 0]
    for bad in (dict(i0=0), dict(i3=0), dict(i7=0), dict(i1=2), dict(i1=-1), dict(i2=-1),
                dict(i4=-1), dict(i5=-1), dict(i6=2), dict(i8=n - 1)):
        refused(EINVAL, f, *changed(ok, **bad))
    for bad in (dict(i0=P + 8), dict(i3=P + 8), dict(i7=P + 1), dict(i9=P + 8)):
        refused(EALIGN, f, *changed(ok, **bad))
    for bad in (dict(i2=1 << 30), dict(i4=1 << 30, i8=1 << 32), dict(i5=1 << 30, i8=1 << 32)):
        refused(ERANGE, f, *changed(ok, **bad))
    f(*changed(ok, i2=0, i0=0, i3=0, i7=0))
