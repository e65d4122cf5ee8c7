"""Refusals of the operators in include/zero_train.h: every argument check runs
before any CUDA call, so it works on a host without a GPU. The addresses are
never read."""
import ctypes as C

import pytest

import fsdp_sharded_mixed_shard_gb300 as Z

EINVAL, EALIGN, ERANGE = -1, -2, -3
BF, P = Z.ZERO_BF16, 1024


def refused(status, fn, *args):
    with pytest.raises(Z.ZeroError) as e:
        fn(*args)
    assert e.value.status == status, (fn.__name__, args)


def changed(args, **at):
    """args with the entries named iN replaced."""
    out = list(args)
    for k, v in at.items():
        out[int(k[1:])] = v
    return out


def test_struct_size():
    assert C.sizeof(Z.ZeroPolicyParams) == 24


def test_embedding():
    ok = [P, 4, 10, P, 50, 8, 1.0, BF, P]
    f = Z.zero_embedding
    for bad in (dict(i0=0), dict(i3=0), dict(i8=0), dict(i1=2), dict(i2=-1), dict(i4=-1),
                dict(i5=-1), dict(i7=Z.ZERO_FP32), dict(i7=9)):
        refused(EINVAL, f, *changed(ok, **bad))
    for bad in (dict(i0=P + 2), dict(i3=P + 1), dict(i8=P + 1)):
        refused(EALIGN, f, *changed(ok, **bad))
    refused(EALIGN, f, *changed(ok, i0=P + 4, i1=8))
    refused(ERANGE, f, *changed(ok, i2=(1 << 28) + 1))
    refused(ERANGE, f, *changed(ok, i4=(1 << 24) + 1))
    f(*changed(ok, i2=0, i0=0, i8=0))  # nothing to do


def test_embedding_grad():
    ok = [P, 4, 10, P, 50, 8, 1.0, BF, 0, P, P]
    f = Z.zero_embedding_grad
    for bad in (dict(i0=0), dict(i3=0), dict(i9=0), dict(i10=0), dict(i1=3), dict(i2=-1),
                dict(i4=-1), dict(i5=-1), dict(i7=2), dict(i8=2)):
        refused(EINVAL, f, *changed(ok, **bad))
    for bad in (dict(i0=P + 1), dict(i3=P + 1), dict(i9=P + 1), dict(i10=P + 8)):
        refused(EALIGN, f, *changed(ok, **bad))
    refused(ERANGE, f, *changed(ok, i2=(1 << 28) + 1))
    refused(ERANGE, f, *changed(ok, i4=(1 << 24) + 1))
    f(*changed(ok, i4=0, i9=0, i10=0))
    assert Z.zero_embedding_workspace_bytes(-1, 5, 5) == 0
    assert Z.zero_embedding_workspace_bytes(1 << 29, 5, 5) == 0
    a, b = (Z.zero_embedding_workspace_bytes(n, 1000, 64) for n in (100, 1000))
    assert 0 < a < b and a % 256 == 0


def test_checkpoints():
    assert Z.zero_ckpt_bytes(3, 100) == 3 * (128 + 4)
    assert Z.zero_ckpt_bytes(0, 100) == 0 and Z.zero_ckpt_bytes(2, 0) == 0
    assert Z.zero_ckpt_bytes(-1, 5) == 0 and Z.zero_ckpt_bytes(1 << 61, 1 << 30) == 0
    for f, ok, outer in ((Z.zero_ckpt_save, [P, 4, 100, 104, BF, P], (0, 5)),
                         (Z.zero_ckpt_load, [P, 4, 100, BF, P, 104], (0, 4))):
        dt, ld = (4, 3) if f is Z.zero_ckpt_save else (3, 5)
        for i in outer:
            refused(EINVAL, f, *changed(ok, **{"i%d" % i: 0}))
            refused(EALIGN, f, *changed(ok, **{"i%d" % i: P + 1}))
        refused(EINVAL, f, *changed(ok, **{"i%d" % ld: 99}))
        refused(EINVAL, f, *changed(ok, **{"i%d" % dt: Z.ZERO_FP32}))
        refused(EINVAL, f, *changed(ok, i1=-1))
        refused(EINVAL, f, *changed(ok, i2=-1))
        f(*changed(ok, i1=0))
    gated = [Z.ZERO_ACT_SWIGLU, P, P, 4, 100, 104, BF, P, 104, P, P]
    plain = changed(gated, i0=Z.ZERO_ACT_GELU, i2=0, i10=0)
    f = Z.zero_ckpt_act
    for bad in (dict(i0=2), dict(i1=0), dict(i2=0), dict(i7=0), dict(i9=0), dict(i10=0),
                dict(i3=-1), dict(i5=99), dict(i8=99), dict(i6=2)):
        refused(EINVAL, f, *changed(gated, **bad))
    for bad in (dict(i2=P), dict(i10=P)):
        refused(EINVAL, f, *changed(plain, **bad))
    for bad in (dict(i1=P + 1), dict(i2=P + 1), dict(i7=P + 1), dict(i9=P + 8), dict(i10=P + 8)):
        refused(EALIGN, f, *changed(gated, **bad))
    f(*changed(plain, i3=0))
    gated = [Z.ZERO_ACT_SWIGLU, P, P, P, 4, 100, 104, BF, 2 * P, 3 * P, 0, 104]
    plain = changed(gated, i0=Z.ZERO_ACT_GELU, i2=0, i9=0)
    f = Z.zero_ckpt_act_grad
    for bad in (dict(i0=-1), dict(i1=0), dict(i2=0), dict(i3=0), dict(i8=0), dict(i9=0),
                dict(i6=99), dict(i11=99), dict(i7=2), dict(i8=P, i11=200)):
        refused(EINVAL, f, *changed(gated, **bad))
    for bad in (dict(i2=P), dict(i9=P)):
        refused(EINVAL, f, *changed(plain, **bad))
    for bad in (dict(i1=P + 8), dict(i2=P + 8), dict(i3=P + 1), dict(i8=P + 1), dict(i9=P + 1),
                dict(i10=P + 1)):
        refused(EALIGN, f, *changed(gated, **bad))
    f(*changed(plain, i5=0))


def test_weight_gradient():
    ok = [P, 4, 100, P, 50, 56, BF, P, 0]
    f = Z.zero_ckpt_wgrad
    for bad in (dict(i0=0), dict(i3=0), dict(i7=0), dict(i1=-1), dict(i2=-1), dict(i4=-1),
                dict(i5=49), dict(i6=2)):
        refused(EINVAL, f, *changed(ok, **bad))
    for bad in (dict(i0=P + 8), dict(i3=P + 1), dict(i7=P + 1), dict(i8=P + 8)):
        refused(EALIGN, f, *changed(ok, **bad))
    for bad in (dict(i1=1 << 31), dict(i2=1 << 31), dict(i4=1 << 31, i5=1 << 31)):
        refused(ERANGE, f, *changed(ok, **bad))
    f(*changed(ok, i2=0, i7=0))


def test_loss():
    ok = [P, 4, 100, 104, BF, P, 4, P]
    f = Z.zero_token_logp
    for bad in (dict(i0=0), dict(i5=0), dict(i7=0), dict(i1=-1), dict(i2=0), dict(i3=99),
                dict(i4=3), dict(i6=1)):
        refused(EINVAL, f, *changed(ok, **bad))
    for bad in (dict(i0=P + 1), dict(i5=P + 2), dict(i7=P + 2)):
        refused(EALIGN, f, *changed(ok, **bad))
    refused(EALIGN, f, *changed(ok, i4=Z.ZERO_FP32, i0=P + 2))
    refused(ERANGE, f, *changed(ok, i2=(1 << 30) + 1, i3=1 << 31))
    # a row whose bytes pass 64 bits
    refused(ERANGE, f, *changed(ok, i2=1 << 62, i3=1 << 62, i4=Z.ZERO_FP32))
    f(*changed(ok, i1=0, i0=0, i5=0, i7=0))
    hp = Z.ZeroPolicyParams(0.2, 0.2, 0.1)
    ok = [P, 4, 100, 104, BF, P, 4, P, P, P, P, hp, 0, P, P, P, P]
    f = Z.zero_policy_loss
    for i in (0, 5, 7, 9, 10, 13, 14):
        refused(EINVAL, f, *changed(ok, **{"i%d" % i: 0}))
    for i in (7, 8, 9, 10, 13, 14, 15):
        refused(EALIGN, f, *changed(ok, **{"i%d" % i: P + 2}))
    refused(EALIGN, f, *changed(ok, i16=P + 1))
    refused(EALIGN, f, *changed(ok, i12=P + 4))
    nan, inf = float("nan"), float("inf")
    for lo, hi, beta in ((-0.1, 0.2, 0), (1.0, 0.2, 0), (0.2, -0.1, 0), (0.2, 0.2, -1),
                         (nan, 0.2, 0), (0.2, nan, 0), (0.2, 0.2, nan), (0.2, inf, 0),
                         (0.2, 0.2, inf)):
        refused(EINVAL, f, *changed(ok, i11=Z.ZeroPolicyParams(lo, hi, beta)))
    most = Z.ZERO_MAX_LOGIT_ROW_BYTES // 2
    refused(ERANGE, f, *changed(ok, i2=most + 1, i3=most + 1))


def test_longest_loss_row():
    """A row of exactly ZERO_MAX_LOGIT_ROW_BYTES passes the length check (the
    refusal is a later one), one element more does not."""
    hp = Z.ZeroPolicyParams(0.2, 0.2, 0.1)
    for dt, size in ((BF, 2), (Z.ZERO_FP16, 2), (Z.ZERO_FP32, 4)):
        v = Z.ZERO_MAX_LOGIT_ROW_BYTES // size
        ok = [P, 4, v, v, dt, P, 4, P, P, P, P, hp, 0, P, P + 2, P, P]
        refused(EALIGN, Z.zero_policy_loss, *ok)
        refused(ERANGE, Z.zero_policy_loss, *changed(ok, i2=v + 1, i3=v + 1))


def test_plant_is_refused():
    """Bad arguments, and in the release build every plant."""
    for args in ((-1,), (99,), (Z.ZERO_PLANT_NO_COPY, 0, 0), (Z.ZERO_PLANT_NO_COPY, 0, 10**10)):
        refused(EINVAL, Z.zero_selftest_plant, *args)
    for what in range(Z.ZERO_PLANT_SHORT + 1):
        refused(-6, Z.zero_selftest_plant, what)


def test_weight_gradient_row_distance():
    """A row distance that no tensor map takes is out of range."""
    ok = [P, 4, 100, P, 50, 56, BF, P, 0]
    for ld in (1 << 36, (1 << 36) + 4, 1 << 62):
        refused(ERANGE, Z.zero_ckpt_wgrad, *changed(ok, i5=ld))
