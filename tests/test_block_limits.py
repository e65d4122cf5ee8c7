"""Refusals of zero_block_join and zero_block_join_grad at the limits of what they
compute in (fp32), on a host without a GPU. The addresses are never read."""
import pytest

import fsdp_sharded_mixed_shard_gb300 as Z
from test_block_abi import ALL, BF, P, join
from test_train_abi import EINVAL, ERANGE, changed, refused

FORWARD = [join(), ALL, P, 2 * P, 4, 100, 104, BF, 3 * P, 4 * P, 5 * P]
BACK = [join(), ALL, P, 2 * P, 3 * P, 4 * P, 5 * P, 4, 100, 104, BF, 6 * P, 7 * P, ALL, 8 * P]
CALLS = [(Z.zero_block_join, FORWARD), (Z.zero_block_join_grad, BACK)]
LEAST, MOST = 2.0 ** -126, 2.0 ** 128 * (1 - 2.0 ** -24)  # of fp32's normal numbers


@pytest.mark.parametrize("f,ok", CALLS)
def test_scales_past_fp32(f, ok):
    for x in (1e39, -1e39, 1e300, 2.0 ** 128):
        refused(EINVAL, f, *changed(ok, i0=join(a=x)))
        refused(EINVAL, f, *changed(ok, i0=join(s=x)))


@pytest.mark.parametrize("f,ok", CALLS)
def test_eps_past_fp32(f, ok):
    for eps in (1e39, 1e300, 1e-39, 1e-60, 5e-324, LEAST * (1 - 2.0 ** -20)):
        refused(EINVAL, f, *changed(ok, i0=join(eps=eps)))


@pytest.mark.parametrize("f,ok", CALLS)
def test_what_fp32_holds_is_taken(f, ok):
    """Such calls go on to the next refusal (too many columns)."""
    wide = dict(i5=8193, i6=8193) if f is Z.zero_block_join else dict(i8=8193, i9=8193)
    for j in (join(a=MOST), join(s=-MOST), join(a=1e-60), join(s=0.0), join(eps=0.0),
              join(eps=LEAST), join(eps=MOST)):
        refused(ERANGE, f, *changed(ok, i0=j, **wide))


def test_no_norm_needs_no_statistics():
    """Without w_post and w_pre the gradient goes past its check of stats, with
    either of them not: seen by the refusal that comes after it (a misaligned dh)."""
    f = Z.zero_block_join_grad
    gate = Z.ZeroJoinWeights(0, 0, P, 0, 0)
    rest = dict(i4=0, i11=6 * P + 1)
    refused(-2, f, *changed(BACK, i1=gate, i13=gate, i5=0, **rest))
    for w in (Z.ZeroJoinWeights(P, 0, 0, 0, 0), Z.ZeroJoinWeights(0, 0, 0, P, 0)):
        dz = 0 if w.w_post else 4 * P
        refused(EINVAL, f, *changed(BACK, i1=w, i13=w, i5=dz, **rest))
