"""The operators of include/zero_train.h on a GB300 against plain 64-bit
implementations: embedding and its table gradient, 8-bit activation
checkpoints and their uses, token log-probabilities and the clipped policy
loss. Bounds are derived in tests/train_util.py and at each test."""
import math

import pytest
import torch

import fsdp_sharded_mixed_shard_gb300 as Z
from train_util import (DT, TINY, U, ZT, act64, act_bound, act_grad64, act_grad_bounds, ckpt64,
                        logp_bound, offset_rows, policy64, rand, split_ckpt, within)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def stream():
    return torch.cuda.current_stream().cuda_stream


def ids(kind, rows, vocab, seed, dtype=torch.int32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if kind == "uniform":
        t = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    elif kind == "one":           # every token the same id
        t = torch.full((rows,), vocab // 2, device="cuda")
    elif kind == "ends":          # only the first and last rows of the table
        t = torch.randint(0, 2, (rows,), generator=g, device="cuda") * (vocab - 1)
    elif kind == "skewed":        # a few frequent ids, a long tail, some padding
        u = torch.rand(rows, generator=g, device="cuda", dtype=torch.float64)
        t = (torch.exp(u * math.log(vocab)) - 1).long().clamp(0, vocab - 1)
        t[torch.rand(rows, generator=g, device="cuda") < 0.1] = -1
    elif kind == "outside":       # ids below 0 and at or past vocab
        t = torch.randint(-3, vocab + 3, (rows,), generator=g, device="cuda")
    elif kind == "padding":
        t = torch.full((rows,), -1, device="cuda")
    return t.to(dtype)


# --------------------------------------------------------------- embedding ----

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,vocab,dim,shift,scale,kind,idt", [
    (1, 7, 8, 0, 1.0, "uniform", torch.int32),
    (1, 1, 1, 1, 0.5, "uniform", torch.int64),
    (5, 1000, 257, 3, 3.0, "outside", torch.int64),
    (1023, 503, 768, 0, 45.25, "skewed", torch.int32),
    (130, 503, 768, 5, 1.0, "uniform", torch.int32),
    (64, 31, 2048, 8, 1.0, "outside", torch.int32),
])
def test_lookup(dtype, rows, vocab, dim, shift, scale, kind, idt):
    """round16(fl32(scale x)): two roundings, u (1 + 2^-12)."""
    _, table = offset_rows(vocab, dim, dim, dtype, shift)
    table.copy_(rand((vocab, dim), dtype, 3, 0.5))
    tok = ids(kind, rows, vocab, 4, idt)
    whole, out = offset_rows(rows, dim, dim, dtype, shift)
    Z.zero_embedding(tok.data_ptr(), tok.element_size(), rows, table.data_ptr(), vocab, dim, scale,
                     ZT[dtype], out.data_ptr(), stream())
    ok = (tok >= 0) & (tok < vocab)
    want = scale * table[tok.long().clamp(0, vocab - 1)].double() * ok[:, None]
    within(out, want, U[dtype] * (1 + 2.0 ** -12) * want.abs() + TINY[dtype], "lookup")
    assert (out[~ok] == 0).all()
    assert (whole[:shift] == 7).all() and (whole[shift + rows * dim:] == 7).all()


def run_grad(tok, dy, vocab, dim, scale, dtype, accumulate, grad):
    n = Z.zero_embedding_workspace_bytes(tok.numel(), vocab, dim)
    work = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    Z.zero_embedding_grad(tok.data_ptr(), tok.element_size(), tok.numel(), dy.data_ptr(), vocab,
                          dim, scale, ZT[dtype], accumulate, grad.data_ptr(), work.data_ptr(),
                          stream())


GRAD_CASES = [
    # rows, vocab, dim, shift, kind, id type
    (0, 37, 40, 0, "uniform", torch.int32),
    (1, 1, 8, 0, "uniform", torch.int32),
    (1, 503, 256, 0, "uniform", torch.int64),
    (300, 11, 264, 0, "uniform", torch.int32),
    (1000, 503, 257, 1, "outside", torch.int64),
    (4097, 1000, 128, 0, "skewed", torch.int32),
    (777, 50257, 64, 0, "skewed", torch.int32),
    (2048, 300, 520, 0, "one", torch.int32),
    (513, 262145, 8, 0, "ends", torch.int32),     # three counting passes
    (1500, 128256, 33, 3, "uniform", torch.int32),
    (64, 64, 2048, 0, "padding", torch.int32),
    (70_000, 700, 16, 0, "skewed", torch.int32),  # several tiles per chunk
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("accumulate", [0, 1])
@pytest.mark.parametrize("rows,vocab,dim,shift,kind,idt", GRAD_CASES)
def test_table_grad(dtype, accumulate, rows, vocab, dim, shift, kind, idt):
    """fp32 sums of n_v terms: (n_v + 2) 2^-24 sum |dy| beside the rounding."""
    tok = ids(kind, rows, vocab, 5, idt)
    _, dy = offset_rows(rows, dim, dim, dtype, shift)
    dy.copy_(rand((rows, dim), dtype, 6, 0.25))
    whole, grad = offset_rows(vocab, dim, dim, dtype, shift)
    before = rand((vocab, dim), dtype, 7, 0.25)
    grad.copy_(before)
    scale = 1.5
    run_grad(tok, dy, vocab, dim, scale, dtype, accumulate, grad)
    ok = (tok >= 0) & (tok < vocab)
    at = tok[ok].long()
    zero = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda")
    want = zero.index_add(0, at, scale * dy[ok].double())
    mag = zero.index_add(0, at, scale * dy[ok].double().abs())
    count = torch.bincount(at, minlength=vocab).double()[:, None]
    if accumulate:
        want, mag = want + before.double(), mag + before.double().abs()
    within(grad, want, U[dtype] * want.abs() + (count + 3) * 2.0 ** -24 * mag + TINY[dtype],
           "table gradient")
    if accumulate:
        untouched = count.squeeze(1) == 0
        assert torch.equal(grad[untouched], before[untouched])
    assert (whole[:shift] == 7).all() and (whole[shift + vocab * dim:] == 7).all()


def test_table_grad_is_the_same_every_time():
    tok = ids("skewed", 9000, 2000, 8)
    dy = rand((9000, 264), "bf16", 9)
    got = []
    for _ in range(4):
        grad = torch.empty(2000, 264, dtype=torch.bfloat16, device="cuda")
        run_grad(tok, dy, 2000, 264, 1.0, "bf16", 0, grad)
        got.append(grad)
    assert all(torch.equal(g, got[0]) for g in got)


def test_table_grad_against_differences():
    """The lookup is linear: <lookup(E + V) - lookup(E), dy> = <V, grad>. Small
    whole numbers keep both sides exact."""
    rows, vocab, dim = 200, 50, 24
    tok = ids("skewed", rows, vocab, 10)
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    whole = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    e, v, dy = whole(vocab, dim), whole(vocab, dim), whole(rows, dim)
    outs = []
    for table in (e + v, e):
        out = torch.empty(rows, dim, dtype=torch.bfloat16, device="cuda")
        Z.zero_embedding(tok.data_ptr(), 4, rows, table.data_ptr(), vocab, dim, 1.0, Z.ZERO_BF16,
                         out.data_ptr(), stream())
        outs.append(out.double())
    grad = torch.empty(vocab, dim, dtype=torch.bfloat16, device="cuda")
    run_grad(tok, dy, vocab, dim, 1.0, "bf16", 0, grad)
    # the most frequent id's sums stay below 256, where bf16 holds whole numbers
    assert grad.double().abs().max() < 256
    assert ((outs[0] - outs[1]) * dy.double()).sum() == (v.double() * grad.double()).sum()


# ------------------------------------------------------------- checkpoints ----

def spread(rows, cols, dtype, seed):
    """Values over many binades, with zeros, an all-zero block, powers of two
    and values on the 127.5-step edge."""
    x = rand((rows, cols), dtype, seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    top = 14 if dtype == "fp16" else 120
    k = torch.randint(-top, top, (rows, -(-cols // 32)), generator=g, device="cuda")
    x = torch.ldexp(x.double(), k.repeat_interleave(32, 1)[:, :cols]).to(DT[dtype])
    if rows > 1:
        x[0] = 0
        x[1, ::2] = 1.0
        x[1, 1::2] = -1.9921875  # 127.5 steps of 2^-6
    return x


CKPT_SIZES = [(1, 1, 1, 0), (1, 32, 32, 0), (3, 33, 33, 1), (2, 128, 128, 0), (17, 130, 130, 2),
              (9, 257, 300, 3), (33, 768, 768, 0), (5, 2050, 2050, 0), (40, 1000, 1008, 8)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,cols,ld,shift", CKPT_SIZES)
def test_ckpt_save_and_load_are_exact(dtype, rows, cols, ld, shift):
    _, x = offset_rows(rows, cols, ld, dtype, shift, fill=float("nan"))
    x.copy_(spread(rows, cols, dtype, 20))
    n = Z.zero_ckpt_bytes(rows, cols)
    buf = torch.full((n + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    Z.zero_ckpt_save(x.data_ptr(), rows, cols, ld, ZT[dtype], buf.data_ptr(), stream())
    q, scale = split_ckpt(buf, rows, cols)
    wq, ws, wv = ckpt64(x)
    assert torch.equal(q, wq) and torch.equal(scale, ws)
    assert (buf[n:] == 0x5A).all()
    whole, out = offset_rows(rows, cols, ld, dtype, shift)
    Z.zero_ckpt_load(buf.data_ptr(), rows, cols, ZT[dtype], out.data_ptr(), ld, stream())
    assert torch.equal(out.double(), wv)
    rest = torch.ones_like(whole, dtype=torch.bool)
    rest[shift:shift + rows * ld].view(rows, ld)[:, :cols] = False
    assert (whole[rest] == 7).all()
    # the stated error: 2^-7 of the block's largest magnitude
    pad = torch.zeros(rows, -(-cols // 32) * 32, dtype=torch.float64, device="cuda")
    pad[:, :cols] = x.double()
    top = pad.view(rows, -1, 32).abs().amax(2, keepdim=True)
    err = pad.clone()
    err[:, :cols] -= wv
    assert (err.view(rows, -1, 32).abs() <= 2.0 ** -7 * top + 2.0 ** -24).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_ckpt_of_the_types_extremes(dtype):
    big, small = torch.finfo(DT[dtype]).max, TINY[dtype]
    x = torch.zeros(4, 64, dtype=DT[dtype], device="cuda")
    x[0, :32], x[0, 32:] = big, -big
    x[1, 0], x[1, 40] = small, -small
    x[2, 3], x[2, 35] = float("inf"), float("nan")
    x[2, 4] = 5.0
    x[3, 0], x[3, 1], x[3, 33] = big, small, float("-inf")
    buf = torch.zeros(Z.zero_ckpt_bytes(4, 64), dtype=torch.uint8, device="cuda")
    Z.zero_ckpt_save(x.data_ptr(), 4, 64, 64, ZT[dtype], buf.data_ptr(), stream())
    q, scale = split_ckpt(buf, 4, 64)
    wq, ws, wv = ckpt64(x)
    assert torch.equal(q, wq) and torch.equal(scale, ws)
    out = torch.empty_like(x)
    Z.zero_ckpt_load(buf.data_ptr(), 4, 64, ZT[dtype], out.data_ptr(), 64, stream())
    assert torch.isnan(out[2]).all() and torch.isnan(out[3, 32:]).all()
    fine = torch.isfinite(wv)
    assert torch.equal(out[fine].double(), wv[fine])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,cols,ld,shift", CKPT_SIZES)
def test_activation_and_its_gradient(dtype, gated, rows, cols, ld, shift):
    act = Z.ZERO_ACT_SWIGLU if gated else Z.ZERO_ACT_GELU
    def place(t):
        _, v = offset_rows(rows, cols, ld, dtype, shift)
        return v.copy_(t)
    x = place(rand((rows, cols), dtype, 30, 3.0))
    u = place(rand((rows, cols), dtype, 31, 2.0)) if gated else None
    dy = place(rand((rows, cols), dtype, 32, 0.5))
    n = Z.zero_ckpt_bytes(rows, cols)
    kx = torch.empty(n, dtype=torch.uint8, device="cuda")
    ku = torch.empty(n, dtype=torch.uint8, device="cuda") if gated else None
    ptr = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
    wy, y = offset_rows(rows, cols, ld, dtype, shift)
    Z.zero_ckpt_act(act, x.data_ptr(), ptr(u), rows, cols, ld, ZT[dtype], y.data_ptr(), ld,
                    kx.data_ptr(), ptr(ku), stream())
    x64, u64 = x.double(), None if u is None else u.double()
    within(y, act64(act, x64, u64), act_bound(act, x64, u64, dtype), "y")
    for t, k in ((x, kx), (u, ku)):
        if t is not None:
            q, s = split_ckpt(k, rows, cols)
            wq, ws, _ = ckpt64(t)
            assert torch.equal(q, wq) and torch.equal(s, ws)
    wx, dx = offset_rows(rows, cols, ld, dtype, shift)
    _, du = offset_rows(rows, cols, ld, dtype, shift)
    _, h = offset_rows(rows, cols, ld, dtype, shift)
    Z.zero_ckpt_act_grad(act, kx.data_ptr(), ptr(ku), dy.data_ptr(), rows, cols, ld, ZT[dtype],
                         dx.data_ptr(), du.data_ptr() if gated else 0, h.data_ptr(), ld, stream())
    xq = ckpt64(x)[2]
    uq = ckpt64(u)[2] if gated else None
    d = dy.double()
    want_x, want_u = act_grad64(act, xq, uq, d)
    bx, bu = act_grad_bounds(act, xq, uq, d, dtype)
    within(dx, want_x, bx, "dx")
    if gated:
        within(du, want_u, bu, "du")
    within(h, act64(act, xq, uq), act_bound(act, xq, uq, dtype), "h")
    for whole in (wy, wx):
        rest = torch.ones_like(whole, dtype=torch.bool)
        rest[shift:shift + rows * ld].view(rows, ld)[:, :cols] = False
        assert (whole[rest] == 7).all()
    # differences of the 64-bit activation at the checkpointed values: h = 2^-14,
    # third derivatives of both functions stay below 4
    eps = 2.0 ** -14
    diff = (act64(act, xq + eps, uq) - act64(act, xq - eps, uq)) / (2 * eps) * d
    um = 1.0 if uq is None else uq.abs()
    within(dx, diff, bx + d.abs() * um * (4 * eps * eps + 1e-9), "dx against differences")
    # in place of dy, without the activation again
    Z.zero_ckpt_act_grad(act, kx.data_ptr(), ptr(ku), dy.data_ptr(), rows, cols, ld, ZT[dtype],
                         dy.data_ptr(), du.data_ptr() if gated else 0, 0, ld, stream())
    assert torch.equal(dy, dx)


@pytest.mark.parametrize("gated", [False, True])
def test_activation_far_out(gated):
    """Large magnitudes end in 0 or the value itself, not in NaN, and a block
    with a NaN gives NaN gradients."""
    act = Z.ZERO_ACT_SWIGLU if gated else Z.ZERO_ACT_GELU
    x = torch.zeros(1, 128, dtype=torch.bfloat16, device="cuda")
    x[0, :32], x[0, 32:64], x[0, 64:96] = 1e25, -1e25, -100.0
    x[0, 96] = float("nan")
    u = torch.full_like(x, 2.0)
    dy = torch.ones_like(x)
    n = Z.zero_ckpt_bytes(1, 128)
    kx, ku = (torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    y, dx, du = (torch.empty_like(x) for _ in range(3))
    g = lambda t: t.data_ptr() if gated else 0  # noqa: E731
    Z.zero_ckpt_act(act, x.data_ptr(), g(u), 1, 128, 128, Z.ZERO_BF16, y.data_ptr(), 128,
                    kx.data_ptr(), g(ku), stream())
    Z.zero_ckpt_act_grad(act, kx.data_ptr(), g(ku), dy.data_ptr(), 1, 128, 128, Z.ZERO_BF16,
                         dx.data_ptr(), g(du), 0, 128, stream())
    f = 2.0 if gated else 1.0
    assert torch.equal(y[0, :32], x[0, :32] * f) and (y[0, 32:64] == 0).all()
    assert (y[0, 64:96].abs() < 1e-30).all() and torch.isnan(y[0, 96])
    assert (dx[0, :32] == f).all() and (dx[0, 32:64] == 0).all()
    assert (dx[0, 64:96].abs() < 1e-30).all() and torch.isnan(dx[0, 96:]).all()


# ----------------------------------------------------------- weight gradient --

WGRAD = [
    # rows, cols, n, ld, shift of dy and dw
    (1, 1, 1, 1, 0), (1, 128, 256, 256, 0), (7, 33, 17, 17, 0), (64, 128, 256, 256, 0),
    (65, 130, 264, 264, 0), (63, 127, 250, 251, 1), (300, 768, 520, 520, 0),
    (129, 257, 72, 80, 8), (1000, 96, 40, 40, 0), (2048, 128, 256, 256, 0),
    (4100, 64, 64, 64, 0), (511, 640, 777, 777, 0), (128, 1024, 2304, 2304, 0),
    (96, 200, 256, 512, 0), (33, 64, 8, 8, 4), (2000, 300, 24, 32, 0),
]


def run_wgrad(x, dy, ld, dtype, dw, scaler=0):
    rows, cols = x.shape
    ck = torch.empty(Z.zero_ckpt_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    Z.zero_ckpt_save(x.data_ptr(), rows, cols, cols, ZT[dtype], ck.data_ptr(), stream())
    Z.zero_ckpt_wgrad(ck.data_ptr(), rows, cols, dy.data_ptr(), dy.shape[1], ld, ZT[dtype],
                      dw.data_ptr(), scaler, stream())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,cols,n,ld,shift", WGRAD)
def test_weight_gradient(dtype, rows, cols, n, ld, shift):
    """Products of two 16-bit values are exact in fp32; rows additions that may
    truncate: (rows + 4) 2^-23 sum |x y| beside the rounding. And in the norm,
    where the additions' errors average out: 2 u."""
    x = rand((rows, cols), dtype, 40)
    _, dy = offset_rows(rows, n, ld, dtype, shift)
    dy.copy_(rand((rows, n), dtype, 41, 0.125))
    whole, dw = offset_rows(cols, n, n, dtype, shift)
    run_wgrad(x, dy, ld, dtype, dw)
    xq = ckpt64(x)[2]
    want = xq.t() @ dy.double()
    mag = xq.abs().t() @ dy.double().abs()
    within(dw, want, U[dtype] * want.abs() + (rows + 4) * 2.0 ** -23 * mag + TINY[dtype], "dw")
    assert (dw.double() - want).norm() <= 2 * U[dtype] * want.norm()
    assert (whole[:shift] == 7).all() and (whole[shift + cols * n:] == 7).all()
    again = torch.empty_like(dw.contiguous())
    run_wgrad(x, dy, ld, dtype, again)
    assert shift or torch.equal(again, dw)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,cols,n,ld,shift", [
    (2000, 2048, 4100, 4101, 3), (2000, 2048, 4096, 4104, 0),    # two column groups per tile
    (5, 40, 33, 35, 1), (1, 64, 9, 9, 1), (7, 32, 130, 132, 6),  # fewer tokens than row distances
    (73, 64, 140, 142, 2), (90, 64, 300, 304, 5),                # 4 of them, and 1
    (8192, 100, 101, 101, 0), (8190, 64, 96, 104, 0),            # tokens split eight ways
])
def test_weight_gradient_layouts(dtype, rows, cols, n, ld, shift):
    test_weight_gradient(dtype, rows, cols, n, ld, shift)


def test_weight_gradient_reads_its_own_rows():
    """NaN in every element around dy's rows, which share their blocks, stays out."""
    rows, cols, n, ld = 75, 64, 149, 151
    x = rand((rows, cols), "bf16", 46)
    whole, dy = offset_rows(rows, n, ld, "bf16", 3)
    whole.fill_(float("nan"))
    dy.copy_(rand((rows, n), "bf16", 47))
    dw = torch.empty(cols, n, dtype=torch.bfloat16, device="cuda")
    run_wgrad(x, dy, ld, "bf16", dw)
    assert torch.isfinite(dw).all()


def test_weight_gradient_exact_on_whole_numbers():
    """Whole numbers small enough that every partial sum is exact, so any tile,
    step or split that is dropped, doubled or misplaced shows."""
    rows, cols, n = 700, 200, 330
    g = torch.Generator(device="cuda")
    g.manual_seed(42)
    x = torch.randint(-2, 3, (rows, cols), generator=g, device="cuda").to(torch.float16)
    x[:, ::32] = 100.0  # steps of 1
    dy = torch.zeros(rows, n, dtype=torch.float16, device="cuda")
    pick = torch.randint(0, rows, (4, n), generator=g, device="cuda")
    for k in range(4):
        dy[pick[k], torch.arange(n, device="cuda")] += 1.0
    dw = torch.empty(cols, n, dtype=torch.float16, device="cuda")
    run_wgrad(x, dy, n, "fp16", dw)
    assert torch.equal(dw.double(), x.double().t() @ dy.double())


def test_weight_gradient_edges():
    dw = torch.full((40, 24), 7.0, dtype=torch.bfloat16, device="cuda")
    Z.zero_ckpt_wgrad(0, 0, 40, 0, 24, 24, Z.ZERO_BF16, dw.data_ptr(), 0, stream())
    assert (dw == 0).all()  # no tokens: a gradient of zeros
    # a NaN block poisons its columns' sums alone; an inf in dy its own column
    x = rand((50, 96), "bf16", 43)
    x[7, 40] = float("nan")
    dy = rand((50, 24), "bf16", 44)
    dy[3, 5] = float("inf")
    dw = torch.empty(96, 24, dtype=torch.bfloat16, device="cuda")
    run_wgrad(x, dy, 24, "bf16", dw)
    bad = ~torch.isfinite(dw)
    assert torch.isnan(dw[32:64]).all() and bad[:, 5].all()
    rest = bad.clone()
    rest[32:64] = False
    rest[:, 5] = False
    assert not rest.any()


# -------------------------------------------------------------------- loss ----

def run_policy(x, ld, dtype, act, old, ref, adv, w, hp, scaler, dl, want_stats=True):
    rows, v = x.shape
    lp, loss = (torch.full((rows,), 9.0, device="cuda") for _ in range(2))
    stats = torch.full((4,), 9.0, device="cuda")
    Z.zero_policy_loss(x.data_ptr(), rows, v, ld, ZT[dtype], act.data_ptr(), act.element_size(),
                       old.data_ptr(), 0 if ref is None else ref.data_ptr(), adv.data_ptr(),
                       w.data_ptr(), hp, 0 if scaler is None else scaler.data_ptr(), lp.data_ptr(),
                       loss.data_ptr(), stats.data_ptr() if want_stats else 0,
                       0 if dl is None else dl.data_ptr(), stream())
    return lp, loss, stats


def policy_inputs(rows, v, ld, dtype, shift, seed, idt=torch.int32):
    whole, x = offset_rows(rows, v, ld, dtype, shift)
    x.copy_(rand((rows, v), dtype, seed, 2.5))
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    act = torch.randint(0, v, (rows,), generator=g, device="cuda")
    lp = x.double().log_softmax(1).gather(1, act[:, None]).squeeze(1)
    rnd = lambda: torch.randn(rows, generator=g, device="cuda", dtype=torch.float64)  # noqa: E731
    d = 0.2 * rnd()
    for edge in (math.log(0.8), math.log(1.25)):  # not on a clip edge
        d = torch.where((d - edge).abs() < 1e-3, torch.full_like(d, edge + 2e-3), d)
    old, ref, adv = (lp - d).float(), (lp + 0.5 * rnd()).float(), rnd().float()
    w = torch.rand(rows, generator=g, device="cuda")
    w[::3] = 0
    if rows == 1:
        w[0] = 0.5
    return whole, x, act.to(idt), old, ref, adv, w


POLICY = [
    # rows, vocab, ld, shift, type
    (1, 1, 1, 0, "fp32"), (1, 50257, 50257, 0, "bf16"), (3, 7, 7, 1, "fp16"),
    (4, 33, 40, 0, "bf16"), (5, 1000, 1000, 0, "fp32"), (9, 1001, 1001, 3, "fp16"),
    (2, 128256, 128256, 0, "bf16"), (7, 5003, 5003, 1, "fp32"), (700, 257, 257, 0, "bf16"),
    (330, 4099, 4104, 5, "fp16"), (3, 262144, 262144, 0, "fp32"), (400, 32000, 32000, 0, "bf16"),
    (40, 50257, 50257, 7, "fp16"), (5, 786368, 786368, 0, "bf16"),
]


@pytest.mark.parametrize("rows,v,ld,shift,dtype", POLICY)
def test_policy_loss(rows, v, ld, shift, dtype):
    whole, x, act, old, ref, adv, w = policy_inputs(rows, v, ld, dtype, shift, 50 + rows)
    hp = Z.ZeroPolicyParams(0.2, 0.25, 0.1)
    scaler = torch.zeros(20, device="cuda")
    scaler[0] = 256.0
    wd, dl = offset_rows(rows, v, ld, dtype, shift)
    lp, loss, stats = run_policy(x, ld, dtype, act, old, ref, adv, w, hp, scaler, dl)
    elp, eloss, estats, eg, lse, p, on = policy64(x, act, old, ref, adv, w, 0.2, 0.25, 0.1, 256.0)
    b = logp_bound(x, act, lse)
    within(lp, elp, torch.where(on, b, torch.zeros_like(b)), "logp")
    # loss and slope: r and exp(d) carry logp's error and their own 2^-21
    r, ed = (elp - old.double()).exp(), (ref.double() - elp).exp()
    delta = b + 2.0 ** -21
    bl = (r * adv.double().abs() + 0.1 * (ed + 1 + (ref.double() - elp).abs())) * 2 * delta
    within(loss, eloss, torch.where(on, bl, torch.zeros_like(bl)), "loss")
    ww = w.double() * on
    within(stats, estats, torch.stack([(ww * bl).sum(), (ww * (ed + 1) * 2 * delta).sum(),
                                       0 * b.sum(), 0 * b.sum()]) + 1e-6 * ww.sum(), "stats")
    slope_err = 256.0 * ww * (r * adv.double().abs() + 0.1 * (ed + 1)) * 2 * delta
    slope = 256.0 * ww * (r * adv.double().abs() + 0.1 * (ed + 1))
    pm = p.clone()
    pm.scatter_add_(1, act.long()[:, None], torch.ones_like(elp)[:, None])
    bg = U[dtype] * eg.abs() + pm * (slope_err + slope * 2 * delta)[:, None] + TINY[dtype]
    within(dl, eg, torch.where(on[:, None], bg, torch.zeros_like(bg)), "dlogits")
    rest = torch.ones_like(wd, dtype=torch.bool)
    rest[shift:shift + rows * ld].view(rows, ld)[:, :v] = False
    assert (wd[rest] == 7).all()
    # the same without a gradient, and with the gradient in the logits' place
    lp2, loss2, stats2 = run_policy(x, ld, dtype, act, old, ref, adv, w, hp, scaler, None)
    assert torch.equal(lp, lp2) and torch.equal(loss, loss2) and torch.equal(stats, stats2)
    out = torch.empty(rows, device="cuda")
    a64 = act.long()
    Z.zero_token_logp(x.data_ptr(), rows, v, ld, ZT[dtype], a64.data_ptr(), 8, out.data_ptr(),
                      stream())
    within(out[on], elp[on], b[on], "token logp")
    run_policy(x, ld, dtype, act, old, ref, adv, w, hp, scaler, x, want_stats=False)
    assert torch.equal(x, dl)


def test_policy_gradient_against_differences():
    """Central differences of the kernel's own weighted loss along random
    directions; fp32 logits, step 2^-5. The loss is smooth away from the clip
    edges: its third derivative along a unit-variance direction stays below 50
    (powers of r <= 2.5 and of the KL term), so the difference is off by at
    most 50 h^2 / 6 sum w, and the losses' own rounding by 2^-20 sum w / h."""
    rows, v = 6, 50
    _, x, act, old, ref, adv, w = policy_inputs(rows, v, v, "fp32", 0, 77)
    old = torch.where((old - ref).abs() > 10, old, old)
    hp = Z.ZeroPolicyParams(0.9, 20.0, 0.05)  # no ratio near an edge
    dl = torch.empty(rows, v, device="cuda")
    _, _, stats = run_policy(x, v, "fp32", act, old, ref, adv, w, hp, None, dl)
    h = 2.0 ** -5
    for k in range(4):
        d = rand((rows, v), "fp32", 80 + k)
        up, dn = (run_policy(x + s * h * d, v, "fp32", act, old, ref, adv, w, hp, None, None)[2][0]
                  for s in (1.0, -1.0))
        got = (dl.double() * d.double()).sum()
        want = (up.double() - dn.double()) / (2 * h)
        total = (w * (1 + adv.abs())).sum().double()
        assert (got - want).abs() <= total * (50 * h * h / 6 + 2.0 ** -20 / h)


def test_policy_rows_left_out_and_odd_values():
    v = 40
    x = rand((8, v), "bf16", 60, 2.0)
    x[0] = float("nan")                  # weight 0: not looked at
    x[1, 5:] = float("-inf")             # tokens ruled out
    x[2] = float("-inf")                 # nothing left
    x[3, 7] = float("inf")
    x[4] = torch.finfo(torch.bfloat16).min  # all of the type's lowest value
    x[5, 3] = float("-inf")              # the taken token is ruled out
    act = torch.tensor([1, 2, 0, 1, 4, 3, -1, v], device="cuda", dtype=torch.int32)
    w = torch.ones(8, device="cuda")
    w[0] = 0
    zero = torch.zeros(8, device="cuda")
    adv = torch.ones(8, device="cuda")
    adv[5] = -1.0
    old = torch.full((8,), -3.0, device="cuda")
    dl = torch.full_like(x, 7.0)
    hp = Z.ZeroPolicyParams(0.2, 0.2, 0.0)
    lp, loss, stats = run_policy(x, v, "bf16", act, old, None, adv, w, hp, None, dl)
    for row in (0, 6, 7):
        assert lp[row] == 0 and loss[row] == 0 and (dl[row] == 0).all()
    assert torch.isfinite(lp[1]) and (dl[1, 5:] == 0).all()
    assert abs(lp[1].item() - x[1].double().log_softmax(0)[2].item()) < 1e-5
    assert torch.isnan(lp[2]) and torch.isnan(dl[2]).all()
    assert torch.isnan(lp[3])
    assert abs(lp[4].item() + math.log(v)) < 1e-5
    assert lp[5].item() == float("-inf") and torch.isfinite(dl[5]).all()
    # KL reported but not in the loss when its coefficient is 0
    ref = lp.clone()
    ref[[0, 2, 3, 5, 6, 7]] = 0
    w2 = w.clone()
    w2[[2, 3, 5]] = 0
    _, loss2, stats2 = run_policy(x, v, "bf16", act, old, ref + 1, adv, w2, hp, None, None)
    assert torch.equal(loss2[[1, 4]], loss[[1, 4]])
    assert abs(stats2[1].item() - 2 * (math.e - 2)) < 1e-4 and stats2[3] == 2
    # no rows: four zeros
    empty = torch.empty(0, v, dtype=torch.bfloat16, device="cuda")
    s = torch.full((4,), 9.0, device="cuda")
    Z.zero_policy_loss(0, 0, v, v, Z.ZERO_BF16, 0, 4, 0, 0, 0, 0, hp, 0, 0, 0, s.data_ptr(), 0,
                       stream())
    assert (s == 0).all() and empty.numel() == 0


def test_results_on_another_stream():
    """Every call takes the stream it is given: the inputs are made on it and
    the result is read after it."""
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        torch.cuda._sleep(2_000_000)
        x = rand((64, 256), "bf16", 70)
        tok = ids("uniform", 64, 100, 71)
        ck = torch.empty(Z.zero_ckpt_bytes(64, 256), dtype=torch.uint8, device="cuda")
        dw = torch.empty(256, 256, dtype=torch.bfloat16, device="cuda")
        grad = torch.empty(100, 256, dtype=torch.bfloat16, device="cuda")
        work = torch.empty(Z.zero_embedding_workspace_bytes(64, 100, 256), dtype=torch.uint8,
                           device="cuda")
        lp = torch.empty(64, device="cuda")
        s = st.cuda_stream
        Z.zero_ckpt_save(x.data_ptr(), 64, 256, 256, Z.ZERO_BF16, ck.data_ptr(), s)
        Z.zero_ckpt_wgrad(ck.data_ptr(), 64, 256, x.data_ptr(), 256, 256, Z.ZERO_BF16,
                          dw.data_ptr(), 0, s)
        Z.zero_embedding_grad(tok.data_ptr(), 4, 64, x.data_ptr(), 100, 256, 1.0, Z.ZERO_BF16, 0,
                              grad.data_ptr(), work.data_ptr(), s)
        Z.zero_token_logp(x.data_ptr(), 64, 256, 256, Z.ZERO_BF16, tok.data_ptr(), 4,
                          lp.data_ptr(), s)
    st.synchronize()
    want = ckpt64(x)[2].t() @ x.double()
    assert (dw.double() - want).norm() <= 2 * U["bf16"] * want.norm()
    want = torch.zeros(100, 256, dtype=torch.float64, device="cuda").index_add(0, tok.long(),
                                                                             x.double())
    assert (grad.double() - want).norm() <= 2 * U["bf16"] * want.norm()
    want = x.double().log_softmax(1).gather(1, tok.long()[:, None]).squeeze(1)
    assert (lp.double() - want).abs().max() < 1e-4


def test_offsets_past_32_bits():
    """Buffers of more than 2^32 bytes and 2^31 elements: the last rows are
    where they should be."""
    big = 2048 * 1_100_000                       # table elements, 4.5 GB
    vocab, dim = 1_100_000, 2048
    table = torch.zeros(big, dtype=torch.bfloat16, device="cuda").view(vocab, dim)
    table[-1] = rand((1, dim), "bf16", 90)[0]
    tok = torch.tensor([vocab - 1, 0, vocab - 1], dtype=torch.int32, device="cuda")
    out = torch.empty(3, dim, dtype=torch.bfloat16, device="cuda")
    Z.zero_embedding(tok.data_ptr(), 4, 3, table.data_ptr(), vocab, dim, 1.0, Z.ZERO_BF16,
                     out.data_ptr(), stream())
    assert torch.equal(out[0], table[-1]) and torch.equal(out[2], table[-1])
    grad = table.fill_(7.0)
    dy = rand((3, dim), "bf16", 91)
    run_grad(tok, dy, vocab, dim, 1.0, "bf16", 0, grad)
    want = (dy[0].double() + dy[2].double()).to(torch.bfloat16)
    assert torch.equal(grad[-1], want) and torch.equal(grad[0], dy[1])
    assert (grad[1:-1:4099] == 0).all() and (grad[-3:-1] == 0).all()
    del table, grad
    rows, cols = 70_000, 32_768                  # 2.3e9 activations
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-1] = rand((1, cols), "bf16", 92)[0]
    ck = torch.empty(Z.zero_ckpt_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    Z.zero_ckpt_save(x.data_ptr(), rows, cols, cols, Z.ZERO_BF16, ck.data_ptr(), stream())
    want = ckpt64(x[-1:])[2]
    x.fill_(7.0)
    Z.zero_ckpt_load(ck.data_ptr(), rows, cols, Z.ZERO_BF16, x.data_ptr(), cols, stream())
    assert torch.equal(x[-1:].double(), want) and (x[:-1:997] == 0).all()
    dy = torch.zeros(rows, 64, dtype=torch.bfloat16, device="cuda")
    dy[-1, 3] = 2.0
    dw = torch.empty(cols, 64, dtype=torch.bfloat16, device="cuda")
    Z.zero_ckpt_wgrad(ck.data_ptr(), rows, cols, dy.data_ptr(), 64, 64, Z.ZERO_BF16, dw.data_ptr(),
                      0, stream())
    assert torch.equal(dw[:, 3].double(), 2.0 * want[0]) and (dw[:, 4:] == 0).all()
    del x, ck, dy, dw
    rows, v = 17_000, 128_256                    # 2.2e9 logits
    x = torch.zeros(rows, v, dtype=torch.bfloat16, device="cuda")
    x[-1] = rand((1, v), "bf16", 93)[0]
    want = x[-1].double().log_softmax(0)
    act = torch.full((rows,), v - 1, dtype=torch.int32, device="cuda")
    w = torch.zeros(rows, device="cuda")
    w[-1] = 1.0
    one, hp = torch.ones(rows, device="cuda"), Z.ZeroPolicyParams(0.2, 0.2, 0.0)
    lp, _, _ = run_policy(x, v, "bf16", act, one * want[-1].float(), None, one, w, hp, None, x)
    assert abs(lp[-1].item() - want[-1].item()) < 1e-4 and (lp[:-1] == 0).all()
    g = want.exp()
    g[-1] -= 1.0
    assert (x[-1].double() - g).norm() <= 2 * U["bf16"] * g.norm()
    assert (x[:-1:997] == 0).all()


@pytest.mark.parametrize("rows,cols,n", [(8192, 2048, 8192), (1024, 768, 2304), (3000, 200, 1111)])
def test_weight_gradient_is_the_same_every_time(rows, cols, n):
    """Alone, and with another gradient between two that nothing waits between."""
    x, dy = [rand((rows, cols), "bf16", k) for k in (94, 95)], [rand((rows, n), "bf16", k, 0.1)
                                                                  for k in (96, 97)]
    dw = [torch.empty(cols, n, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    run_wgrad(x[0], dy[0], n, "bf16", dw[0])
    torch.cuda.synchronize()
    alone = dw[0].clone()
    for _ in range(10):
        dw[0].zero_()
        torch.cuda.synchronize()
        for k in (0, 1, 0):
            run_wgrad(x[k], dy[k], n, "bf16", dw[k])
        assert torch.equal(dw[0], alone)
