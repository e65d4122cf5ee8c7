"""The operators of include/zero_block.h on a GB300 against plain 64-bit
implementations. Bounds are derived in tests/block_util.py and at each test."""
import math

import pytest
import torch

import fsdp_sharded_mixed_shard_gb300 as Z
from block_util import (Join64, factors, fp8_64, product_bound, read_copy, scale_bytes, numbers,
                        two_to)
from train_util import DT, TINY, U, ZT, offset_rows, rand, within

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


def stream():
    return torch.cuda.current_stream().cuda_stream


def place(t, ld, shift, dtype):
    """A copy of t with row distance ld, `shift` elements into its allocation."""
    return offset_rows(*t.shape, ld, dtype, shift)[1].copy_(t)


def target(rows, cols, ld, shift, dtype):
    """(whole allocation, the array in it), filled with a pattern."""
    return offset_rows(rows, cols, ld, dtype, shift)


def untouched(whole, view):
    """Nothing but the array was written."""
    view.fill_(7.0)
    assert bool((whole == 7.0).all())


def at(t):
    return 0 if t is None else t.data_ptr()


# ----------------------------------------------------------------- dropout ----

DROPS = [  # rows, cols, ld, shift, residual, p
    (1, 1, 1, 0, False, 0.5), (1, 768, 768, 0, True, 0.1), (16, 768, 768, 0, True, 0.1),
    (37, 255, 255, 1, True, 0.25), (5, 257, 263, 3, False, 0.9), (130, 2050, 2056, 0, True, 0.1),
    (64, 513, 520, 0, False, 0.0), (3, 9, 9, 5, True, 1.0 - 2.0 ** -20), (257, 96, 96, 8, True, 0.3),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,cols,ld,shift,res,p", DROPS)
def test_dropout(dtype, rows, cols, ld, shift, res, p):
    """fl(x c) + r: c is off by 2^-24, product and sum round: 3 2^-24 of the
    magnitudes, then once to 16 bits."""
    seed, call = 0x1234567890ABCDEF, 0xFFFFFFFE
    step = torch.tensor([0xFFFFFFFD - (1 << 32)], dtype=torch.int32, device="cuda")
    x = place(rand((rows, cols), dtype, 1, 3.0), ld, shift, dtype)
    r = place(rand((rows, cols), dtype, 2), ld + 1, shift + 1, dtype) if res else None
    whole, out = target(rows, cols, ld + 1, shift + 1, dtype)
    Z.zero_dropout(Z.ZeroDropoutParams(p, seed, call, at(step)), at(x), at(r), rows, cols, ld,
                   ZT[dtype], at(out), ld + 1, stream())
    f = factors(rows, cols, p, seed, call, 0xFFFFFFFD, "cuda")
    xd = x.double() * f
    rd = r.double() if res else torch.zeros_like(xd)
    want = xd + rd
    err = 2.0 ** -22 * (xd.abs() + rd.abs())
    within(out, want, err + U[dtype] * (want.abs() + err) + TINY[dtype], "dropout")
    if not res:
        assert bool((out[f == 0] == 0).all())
    untouched(whole, out)


def test_dropout_leaves_out_what_is_not_finite():
    x = torch.full((8, 512), float("inf"), device="cuda", dtype=torch.float16)
    x[::2] = float("nan")
    out = torch.empty_like(x)
    Z.zero_dropout(Z.ZeroDropoutParams(0.5, 3, 4, 0), at(x), 0, 8, 512, 512, Z.ZERO_FP16, at(out),
                   512, stream())
    f = factors(8, 512, 0.5, 3, 4, 0, "cuda")
    assert bool((out[f == 0] == 0).all()) and not bool(torch.isfinite(out[f > 0]).any())
    assert 0.4 < (f > 0).double().mean().item() < 0.6


def test_dropout_in_place_off_the_grid():
    rows, cols = 61, 1001
    p = Z.ZeroDropoutParams(0.3, 11, 12, 0)
    x, r = (place(rand((rows, cols), "fp16", k), cols, 3, "fp16") for k in (1, 2))
    run = lambda x, r, o: Z.zero_dropout(p, at(x), at(r), rows, cols, cols, Z.ZERO_FP16,  # noqa: E731
                                         at(o), cols, stream())
    out = target(rows, cols, cols, 3, "fp16")[1]
    run(x, r, out)
    for mine in (x, r):
        before = mine.clone()
        run(x, r, mine)
        assert torch.equal(mine, out)
        mine.copy_(before)


def test_dropout_in_place_and_again():
    """In place over x or the residual, the same bits; another call, step, seed
    or row: other masks."""
    x, r = rand((77, 1000), "bf16", 5), rand((77, 1000), "bf16", 6)
    p = Z.ZeroDropoutParams(0.3, 11, 12, 0)
    run = lambda p, x, r, o: Z.zero_dropout(p, at(x), at(r), 77, 1000, 1000, Z.ZERO_BF16,  # noqa: E731
                                            at(o), 1000, stream())
    a, b, c = torch.empty_like(x), x.clone(), r.clone()
    run(p, x, r, a)
    run(p, b, r, b)
    run(p, x, c, c)
    assert torch.equal(a, b) and torch.equal(a, c)
    ones, out = torch.ones_like(x), [torch.empty_like(x) for _ in range(4)]
    step = torch.ones(1, dtype=torch.int32, device="cuda")
    for o, q in zip(out, (p, Z.ZeroDropoutParams(0.3, 12, 12, 0), Z.ZeroDropoutParams(0.3, 11, 13, 0),
                          Z.ZeroDropoutParams(0.3, 11, 12, at(step)))):
        run(q, ones, None, o)
    for o in out[1:]:
        same = (o == out[0]).double().mean().item()  # 0.7^2 + 0.3^2 = 0.58
        assert 0.55 < same < 0.61
    assert not torch.equal(out[0][0], out[0][1])


# -------------------------------------------------------------------- join ----

NAMES = ("w_post", "b_post", "gate", "w_pre", "b_pre")


def join_case(dtype, rows, cols, ld, shift, layer, names, p, a, s, seed=0, eps=1e-5, offset=0.0):
    """Inputs of a join; parameters sit one element off the rows' alignment."""
    c = dict(dtype=dtype, rows=rows, cols=cols, ld=ld, layer=layer, a=a, s=s, eps=eps, p=p)
    for k, (name, sd) in enumerate((("h", 3.0), ("y", 1.0), ("dz", 0.1), ("dh_out", 0.1))):
        t = rand((rows, cols), dtype, 10 * seed + k, sd)
        if name in ("h", "y"):
            t = (t.double() + offset).to(DT[dtype])
        c[name] = place(t, ld, shift, dtype)
    c["w"] = {}
    for k, name in enumerate(NAMES):
        t = None
        if name in names:
            t = place(rand((1, cols), dtype, 10 * seed + 5 + k, 0.2) + (0.0 if name[0] == "b" else 1.0),
                      cols, shift + (k & 1), dtype)[0]
        c["w"][name] = t
    c["seed"], c["call"], c["step"] = 77 + seed, 5, 9
    c["d_step"] = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    c["keep"] = factors(rows, cols, p, c["seed"], c["call"], c["step"], "cuda")
    c["ref"] = Join64(layer, eps, a, s, c["keep"], c["w"], dtype)
    return c


def params_of(c):
    drop = Z.ZeroDropoutParams(c["p"], c["seed"], c["call"], at(c["d_step"]))
    return Z.ZeroJoinParams(Z.ZERO_NORM_LAYER if c["layer"] else Z.ZERO_NORM_RMS, c["eps"], c["a"],
                            c["s"], drop)


def weights_of(w):
    return Z.ZeroJoinWeights(*[at(w[k]) for k in NAMES])


def forward(c, h_out, z, stats):
    Z.zero_block_join(params_of(c), weights_of(c["w"]), at(c["h"]), at(c["y"]), c["rows"], c["cols"],
                      c["ld"], ZT[c["dtype"]], at(h_out), at(z), at(stats), stream())


def backward(c, h_out, stats, dh, dy, grads, dz=True, dh_out=True):
    work = torch.full((Z.zero_block_join_workspace_bytes(c["rows"], c["cols"]) + 64,), 255,
                      dtype=torch.uint8, device="cuda")
    Z.zero_block_join_grad(params_of(c), weights_of(c["w"]), at(h_out), at(c["y"]), at(stats),
                           at(c["dz"]) if dz else 0, at(c["dh_out"]) if dh_out else 0, c["rows"],
                           c["cols"], c["ld"], ZT[c["dtype"]], at(dh), at(dy), weights_of(grads),
                           at(work), stream())
    torch.cuda.synchronize()
    assert bool((work[-64:] == 255).all())


JOINS = [  # rows, cols, ld, shift, layer, parameters, p, a, s
    (1, 1, 1, 0, False, ("w_pre",), 0.0, 1.0, 1.0),
    (1, 8, 8, 0, True, NAMES, 0.0, 1.0, 1.0),
    (3, 40, 40, 1, True, NAMES, 0.2, 1.5, 0.5),
    (16, 768, 768, 0, True, ("w_pre", "b_pre"), 0.1, 1.0, 1.0),
    (401, 768, 768, 0, True, ("w_pre", "b_pre"), 0.0, 1.0, 1.0),
    (1003, 96, 104, 0, False, ("w_post", "gate", "w_pre"), 0.1, 1.0, 0.25),
    (613, 257, 257, 3, True, NAMES, 0.1, 1.0, 0.5),
    (700, 512, 512, 0, False, ("w_post", "w_pre"), 0.0, 0.7, 1.0),
    (333, 1111, 1111, 0, True, NAMES, 0.1, 1.0, 0.5),
    (640, 2048, 2048, 0, False, ("w_post", "gate", "w_pre"), 0.0, 1.0, 0.25),
    (640, 2048, 2056, 8, False, ("gate", "w_pre"), 0.1, 1.0, 0.25),
    (161, 4096, 4096, 0, True, NAMES, 0.0, 1.0, 0.25),
    (160, 4097, 4097, 0, True, NAMES, 0.1, 1.0, 0.25),
    (155, 5000, 5000, 0, False, ("w_post", "gate", "w_pre"), 0.0, 1.0, 1.0),
    (311, 8192, 8192, 0, False, ("w_post", "gate", "w_pre"), 0.0, 1.0, 0.25),
    (40, 8191, 8191, 1, True, NAMES, 0.1, 1.0, 1.0),
    (9, 64, 64, 0, True, (), 0.5, 1.0, 1.0),
    (9, 64, 64, 0, False, ("gate",), 0.0, 0.0, 2.0),
    (9, 100, 100, 0, True, ("w_post",), 0.0, 1.0, 1.0),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(JOINS)))
def test_join_and_its_gradient(dtype, case):
    rows, cols, ld, shift, layer, names, p, a, s = JOINS[case]
    c = join_case(dtype, rows, cols, ld, shift, layer, names, p, a, s, seed=case)
    wh, h_out = target(rows, cols, ld, shift, dtype)
    wz, z = target(rows, cols, ld, shift, dtype) if "w_pre" in names else (None, None)
    stats = torch.full((rows + 1, 4), 7.0, device="cuda")
    forward(c, h_out, z, stats)
    ref = c["ref"]
    within(h_out, *ref.h_out(c["h"].double(), c["y"].double()), "h_out")
    if z is not None:
        within(z, *ref.z(h_out.double()), "z")
    assert bool((stats[rows] == 7.0).all())
    # the gradient, at the stored h_out
    dz = c["dz"].double() if z is not None else None
    for with_stream in (True, False):
        wdh, dh = target(rows, cols, ld, shift, dtype)
        wdy, dy = target(rows, cols, ld, shift, dtype)
        grads, wholes = {k: None for k in NAMES}, {}
        for k in names:
            wholes[k], g = target(1, cols, cols, shift + 1, dtype)
            grads[k] = g[0]
        backward(c, h_out, stats, dh, dy, grads, z is not None, with_stream)
        want = ref.grads(h_out.double(), c["y"].double(), dz,
                         c["dh_out"].double() if with_stream else None)
        within(dh, *want["dh"], "dh")
        within(dy, *want["dy"], "dy")
        for k in names:
            within(grads[k], *want[k], k)
            untouched(wholes[k], grads[k])
        untouched(wdh, dh)
        untouched(wdy, dy)
    untouched(wh, h_out)
    if z is not None:
        untouched(wz, z)


def test_join_far_from_zero():
    """A mean of 200 spreads: the squares are taken from the mean. fp16 keeps
    the inputs' own grid at 2^-3, far above the bound."""
    c = join_case("fp16", 50, 700, 704, 0, True, NAMES, 0.0, 1.0, 1.0, offset=200.0)
    h_out, z = torch.empty(50, 704, device="cuda", dtype=torch.float16)[:, :700], \
        torch.empty(50, 704, device="cuda", dtype=torch.float16)[:, :700]
    stats = torch.empty(50, 4, device="cuda")
    forward(c, h_out, z, stats)
    within(h_out, *c["ref"].h_out(c["h"].double(), c["y"].double()), "h_out")
    within(z, *c["ref"].z(h_out.double()), "z")


@pytest.mark.parametrize("layer", [False, True])
def test_join_gradient_against_differences(layer):
    """The formula's gradient against central differences of the 64-bit forward
    (block_util's, which the kernels are held against): third-order error."""
    names = NAMES if layer else ("w_post", "gate", "w_pre")
    c = join_case("bf16", 3, 24, 24, 0, layer, names, 0.25, 1.25, 0.5, seed=3)
    ref, y, h = c["ref"], c["y"].double(), c["h"].double()
    dz, up = c["dz"].double(), c["dh_out"].double()

    def value():
        n, _, _ = ref.branch(y)
        b = n * ref.keep * (ref.w["gate"] if ref.w["gate"] is not None else 1.0)
        ho = ref.a * h + ref.s * b
        return ((ref.z(ho)[0] * dz).sum() + (ho * up).sum()).item()

    n, _, _ = ref.branch(y)
    ho = ref.a * h + ref.s * n * ref.keep * ref.w["gate"]
    want = ref.grads(ho, y, dz, up)
    eps = 1e-5
    for name, t in [("dy", y), ("dh", h)] + [(k, ref.w[k]) for k in names]:
        flat, g = t.view(-1), want[name][0].reshape(-1)
        for i in range(0, flat.numel(), 5):
            x = flat[i].item()
            flat[i] = x + eps
            hi = value()
            flat[i] = x - eps
            lo = value()
            flat[i] = x
            assert abs((hi - lo) / (2 * eps) - g[i].item()) < 1e-6 * (1 + abs(g[i].item())), name


@pytest.mark.parametrize("cols", [96, 1111, 8192])
def test_join_in_place_is_the_same(cols):
    """h_out over h and z over y; dh over dh_out and dy over dz, and the other
    way round; the same bits every time."""
    rows = 320
    c = join_case("bf16", rows, cols, cols, 0, True, NAMES, 0.1, 1.0, 0.5)
    new = lambda: torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    h_out, z, stats = new(), new(), torch.empty(rows, 4, device="cuda")
    forward(c, h_out, z, stats)
    d = dict(c, h=c["h"].clone(), y=c["y"].clone())
    s2 = torch.empty_like(stats)
    forward(d, d["h"], d["y"], s2)
    assert torch.equal(d["h"], h_out) and torch.equal(d["y"], z) and torch.equal(stats, s2)
    d = dict(c, y=c["y"].clone())
    z2 = new()
    forward(d, d["y"], z2, s2)
    assert torch.equal(d["y"], h_out) and torch.equal(z2, z)
    results = []
    for how in range(3):
        d = dict(c, dz=c["dz"].clone(), dh_out=c["dh_out"].clone())
        dh, dy = [(new(), new()), (d["dh_out"], d["dz"]), (d["dz"], d["dh_out"])][how]
        grads = {k: torch.empty(cols, device="cuda", dtype=torch.bfloat16) for k in NAMES}
        backward(d, h_out, stats, dh, dy, grads)
        results.append([dh, dy] + [grads[k] for k in NAMES])
    for r in results[1:]:
        for x, y in zip(results[0], r):
            assert torch.equal(x, y)


def test_join_rows_that_are_not_finite():
    """A row with an infinity or NaN is NaN where it is normalised, the other
    rows as they were; a row of zeros stays finite."""
    rows, cols = 12, 768
    for layer in (False, True):
        names = NAMES if layer else ("w_post", "gate", "w_pre")
        c = join_case("bf16", rows, cols, cols, 0, layer, names, 0.0, 1.0, 1.0)
        c["y"][3, 100] = float("inf")
        c["y"][5, 700] = float("nan")
        c["h"][7, 0] = -float("inf")
        c["y"][9] = 0
        c["h"][9] = 0
        c["y"][10] = 3e38  # its squares pass fp32's range
        h_out, z = (torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        forward(c, h_out, z, torch.empty(rows, 4, device="cuda"))
        bad = [3, 5, 7, 10]
        for r in bad:
            assert bool(torch.isnan(z[r]).all())
        good = [r for r in range(rows) if r not in bad]
        want, bound = c["ref"].h_out(c["h"].double(), c["y"].double())
        within(h_out[good], want[good], bound[good], "h_out")
        want, bound = c["ref"].z(h_out.double())
        within(z[good], want[good], bound[good], "z")


@pytest.mark.parametrize("cols", [264, 263])
def test_join_leaves_out_what_is_not_finite(cols):
    """Without a norm after the block, an infinity that dropout leaves out counts for
    nothing: not in h_out, z or any gradient."""
    rows = 40
    c = join_case("bf16", rows, cols, cols, 0, False, ("gate", "w_pre"), 0.5, 1.0, 1.0, seed=8)
    clean = c["y"].clone()
    c["y"][c["keep"] == 0] = float("inf")
    new = lambda: torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    h_out, z, dh, dy, stats = new(), new(), new(), new(), torch.empty(rows, 4, device="cuda")
    forward(c, h_out, z, stats)
    grads = {k: torch.empty_like(c["w"][k]) if k in ("gate", "w_pre") else None for k in NAMES}
    backward(c, h_out, stats, dh, dy, grads)
    within(h_out, *c["ref"].h_out(c["h"].double(), clean.double()), "h_out")
    want = c["ref"].grads(h_out.double(), clean.double(), c["dz"].double(), c["dh_out"].double())
    for name, got in (("dh", dh), ("dy", dy), ("gate", grads["gate"]), ("w_pre", grads["w_pre"])):
        within(got, *want[name], name)


def test_join_with_no_rows():
    grads = {k: torch.full((100,), 7.0, device="cuda", dtype=torch.bfloat16) for k in NAMES}
    w = weights_of(grads)
    p = Z.ZeroJoinParams(Z.ZERO_NORM_LAYER, 1e-5, 1.0, 1.0, Z.ZeroDropoutParams(0.0, 0, 0, 0))
    Z.zero_block_join_grad(p, w, 0, 0, 0, 0, 0, 0, 100, 100, Z.ZERO_BF16, 0, 0, w, 0, stream())
    torch.cuda.synchronize()
    for g in grads.values():
        assert bool((g == 0).all())


# --------------------------------------------------------------------- fp8 ----

def copy_of(x, rows, cols, ld, dtype, fmt):
    buf = torch.full((Z.zero_fp8_bytes(rows, cols) + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    Z.zero_fp8_quant(at(x), rows, cols, ld, ZT[dtype], Z.ZERO_E4M3 if fmt == "e4m3" else Z.ZERO_E5M2,
                     at(buf), stream())
    torch.cuda.synchronize()
    assert bool((buf[-64:] == 0xAB).all())
    return buf


def weight_of(w, k, n, dtype):
    buf = torch.full((Z.zero_fp8_weight_bytes(k, n) + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    Z.zero_fp8_quant_weight(at(w), k, n, ZT[dtype], at(buf), stream())
    torch.cuda.synchronize()
    assert bool((buf[-64:] == 0xAB).all())
    return buf


def same(got, want):
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(), want.nan_to_num())


COPIES = [(1, 1, 1, 0), (3, 100, 100, 1), (130, 128, 128, 0), (5, 129, 136, 8), (257, 1111, 1111, 0),
          (64, 2048, 2048, 0), (9, 8192, 8200, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols,ld,shift", COPIES)
def test_fp8_copy(dtype, fmt, rows, cols, ld, shift):
    """Values and scale bytes exactly, blocks of all magnitudes among them."""
    x = rand((rows, cols), dtype, 3, 1.0).double()
    mag = torch.randint(-20, 14, (rows, -(-cols // 128)), device="cuda").repeat_interleave(128, 1)
    x = (x * two_to(mag[:, :cols])).to(DT[dtype])
    if rows > 2:
        x[1, :100] = 0
        x[2] = x[2] * (1e-30 if dtype == "bf16" else 1.0)
        x[0, -1] = float("nan")
        x[rows - 1, 0] = -float("inf")
    x = place(x, ld, shift, dtype)
    got_s, got, pad = read_copy(copy_of(x, rows, cols, ld, dtype, fmt), rows, cols, fmt)
    want_s, want = fp8_64(x, fmt, 1)
    assert torch.equal(got_s, want_s.long())
    same(got, want)
    if rows > 2:  # a block that is not finite holds NaN past the last column too
        pad = pad[1:rows - 1]
    assert bool((pad == 0).all())


def test_fp8_rounding_and_edges():
    """Every finite fp16 number as the second element of a block whose largest
    is 448 (E4M3) or 57344 (E5M2), and as the largest itself."""
    every = torch.arange(1 << 16, dtype=torch.int32, device="cuda").to(torch.int16)
    every = every.view(torch.float16)
    every = every[torch.isfinite(every)]
    for fmt, most in (("e4m3", 448.0), ("e5m2", 57344.0)):
        x = torch.zeros(every.numel(), 128, dtype=torch.float16, device="cuda")
        x[:, 0] = most
        x[:, 1] = every.clamp(-most, most)
        for t in (x, torch.cat([x[:, 1:], x[:, :1] * 0], 1).contiguous()):
            rows = t.shape[0]
            got_s, got, _ = read_copy(copy_of(t, rows, 128, 128, "fp16", fmt), rows, 128, fmt)
            want_s, want = fp8_64(t, fmt, 1)
            assert torch.equal(got_s, want_s.long())
            same(got, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("k,n,shift", [(1, 1, 0), (128, 128, 0), (100, 300, 1), (515, 640, 0),
                                       (1111, 2222, 3), (768, 2304, 8)])
def test_fp8_weight_copy(dtype, k, n, shift):
    w = place(rand((k, n), dtype, 4, 0.02), n, shift, dtype)
    if k > 300:
        w[130, 200] = float("inf")
        w[256:384, 128:256] = 0
    buf = weight_of(w, k, n, dtype)
    kb, nb = -(-k // 128), -(-n // 128)
    want_s, want = fp8_64(w, "e4m3", 128)
    q = buf[:k * nb * 128].view(k, nb * 128)
    first = k * nb * 128
    by_col = scale_bytes(buf[first:], n, kb)
    by_row = scale_bytes(buf[first + nb * (-(-kb // 4)) * 512:], k, nb)
    assert torch.equal(by_row, want_s.long().repeat_interleave(128, 0)[:k])
    assert torch.equal(by_col, want_s.long().t().repeat_interleave(128, 0)[:n])
    unit = two_to(by_row - 127).repeat_interleave(128, 1)
    same((numbers(q, "e4m3") * unit)[:, :n], want)
    if k <= 300:
        assert bool((q[:, n:] == 0).all())


PRODUCTS = [  # rows, k, n, ld past n (and past k), shift of the output
    (1, 1, 1, 0, 0), (1, 128, 128, 0, 0), (3, 100, 40, 3, 1), (16, 768, 2304, 0, 0),
    (130, 257, 511, 0, 0), (256, 1024, 192, 0, 0), (257, 640, 385, 7, 8), (1003, 1111, 2222, 0, 0),
    (40, 8192, 256, 0, 0), (300, 4100, 2048, 8, 0), (5000, 384, 4000, 0, 0), (2, 2048, 9001, 1, 3),
    (16, 5000, 2048, 0, 0), (4096, 2048, 2048, 0, 0), (700, 520, 1500, 4, 0),
]


@pytest.mark.parametrize("dtype,fmt", [("bf16", "e4m3"), ("fp16", "e4m3"), ("bf16", "e5m2")])
@pytest.mark.parametrize("rows,k,n,past,shift", PRODUCTS)
def test_fp8_products(dtype, fmt, rows, k, n, past, shift):
    """y = x W and dx = dy W^T against the copies' values in 64 bits; blocks of
    very different scales, so that a scale that goes astray shows."""
    def blocks(shape, seed, sd, lo, hi, br):
        t = rand(shape, dtype, seed, sd).double()
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        e = torch.randint(lo, hi, (-(-shape[0] // br), -(-shape[1] // 128)), generator=g, device="cuda")
        e = e.repeat_interleave(br, 0).repeat_interleave(128, 1)[:shape[0], :shape[1]]
        return (t * two_to(e)).to(DT[dtype])

    x, dy = blocks((rows, k), 1, 1.0, -3, 4, 1), blocks((rows, n), 2, 1e-2, -3, 4, 1)
    w = blocks((k, n), 3, 0.02, -4, 3, 128)
    f = Z.ZERO_E4M3 if fmt == "e4m3" else Z.ZERO_E5M2
    x8, w8, dy8 = (copy_of(x, rows, k, k, dtype, fmt), weight_of(w, k, n, dtype),
                   copy_of(dy, rows, n, n, dtype, fmt))
    scaler = torch.zeros(20, device="cuda")
    wy, y = target(rows, n, n + past, shift, dtype)
    wd, dx = target(rows, k, k + past, shift, dtype)
    Z.zero_fp8_linear(at(x8), f, rows, at(w8), k, n, ZT[dtype], at(y), n + past, at(scaler), stream())
    Z.zero_fp8_linear_dgrad(at(dy8), f, rows, at(w8), k, n, ZT[dtype], at(dx), k + past, at(scaler),
                            stream())
    xv, wv, dv = (t[1] for t in (fp8_64(x, fmt, 1), fp8_64(w, "e4m3", 128), fp8_64(dy, fmt, 1)))
    want = xv @ wv
    within(y, want, product_bound(want, xv, wv, k, dtype), "y")
    want = dv @ wv.t()
    within(dx, want, product_bound(want, dv, wv.t(), n, dtype), "dx")
    assert bool((scaler == 0).all())
    untouched(wy, y)
    untouched(wd, dx)


@pytest.mark.parametrize("up,down", [(-100, 90), (100, -110), (-60, -40), (30, 40)])
def test_fp8_products_of_far_scales(up, down):
    """Scales far from 1, whose product is not: they add up as exponents do."""
    rows, k, n = 40, 384, 264
    x = (rand((rows, k), "bf16", 1).double() * 2.0 ** up).to(torch.bfloat16)
    w = (rand((k, n), "bf16", 2).double() * 2.0 ** down).to(torch.bfloat16)
    x8, w8 = copy_of(x, rows, k, k, "bf16", "e4m3"), weight_of(w, k, n, "bf16")
    y = torch.empty(rows, n, device="cuda", dtype=torch.bfloat16)
    Z.zero_fp8_linear(at(x8), 0, rows, at(w8), k, n, Z.ZERO_BF16, at(y), n, 0, stream())
    xv, wv = fp8_64(x, "e4m3", 1)[1], fp8_64(w, "e4m3", 128)[1]
    want = xv @ wv
    within(y, want, product_bound(want, xv, wv, k, "bf16"), "y")


def test_fp8_products_of_what_is_not_finite():
    """A row whose block is not finite is NaN, a weight's block its columns (x W)
    and its rows (dy W^T); the rest as it was."""
    rows, k, n = 300, 700, 600
    x, w, dy = rand((rows, k), "bf16", 1), rand((k, n), "bf16", 2, 0.02), rand((rows, n), "bf16", 3)
    x[17, 400] = float("inf")
    dy[200, 3] = float("nan")
    w[300, 500] = -float("inf")
    x8, w8, dy8 = (copy_of(x, rows, k, k, "bf16", "e4m3"), weight_of(w, k, n, "bf16"),
                   copy_of(dy, rows, n, n, "bf16", "e4m3"))
    y = torch.empty(rows, n, device="cuda", dtype=torch.bfloat16)
    dx = torch.empty(rows, k, device="cuda", dtype=torch.bfloat16)
    Z.zero_fp8_linear(at(x8), 0, rows, at(w8), k, n, Z.ZERO_BF16, at(y), n, 0, stream())
    Z.zero_fp8_linear_dgrad(at(dy8), 0, rows, at(w8), k, n, Z.ZERO_BF16, at(dx), k, 0, stream())
    bad_y = torch.zeros(rows, n, dtype=torch.bool, device="cuda")
    bad_y[17] = True
    bad_y[:, 384:512] = True
    bad_x = torch.zeros(rows, k, dtype=torch.bool, device="cuda")
    bad_x[200] = True
    bad_x[:, 256:384] = True
    assert torch.equal(torch.isnan(y), bad_y) and torch.equal(torch.isnan(dx), bad_x)
    xv, wv = fp8_64(x, "e4m3", 1)[1], fp8_64(w, "e4m3", 128)[1]
    fine_x, fine_w = xv.nan_to_num(), wv.nan_to_num()
    want = fine_x @ fine_w
    within(y[~bad_y], want[~bad_y], product_bound(want, fine_x, fine_w, k, "bf16")[~bad_y], "y")


def test_fp8_products_of_nothing():
    """An empty reduction gives zeros; blocks of zeros too."""
    y = torch.full((5, 40), 7.0, device="cuda", dtype=torch.bfloat16)
    Z.zero_fp8_linear(0, 0, 5, 0, 0, 33, Z.ZERO_BF16, at(y), 40, 0, stream())
    assert bool((y[:, :33] == 0).all()) and bool((y[:, 33:] == 7).all())
    zero = torch.zeros(5, 300, device="cuda", dtype=torch.bfloat16)
    w = rand((300, 40), "bf16", 1)
    x8, w8 = copy_of(zero, 5, 300, 300, "bf16", "e4m3"), weight_of(w, 300, 40, "bf16")
    Z.zero_fp8_linear(at(x8), 0, 5, at(w8), 300, 40, Z.ZERO_BF16, at(y), 40, 0, stream())
    assert bool((y == 0).all())


def test_fp8_products_repeat_their_bits():
    """Alone, and between others that nothing waits for: a split reduction, one
    whole turn of tiles, more tiles than the device holds."""
    for rows, k, n in ((40, 8192, 256), (2048, 2048, 2048), (4000, 512, 8000)):
        x, w = rand((rows, k), "bf16", 1), rand((k, n), "bf16", 2, 0.02)
        x8, w8 = copy_of(x, rows, k, k, "bf16", "e4m3"), weight_of(w, k, n, "bf16")
        out = [torch.empty(rows, n, device="cuda", dtype=torch.bfloat16) for _ in range(4)]
        for o in out:
            Z.zero_fp8_linear(at(x8), 0, rows, at(w8), k, n, Z.ZERO_BF16, at(o), n, 0, stream())
        torch.cuda.synchronize()
        for o in out[1:]:
            assert torch.equal(o, out[0])


# ------------------------------------------------------------------ a block ----

def test_block_captured_and_replayed():
    """A linear layer, its join and their gradients in one graph on a stream of
    its own; replayed with the device's step moved on, it draws that step's
    masks, and equals the same calls made one by one."""
    rows, dim, hidden = 200, 256, 512
    c = join_case("bf16", rows, dim, dim, 0, True, NAMES, 0.2, 1.0, 0.5)
    x, w = rand((rows, hidden), "bf16", 50), rand((hidden, dim), "bf16", 51, 0.05)
    new = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    y, h_out, z, dh, dy = (new(rows, dim) for _ in range(5))
    dx, stats = new(rows, hidden), torch.zeros(rows, 4, device="cuda")
    grads = {k: new(dim) for k in NAMES}
    work = torch.zeros(Z.zero_block_join_workspace_bytes(rows, dim), dtype=torch.uint8, device="cuda")
    x8, w8, dy8 = (torch.zeros(b, dtype=torch.uint8, device="cuda") for b in (
        Z.zero_fp8_bytes(rows, hidden), Z.zero_fp8_weight_bytes(hidden, dim),
        Z.zero_fp8_bytes(rows, dim)))
    drop = Z.ZeroDropoutParams(0.3, 8, 9, at(c["d_step"]))
    outs = [y, h_out, z, dh, dy, dx] + list(grads.values())

    def block(st):
        bf = Z.ZERO_BF16
        Z.zero_fp8_quant_weight(at(w), hidden, dim, bf, at(w8), st)
        Z.zero_fp8_quant(at(x), rows, hidden, hidden, bf, 0, at(x8), st)
        Z.zero_fp8_linear(at(x8), 0, rows, at(w8), hidden, dim, bf, at(y), dim, 0, st)
        Z.zero_block_join(params_of(c), weights_of(c["w"]), at(c["h"]), at(y), rows, dim, dim, bf,
                          at(h_out), at(z), at(stats), st)
        Z.zero_block_join_grad(params_of(c), weights_of(c["w"]), at(h_out), at(y), at(stats),
                               at(c["dz"]), at(c["dh_out"]), rows, dim, dim, bf, at(dh), at(dy),
                               weights_of(grads), at(work), st)
        Z.zero_fp8_quant(at(dy), rows, dim, dim, bf, 1, at(dy8), st)
        Z.zero_fp8_linear_dgrad(at(dy8), 1, rows, at(w8), hidden, dim, bf, at(dx), hidden, 0, st)
        Z.zero_dropout(drop, at(dx), 0, rows, hidden, hidden, bf, at(dx), hidden, st)

    want = []
    for step in (9, 10):
        c["d_step"].fill_(step)
        block(stream())
        want.append([o.clone() for o in outs])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        block(torch.cuda.current_stream().cuda_stream)
    for k, step in enumerate((9, 10, 9)):
        for o in outs:
            o.zero_()
        c["d_step"].fill_(step)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want[k % 2]):
            assert torch.equal(a, b)
    assert not torch.equal(want[0][1], want[1][1])
    assert math.isfinite(dx.double().norm().item())


def test_offsets_past_32_bits():
    """Rows 2^31 elements apart: every operator's result is that of the same rows
    side by side."""
    rows, cols, ld = 3, 264, 1 << 31
    far = lambda: torch.empty((rows - 1) * ld + cols, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    view = lambda t: t.as_strided((rows, cols), (ld, 1))  # noqa: E731
    bf, st = Z.ZERO_BF16, stream()
    a, b, c, d = (far() for _ in range(4))
    x, y = rand((rows, cols), "bf16", 1), rand((rows, cols), "bf16", 2)
    near = [torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16) for _ in range(4)]
    p = Z.ZeroDropoutParams(0.25, 5, 6, 0)
    view(a).copy_(x)
    view(b).copy_(y)
    Z.zero_dropout(p, at(a), at(b), rows, cols, ld, bf, at(c), ld, st)
    Z.zero_dropout(p, at(x), at(y), rows, cols, cols, bf, at(near[0]), cols, st)
    assert torch.equal(view(c), near[0])
    n = Z.zero_fp8_bytes(rows, cols)
    q = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    Z.zero_fp8_quant(at(a), rows, cols, ld, bf, 0, at(q[0]), st)
    Z.zero_fp8_quant(at(x), rows, cols, cols, bf, 0, at(q[1]), st)
    assert torch.equal(*q)
    w8 = weight_of(rand((cols, cols), "bf16", 3), cols, cols, "bf16")
    Z.zero_fp8_linear(at(q[0]), 0, rows, at(w8), cols, cols, bf, at(c), ld, 0, st)
    Z.zero_fp8_linear(at(q[0]), 0, rows, at(w8), cols, cols, bf, at(near[0]), cols, 0, st)
    assert torch.equal(view(c), near[0])
    # the join in place over h and y, its gradient over dh_out and dz
    w = {k: rand((1, cols), "bf16", 10 + i)[0] for i, k in enumerate(NAMES)}
    g = [{k: torch.empty_like(v) for k, v in w.items()} for _ in range(2)]
    hp = Z.ZeroJoinParams(Z.ZERO_NORM_LAYER, 1e-5, 1.0, 0.5, p)
    work = torch.empty(Z.zero_block_join_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    stats = [torch.empty(rows, 4, device="cuda") for _ in range(2)]
    view(c).copy_(x)
    view(d).copy_(y)
    Z.zero_block_join(hp, weights_of(w), at(a), at(b), rows, cols, ld, bf, at(a), at(b), at(stats[0]), st)
    Z.zero_block_join(hp, weights_of(w), at(x), at(y), rows, cols, cols, bf, at(near[0]), at(near[1]),
                      at(stats[1]), st)
    assert torch.equal(view(a), near[0]) and torch.equal(view(b), near[1])
    Z.zero_block_join_grad(hp, weights_of(w), at(a), at(b), at(stats[0]), at(c), at(d), rows, cols, ld,
                           bf, at(d), at(c), weights_of(g[0]), at(work), st)
    Z.zero_block_join_grad(hp, weights_of(w), at(near[0]), at(near[1]), at(stats[1]), at(x), at(y), rows,
                           cols, cols, bf, at(near[2]), at(near[3]), weights_of(g[1]), at(work), st)
    assert torch.equal(view(d), near[2]) and torch.equal(view(c), near[3])
    for k in NAMES:
        assert torch.equal(g[0][k], g[1][k])


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, that run beside one
    another give what they give alone."""
    rows, dim, hidden = 3000, 512, 1024
    side = [torch.cuda.Stream() for _ in range(2)]
    cases = []
    for k in range(2):
        c = join_case("bf16", rows, dim, dim, 0, bool(k), NAMES if k else ("w_post", "gate", "w_pre"),
                      0.1, 1.0, 0.5, seed=20 + k)
        x, w = rand((rows, hidden), "bf16", 30 + k), rand((hidden, dim), "bf16", 32 + k, 0.05)
        t = dict(c=c, x8=copy_of(x, rows, hidden, hidden, "bf16", "e4m3"),
                 w8=weight_of(w, hidden, dim, "bf16"), stats=torch.empty(rows, 4, device="cuda"),
                 work=torch.empty(Z.zero_block_join_workspace_bytes(rows, dim), dtype=torch.uint8,
                                  device="cuda"),
                 out=[torch.empty(rows, dim, device="cuda", dtype=torch.bfloat16) for _ in range(5)],
                 g={n: None if v is None else torch.empty_like(v) for n, v in c["w"].items()})
        cases.append(t)
    torch.cuda.synchronize()

    def run(t, st):
        c, (y, h_out, z, dh, dy), bf = t["c"], t["out"], Z.ZERO_BF16
        Z.zero_fp8_linear(at(t["x8"]), 0, rows, at(t["w8"]), hidden, dim, bf, at(y), dim, 0, st)
        Z.zero_block_join(params_of(c), weights_of(c["w"]), at(c["h"]), at(y), rows, dim, dim, bf,
                          at(h_out), at(z), at(t["stats"]), st)
        Z.zero_block_join_grad(params_of(c), weights_of(c["w"]), at(h_out), at(y), at(t["stats"]),
                               at(c["dz"]), at(c["dh_out"]), rows, dim, dim, bf, at(dh), at(dy),
                               weights_of(t["g"]), at(t["work"]), st)

    results = lambda t: [o.clone() for o in t["out"] + [v for v in t["g"].values() if v is not None]]  # noqa: E731
    alone = []
    for t, s in zip(cases, side):
        run(t, s.cuda_stream)
        torch.cuda.synchronize()
        alone.append(results(t))
    for _ in range(20):
        for t, s in zip(cases, side):
            run(t, s.cuda_stream)
    torch.cuda.synchronize()
    for t, want in zip(cases, alone):
        for a, b in zip(results(t), want):
            assert torch.equal(a, b)
