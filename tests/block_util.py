"""64-bit references and derived error bounds for the operators of
include/zero_block.h (used by tests/test_gpu_block.py).

u: unit roundoff of the 16-bit type (train_util.U). An operator computes in
fp32, whose roundings are off by 2^-24 of the result each, and rounds once."""
import numpy as np
import torch

from train_util import TINY, U

# Longest chain of additions in a row's sum: 16 in a thread (two vectors of
# eight), 5 in its warp, 16 warps; with the product and the scaling fewer than
# 64 roundings, so a sum is off by 2^-18 of the sum of magnitudes.
SUM = 2.0 ** -18
# 1 / sqrt: half the relative error of the mean square (2^-18), rsqrtf 2 ulp
ROOT = 2.0 ** -18
# sums over rows: at most 2^31 / 152 per thread in principle, but in these tests
# below 64 in a thread, 16 teams, 19 partial vectors and 8 warps: fewer than 128
ROWS = 2.0 ** -17


# ----------------------------------------------------------------- dropout ----

def threshold(p):
    return min(int(p * 65536 + 0.5), 65535)


def draws(rows, cols, seed, call, step):
    """The generator's 16 bits per element: Philox 4x32, 7 rounds, in numpy."""
    groups = -(-cols // 8)
    low = np.uint64(0xFFFFFFFF)
    c = np.zeros((4, rows, groups), np.uint64)
    c[0] = np.arange(groups, dtype=np.uint64)
    c[1] = np.arange(rows, dtype=np.uint64)[:, None]
    c[2], c[3] = call, step & 0xFFFFFFFF
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(7):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = np.stack([(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low,
                      (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low])
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    h = np.empty((rows, groups, 8), np.int64)
    for j in range(8):
        h[:, :, j] = (c[j // 2] >> np.uint64(16 * (j % 2))) & np.uint64(0xFFFF)
    return h.reshape(rows, groups * 8)[:, :cols]


def factors(rows, cols, p, seed, call, step, dev):
    """0 or 1 / (1 - p) for each element, p as it is rounded."""
    t = threshold(p)
    if t == 0:
        return torch.ones(rows, cols, dtype=torch.float64, device=dev)
    keep = torch.from_numpy(draws(rows, cols, seed, call, step) >= t).to(dev)
    return keep.double() * (65536.0 / (65536 - t))


# -------------------------------------------------------------------- join ----

def norm64(x, layer, eps):
    """(normed, mean, 1 / root) and the normed value's fp32 error."""
    mean = x.mean(1, keepdim=True) if layer else torch.zeros_like(x[:, :1])
    c = x - mean
    r = 1 / ((c * c).mean(1, keepdim=True) + eps).sqrt()
    xhat = c * r
    off = SUM * x.abs().mean(1, keepdim=True) if layer else 0.0  # of the mean
    # eps, 1/n and the centring round too; near eps the root moves with it
    err = ROOT * xhat.abs() + r * (off + 2.0 ** -23 * x.abs()) + 2.0 ** -22 * xhat.abs()
    if layer:  # a mean that is off by `off` adds off^2 to the mean square
        err = err + xhat.abs() * (r * off) ** 2
    return xhat, mean, r, err


def norm_back64(g, eg, xhat, ex, r, layer, parts=None):
    """Gradient through a norm and its fp32 error: r (g - xhat mean(g xhat) -
    mean(g)), eg and ex the errors of g and xhat; parts: the magnitudes that g is
    summed from, where its sums over the row are taken part by part."""
    parts = g.abs() if parts is None else parts
    m = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    c1, c2 = m(g * xhat), m(g) if layer else torch.zeros_like(g[:, :1])
    out = r * (g - xhat * c1 - c2)
    e1 = m(eg * xhat.abs()) + m(parts * ex) + SUM * m(parts * xhat.abs())
    e2 = (m(eg) + SUM * m(parts)) if layer else 0.0
    mag = g.abs() + (xhat * c1).abs() + c2.abs()
    err = r * (eg + xhat.abs() * e1 + ex * c1.abs() + e2 + 2.0 ** -21 * mag) + ROOT * r * mag
    return out, err


def rounded(want, err, dtype):
    return err + U[dtype] * (want.abs() + err) + TINY[dtype]


class Join64:
    """The join and its gradient in 64 bits; w: dict of parameters (or None)."""

    def __init__(self, layer, eps, a, s, keep, w, dtype):
        self.layer, self.eps, self.a, self.s, self.keep, self.dtype = layer, eps, a, s, keep, dtype
        self.w = {k: None if t is None else t.double() for k, t in w.items()}

    def branch(self, y):
        """b before dropout, its error, and the norm's parts."""
        w = self.w
        if w["w_post"] is None:
            return y, torch.zeros_like(y), None
        xhat, mean, r, ex = norm64(y, self.layer, self.eps)
        n = xhat * w["w_post"] + (w["b_post"] if w["b_post"] is not None else 0.0)
        en = ex * w["w_post"].abs() + 2.0 ** -23 * ((xhat * w["w_post"]).abs() + n.abs())
        return n, en, (xhat, mean, r, ex)

    def h_out(self, h, y):
        n, en, _ = self.branch(y)
        g = self.w["gate"] if self.w["gate"] is not None else torch.ones_like(n[0])
        b = self.s * g * torch.where(self.keep > 0, n * self.keep, torch.zeros_like(n))
        out = self.a * h + b
        err = (self.s * g * self.keep).abs() * en + 2.0 ** -21 * ((self.a * h).abs() + b.abs())
        return out, rounded(out, err, self.dtype)

    def z(self, h_out):
        xhat, mean, r, ex = norm64(h_out, self.layer, self.eps)
        b = self.w["b_pre"] if self.w["b_pre"] is not None else 0.0
        z = xhat * self.w["w_pre"] + b
        err = ex * self.w["w_pre"].abs() + 2.0 ** -22 * ((xhat * self.w["w_pre"]).abs() + z.abs())
        return z, rounded(z, err, self.dtype)

    def grads(self, h_out, y, dz, dh_out):
        """{name: (gradient, bound)}."""
        w, out = self.w, {}
        d = dh_out if dh_out is not None else torch.zeros_like(h_out)
        ed = torch.zeros_like(d)
        parts = d.abs()  # D's sums over a row are those of its terms
        if w["w_pre"] is not None:
            xhat, _, r, ex = norm64(h_out, self.layer, self.eps)
            g = dz * w["w_pre"]
            through, ed = norm_back64(g, 2.0 ** -23 * g.abs(), xhat, ex, r, self.layer)
            c1, c2 = (g * xhat).mean(1, keepdim=True), g.mean(1, keepdim=True)
            parts = parts + r * (g.abs() + (xhat * c1).abs() + (c2.abs() if self.layer else 0.0))
            d = d + through
            ed = ed + 2.0 ** -23 * (d.abs() + through.abs())
            out["w_pre"] = self.sums(dz * xhat, dz.abs() * ex)
            out["b_pre"] = self.sums(dz, torch.zeros_like(dz))
        dh = self.a * d
        out["dh"] = dh, rounded(dh, abs(self.a) * ed + 2.0 ** -23 * dh.abs(), self.dtype)
        n, en, post = self.branch(y)
        e = self.s * self.keep * d
        ee = (self.s * self.keep).abs() * ed + 2.0 ** -21 * e.abs()
        if w["gate"] is not None:
            # summed as w_post sum e xhat + b_post sum e, whose terms may cancel
            # in n: the sums' error is that of both
            parts = n.abs()
            if post is not None:
                parts = (post[0] * w["w_post"]).abs()
                parts = parts + (w["b_post"].abs() if w["b_post"] is not None else 0.0)
            out["gate"] = self.sums(e * n, ee * parts + e.abs() * (en + ROWS * parts))
            e, ee = e * w["gate"], ee * w["gate"].abs() + 2.0 ** -23 * (e * w["gate"]).abs()
        if post is not None:
            xhat, _, r, ex = post
            out["w_post"] = self.sums(e * xhat, ee * xhat.abs() + e.abs() * ex)
            out["b_post"] = self.sums(e, ee)
            q = e * w["w_post"]
            parts = parts * (self.s * self.keep * w["w_post"]).abs()
            if w["gate"] is not None:
                parts = parts * w["gate"].abs()
            e, ee = norm_back64(q, ee * w["w_post"].abs() + 2.0 ** -23 * q.abs(), xhat, ex, r,
                                self.layer, parts)
        out["dy"] = e, rounded(e, ee, self.dtype)
        return out

    def sums(self, terms, err):
        want = terms.sum(0)
        e = err.sum(0) + ROWS * terms.abs().sum(0)
        return want, rounded(want, e, self.dtype)


# --------------------------------------------------------------------- fp8 ----

FORMATS = {"e4m3": (3, -6, 448.0), "e5m2": (2, -14, 57344.0)}


def two_to(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def fp8_64(x, fmt, block_rows):
    """(scale bytes [rows / block_rows, blocks], values) of the copy of x."""
    bits, low, most = FORMATS[fmt]
    rows, cols = x.shape
    br, bc = -(-rows // block_rows), -(-cols // 128)
    b = torch.zeros(br * block_rows, bc * 128, dtype=torch.float64, device=x.device)
    b[:rows, :cols] = x.double()
    b = b.view(br, block_rows, bc, 128)
    fine = torch.isfinite(b).all(3, keepdim=True).all(1, keepdim=True)
    top = torch.where(fine, b, torch.zeros_like(b)).abs().amax((1, 3), keepdim=True)
    m, e = torch.frexp(top / most)
    k = torch.where(m == 0.5, e - 1, e).clamp(min=-126)
    k = torch.where(top == 0, torch.zeros_like(k), k)
    v = torch.where(fine, b, torch.zeros_like(b)) / two_to(k)
    step = two_to((torch.frexp(v).exponent - 1).clamp(min=low) - bits)
    val = torch.where(fine, (v / step).round() * step * two_to(k), torch.full_like(b, float("nan")))
    byte = torch.where(fine, k + 127, torch.full_like(k, 255)).view(br, bc)
    return byte, val.reshape(br * block_rows, bc * 128)[:rows, :cols]


def scale_bytes(tiles, rows, blocks):
    """[rows, blocks] scale bytes out of their tiles."""
    groups = -(-blocks // 4)
    t = tiles[:-(-rows // 128) * groups * 512].view(-(-rows // 128), groups, 32, 4, 4)
    return t.permute(0, 3, 2, 1, 4).reshape(-1, groups * 4)[:rows, :blocks].long()


def numbers(q, fmt):
    return q.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2).double()


def read_copy(buf, rows, cols, fmt):
    """(scale bytes, values, padding) of an activation's copy."""
    blocks = -(-cols // 128)
    q = buf[:rows * blocks * 128].view(rows, blocks * 128)
    s = scale_bytes(buf[rows * blocks * 128:], rows, blocks)
    unit = two_to(s - 127).repeat_interleave(128, 1)
    return s, (numbers(q, fmt) * unit)[:, :cols], q[:, cols:]


def product_bound(want, x, w, k, dtype):
    """The tensor core adds 32 products at a time, each kept to at least 2^-23 of
    the largest (32 of them), then the running sum, rounded or cut to 2^-23:
    at most k / 32 + 32 times 2^-23 of the sum of magnitudes."""
    mag = x.abs() @ w.abs()
    return rounded(want, (k / 32 + 33) * 2.0 ** -23 * mag, dtype)
