"""The gated feed-forward block in 64 bits, with elementwise error bounds for the library's
arithmetic.

u is half a step of the 16-bit type relative to the value (finfo.eps / 2), tiny half its smallest
step, e = 2^-23 bounds one fp32 operation (the matrix cores may truncate); a length-n fp32 sum of
terms a_i is off by at most n e sum |a_i|.

g          bg = H e (|x| |Wg|^T) (16-bit products are exact in fp32); u's likewise bu
a          all slopes are at most 1.2: 1.2 times g's error, and the evaluation: the exponential's
           argument is formed in a few operations, each off by e of itself, of size at most
           2 (|g| + g^2 + |g|^3) for every activation, and some 16 operations follow:
           ea = |a| e (16 + 8 (|g| + g^2 + |g|^3)) + 1e-30 (underflow)
slope      second derivatives are at most 1: g's error, and es = e (1 + |g|) (16 + 8 (|g| + g^2 +
           |g|^3)) (1 + |slope|); relu: wrong by 1 where g is within its error of 0
h          errors of a and u through the product, one fp32 operation, one rounding
kept       a and b = u slope with their errors, rounded to 16 bits of significand (2^-16)
y          h's error through |Wd|, F e (|h| |Wd|^T), one rounding
dh         H e (|dy| |Wd|), not rounded
du, dg     products of dh with the kept a and b, one operation, one rounding
dx         their errors through the weights, 2 F e of the absolute sums, one rounding
dw         errors of dg, du, h through |x| and |dy|, T e of the absolute sums, then the output's
All first order; relative errors of a few u appear in products of two, so a factor 1.05 covers
the products of errors.
"""
import math

import torch

E = 2.0 ** -23


def act(name, g):
    """Value and slope in g's type."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    if name == "gelu":
        c = torch.special.ndtr(g)
        return g * c, c + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (g + 0.044715 * g ** 3))
        return (g * (1 + t) / 2,
                (1 + t) / 2 + g * (1 - t * t) / 2 * k * (1 + 3 * 0.044715 * g * g))
    pos = (g > 0).to(g.dtype)
    return g * pos, pos


def reference(x, wg, wu, wd, name, dy=None):
    """{name: (fp64 value, bound)} on x's device; the weights' gradients before their rounding."""
    dt = x.dtype
    u = torch.finfo(dt).eps / 2
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
    (T, H), F = x.shape, wg.shape[0]
    X, G, U, D = (t.double() for t in (x, wg, wu, wd))
    g, v = X @ G.t(), X @ U.t()
    bg, bv = H * E * (X.abs() @ G.abs().t()), H * E * (X.abs() @ U.abs().t())
    a, slope = act(name, g)
    r = g.abs()
    size = 16 + 8 * (r + r ** 2 + r ** 3)
    ea = a.abs() * E * size + 1e-30

    da = 1.2 * bg + ea
    h = a * v
    bh = da * v.abs() + a.abs() * bv + E * h.abs()
    bh = bh + u * (h.abs() + bh) + tiny
    y = h @ D.t()
    by = bh @ D.abs().t() + F * E * ((h.abs() + bh) @ D.abs().t())
    out = {"u": u, "tiny": tiny, "y": (y, 1.05 * (by + u * y.abs()) + tiny)}
    if dy is None:
        return out
    es = bg + E * (1 + r) * size * (1 + slope.abs())
    if name == "relu":
        es = (r <= bg).double()
    b = v * slope
    db = bv * slope.abs() + v.abs() * es + E * b.abs()
    sa, sb = da + 2.0 ** -16 * (a.abs() + da) + 1e-38, db + 2.0 ** -16 * (b.abs() + db) + 1e-38
    Y = dy.double()
    dh = Y @ D
    bdh = H * E * (Y.abs() @ D.abs())
    du = dh * a
    bdu = bdh * a.abs() + dh.abs() * sa + E * du.abs()
    bdu = 1.05 * (bdu + u * du.abs()) + tiny
    dg = dh * b
    bdg = bdh * b.abs() + dh.abs() * sb + E * dg.abs()
    bdg = 1.05 * (bdg + u * dg.abs()) + tiny
    dx = dg @ G + du @ U
    ag, au = dg.abs() + bdg, du.abs() + bdu
    bx = bdg @ G.abs() + bdu @ U.abs() + 2 * F * E * (ag @ G.abs() + au @ U.abs())
    out["dx"] = (dx, 1.05 * (bx + u * dx.abs()) + tiny)
    n = max(T, 1) * E
    out["dw_gate"] = (dg.t() @ X, 1.05 * (bdg.t() @ X.abs() + n * (ag.t() @ X.abs())))
    out["dw_up"] = (du.t() @ X, 1.05 * (bdu.t() @ X.abs() + n * (au.t() @ X.abs())))
    out["dw_down"] = (Y.t() @ h, 1.05 * (Y.abs().t() @ bh + n * (Y.abs().t() @ (h.abs() + bh))))
    return out


def few_bound(x, wg, wu, wd, name):
    """y, and the bound where h is held in two 16-bit parts: the second is off by u of itself, so h
    by u^2 (and the type's smallest step), and the contraction is over both parts."""
    dt = x.dtype
    u = torch.finfo(dt).eps / 2
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
    H, F = x.shape[1], wg.shape[0]
    X, G, U, D = (t.double() for t in (x, wg, wu, wd))
    g, v = X @ G.t(), X @ U.t()
    bg, bv = H * E * (X.abs() @ G.abs().t()), H * E * (X.abs() @ U.abs().t())
    a = act(name, g)[0]
    r = g.abs()
    da = 1.2 * bg + a.abs() * E * (16 + 8 * (r + r ** 2 + r ** 3)) + 1e-30
    h = a * v
    bh = da * v.abs() + a.abs() * bv + E * h.abs()
    bh = bh + u * u * (h.abs() + bh) + tiny
    y = h @ D.t()
    by = bh @ D.abs().t() + 2 * F * E * ((1 + u) * (h.abs() + bh) @ D.abs().t())
    return h, y, 1.05 * (by + u * y.abs()) + tiny


def check(got, want, bound, name):
    got = got.double()
    err = (got - want).abs()
    over = ~(err <= bound)
    assert not bool(over.any()), (name, int(over.sum()), float(err.max()),
                                  float((err / (bound + 1e-300)).max()))


def check_dw(got, ref, name, base=None):
    """A weight's gradient in its own type; base: what it was added to."""
    want, bound = ref[name]
    if base is not None:
        want = want + base.double()
        bound = bound + E * want.abs()
    if got.dtype == torch.float32:
        bound = bound + E * want.abs()
    else:
        bound = bound + ref["u"] * want.abs() * 1.05 + ref["tiny"]
    check(got, want, bound, name)


def check_norm(got, want, most, name):
    """Independent roundings of mean zero: the relative 2-norm of the error is at most what each
    element's largest relative errors add up to (most), where no cancellation of the whole is."""
    n = want.norm()
    if n:
        off = float((got.double() - want).norm() / n)
        assert off <= most, (name, off, most)
