"""The head's loss and gradients in 64 bits, with elementwise error bounds for
the library's arithmetic.

u is half a step of the 16-bit type relative to the value (finfo.eps / 2),
e = 2^-23 bounds one fp32 operation (the matrix cores may truncate), a length-n
fp32 sum of terms a_i is off by at most n e sum |a_i|.

logits     |dl| <= H e (|x| |w|^T)                (16-bit products are exact in fp32)
lse        the exponentials are off by a relative eexp <= 4e + 2e |l - m| + e/8 |l| (one
           multiply-add with log2 e in fp32, which is off by 1.34e-8 < e/8 of itself, and the
           instruction, whose error is one step),
           their sums by (V + 64) e and the logarithm by 4e (|lse| + |m| + 2):
           |dlse| <= max|dl| + eexp + (V + 64) e + 4e (|lse| + |m| + 2)
loss       |dloss| <= |dlse| + |dl at the label| + 4e (|lse| + |l|)
p          relative r = |dl| + |dlse| + 4e + 4e |l - lse| + e (|l| + |lse|)
g          |dg| <= u |d| + p (r + u) (1 + u) + e |d|: one rounding of the difference and, where
           the exponentials were kept, one of the probability before it; plus half the type's smallest step (fp16, 2^-25 after
           the scale of 2^15)
dx         |g|'s error through |w|, the sum's V e (|g| |w|), the scaling 2e |dx|, the output's u |dx|
           plus half its smallest step
dw         likewise over the tokens
All first order; a factor 1.01 covers the products of errors.
"""
import torch

E = 2.0 ** -23


def reference(x, w, y, loss_scale=1.0, mean=True):
    """fp64 values and bounds on x's device.  x [T, H], w [V, H], y [T] int64."""
    V, H = w.shape
    T = x.shape[0]
    dt = x.dtype
    u = torch.finfo(dt).eps / 2
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2  # half the smallest step
    keep = torch.nonzero((y >= 0) & (y < V))[:, 0]
    n = keep.numel()
    xk, wk, yk = x[keep].double(), w.double(), y[keep]
    out = {"valid": n}
    c = loss_scale / (max(n, 1) if mean else 1)
    l = xk @ wk.t()
    dl = H * E * (xk.abs() @ wk.abs().t())
    if n:
        m = l.amax(1)
        lse = torch.logsumexp(l, 1)
        far = (l - m[:, None]).abs()
        eexp = ((4 * E + 2 * E * far + E / 8 * l.abs()) * torch.exp(l - lse[:, None])).sum(1)
        dlse = dl.amax(1) + eexp + (V + 64) * E + 4 * E * (lse.abs() + m.abs() + 2)
    else:
        lse = dlse = torch.zeros(0, dtype=torch.float64, device=x.device)
    rows = torch.arange(n, device=x.device)
    ly = l[rows, yk]
    tok = lse - ly
    dtok = dlse + dl[rows, yk] + 4 * E * (lse.abs() + ly.abs())
    for name, v, b in (("lse", lse, dlse), ("token_loss", tok, dtok)):
        full, bound = (torch.zeros(T, dtype=torch.float64, device=x.device) for _ in range(2))
        full[keep], bound[keep] = v, 1.01 * b
        out[name] = (full, bound)
    div = max(n, 1) if mean else 1
    out["loss"] = (float(tok.sum()) / div,
                   1.01 * float(dtok.sum()) / div + E * abs(float(tok.sum())) / div)
    p = torch.exp(l - lse[:, None])
    d = p.clone()
    d[rows, yk] -= 1.0
    r = dl + dlse[:, None] + 4 * E + 4 * E * (l - lse[:, None]).abs() \
        + E * (l.abs() + lse.abs()[:, None])
    floor = tiny * 2.0 ** -15 if dt == torch.float16 else tiny
    dg = u * d.abs() + p * (r + u) * (1 + u) + E * d.abs() + 2 * floor
    g = d.abs() + dg
    dxk = c * (d @ wk)
    bx = c * (dg @ wk.abs() + V * E * (g @ wk.abs())) + (2 * E + u) * dxk.abs()
    dx, bdx = (torch.zeros(T, H, dtype=torch.float64, device=x.device) for _ in range(2))
    dx[keep], bdx[keep] = dxk, 1.01 * bx + tiny
    out["dx"] = (dx, bdx)
    dw = c * (d.t() @ xk)
    bw = c * (dg.t() @ xk.abs() + max(n, 1) * E * (g.t() @ xk.abs())) + 2 * E * dw.abs()
    out["dw"] = (dw, 1.01 * bw)           # before the output's rounding
    out["u"], out["tiny"] = u, tiny
    return out


def check(got, want, bound, name):
    got = got.double()
    err = (got - want).abs()
    over = err > bound
    assert not bool(over.any()) and not bool(torch.isnan(got).any()), (
        name, int(over.sum()), float(err.max()), float((err / (bound + 1e-300)).max()))


def check_dw(got, ref, base=None):
    """dw [V, H] in its own type; base: what it was added to."""
    want, bound = ref["dw"]
    if base is not None:
        want = want + base.double()
        bound = bound + E * want.abs()
    if got.dtype == torch.float32:
        bound = bound + E * want.abs()
    else:
        bound = bound + ref["u"] * want.abs() * 1.01 + ref["tiny"]
    check(got, want, bound, "dw")
