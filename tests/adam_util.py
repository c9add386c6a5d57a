"""The list update on the CPU: in fp32 with one rounding an operation (numpy), the 8-bit moments
with their hash, and in 64 bits with bounds for what the fp32 roundings can move."""
import numpy as np

BLOCK = 128
E = 2.0 ** -24  # half a step of fp32, relative


def mix(x):
    x = np.asarray(x, dtype=np.uint32).copy()
    with np.errstate(over="ignore"):
        x ^= x >> np.uint32(16)
        x *= np.uint32(0x7FEB352D)
        x ^= x >> np.uint32(15)
        x *= np.uint32(0x846CA68B)
        x ^= x >> np.uint32(16)
    return x


def random_bits(seed, tensor, start, n):
    i = np.arange(start, start + n, dtype=np.uint64)
    with np.errstate(over="ignore"):
        key = mix(mix(np.uint32(seed)) + np.uint32(tensor))
        key = mix(key + (i >> np.uint64(12)).astype(np.uint32))
        return mix(key + (i & np.uint64(4095)).astype(np.uint32))


def decode(code, exp, octaves, bits, n=None):
    code = np.asarray(code, dtype=np.uint32)
    n = code.size if n is None else n
    base = 8 * np.maximum(np.asarray(exp, dtype=np.int64) - (octaves - 1), 0)
    base = np.repeat(base, BLOCK)[:n].astype(np.uint32)
    a = code & np.uint32((1 << bits) - 1)
    x = np.where(a > 0, (a + base) << np.uint32(20), np.uint32(0))
    if bits == 7:
        x = x | (code >> np.uint32(7)) << np.uint32(31)
    return x.astype(np.uint32).view(np.float32)


def encode(x, random16, octaves, bits):
    """Codes and exponents of fp32 values (a tensor's, from its start)."""
    x = np.asarray(x, dtype=np.float32)
    n = x.size
    pattern = x.view(np.uint32).astype(np.uint64) & np.uint64(0x7FFFFFFF)
    p = (pattern + (random16.astype(np.uint64) << np.uint64(4)) + np.uint64(8)) >> np.uint64(20)
    p = np.minimum(p, 0x7FF).astype(np.int64)
    blocks = -(-n // BLOCK)
    padded = np.zeros(blocks * BLOCK, dtype=np.int64)
    padded[:n] = p
    exp = padded.reshape(blocks, BLOCK).max(axis=1) >> 3
    base = np.repeat(8 * np.maximum(exp - (octaves - 1), 0), BLOCK)[:n]
    code = np.maximum(p - base, 0)
    if bits == 7:
        code |= (x.view(np.uint32) >> 31).astype(np.int64) << 7
    else:
        code = np.where(x > 0, np.maximum(code, 1), code)
    return code.astype(np.uint8), exp.astype(np.uint8)


def scalars(lr, b1, b2, eps, step, loss_scale, wd, lr_scale, coef):
    f = np.float32
    return dict(b1=f(b1), omb1=f(1.0 - b1), b2=f(b2), omb2=f(1.0 - b2), eps=f(eps),
                root=f((1.0 - b2 ** step) ** 0.5), scale=f(1.0 / loss_scale), c=f(coef),
                step_size=f(lr / (1.0 - b1 ** step) * lr_scale),
                decay=f(1.0 - lr * (lr_scale * wd)))


def update32(g, p, m, v, s):
    """fp32 arrays; every operation rounded once."""
    with np.errstate(all="ignore"):
        gc = (g * s["scale"]) * s["c"]
        m = s["b1"] * m + s["omb1"] * gc
        v = s["b2"] * v + s["omb2"] * (gc * gc)
        den = np.sqrt(v) / s["root"] + s["eps"]
        p = p * s["decay"] - (m / den) * s["step_size"]
    return p, m, v


def update64(g, p, m, v, s, bits=32):
    """The same in fp64 with the fp32 scalars, and how far each fp32 result can be off.

    Roundings (each at most E relative to its result): gc two; m the products b1 m (one) and
    (1-b1) gc (one more than gc's two) and their sum; v's terms are positive, gc^2 carries twice
    gc's two and one, its product one, the sum one, under 8 E in all; the root halves that and
    adds one, the division and the sum with eps one each, under 7 E; the division, the product,
    then p's product and the difference.  1.01 covers the second order.

    With 8-bit moments the root and the reciprocals are off by one unit in the last place (2 E):
    the root 4 E + 2 E, the product with the rounded 1 / root two more (and one for this
    reference's own rounded root), the sum with eps one, the reciprocal 2 E, its product and
    the next one each: 14 E."""
    s = {k: np.float64(x) for k, x in s.items()}
    g, p, m, v = (np.asarray(x, dtype=np.float64) for x in (g, p, m, v))
    gc = g * s["scale"] * s["c"]
    m1 = s["b1"] * m + s["omb1"] * gc
    dm = E * (np.abs(s["b1"] * m) + np.abs(m1) + 3 * np.abs(s["omb1"] * gc))
    v1 = s["b2"] * v + s["omb2"] * gc * gc
    dv = 8 * E * v1
    den = np.sqrt(v1) / s["root"] + s["eps"]
    u = m1 / den * s["step_size"]
    du = np.abs(u) * (9 if bits == 32 else 14) * E + dm / den * s["step_size"]
    p1 = p * s["decay"] - u
    dp = E * (np.abs(p * s["decay"]) + np.abs(p1)) + du
    return (p1, m1, v1), tuple(1.01 * d for d in (dp, dm, dv))
