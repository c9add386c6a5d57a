"""Cases of AdamW over a list of tensors (moments in 32 or in 8 bits) and of the gated
feed-forward block with its gradients: what is measured, the operators in plain torch, and
the exact values.

Operators (the "op" of a case):
  adam32  one AdamW step over many tensors, moments in fp32
  adam8   the same with moments in 8 bits, and those read back
  ffn     gated feed-forward block, forward
  train   forward that keeps what the gradients need, then the gradients

Shapes are those of the workloads in synth/workloads.py (GPT-2 1.5B: 1600 x 6400; Llama-3-8B:
4096 x 14336; Llama-2-70B: 8192 x 28672; the tiny list) and generic small ones.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"fp16": 2, "bf16": 2, "fp32": 4}
BETA1, BETA2, EPS = 0.9, 0.999, 1e-8
BLOCK = 128  # elements that share an exponent; tensors start at multiples of it in the moments


# ------------------------------------------------------------------ tensor lists
def _gpt2():
    h, f = 1600, 6400
    t = [50257 * h, 1024 * h]
    for _ in range(48):
        t += [h, h, h * 3 * h, 3 * h, h * h, h, h, h, h * f, f, f * h, h]
    return t + [h, h]


def _sizes(case):
    kind = case["tensors"]
    if kind == "gpt2":
        return _gpt2()
    if kind == "gpt2_vectors":
        return [n for n in _gpt2() if n <= 6400]
    if kind == "llama3_block":
        h, kv, f = 4096, 1024, 14336
        return [h * h, kv * h, kv * h, h * h, f * h, f * h, h * f, h, h]
    if kind == "tiny":
        return [1000 * 1000, 1000, 3]
    g = torch.Generator().manual_seed(case["size_seed"])
    u = torch.rand(case["count"], generator=g, dtype=torch.float64)
    return [int(round(case["low"] * (case["high"] / case["low"]) ** float(x))) for x in u]


def _offsets(sizes):
    """Where each tensor starts in the flat moments, and their length."""
    at, out = 0, []
    for n in sizes:
        out.append(at)
        at += (n + BLOCK - 1) // BLOCK * BLOCK
    return out, at


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the norm weights and biases of GPT-2, kept in full precision: hundreds of short
        # tensors, latency counts
        dict(name="adam32_gpt2_vectors", op="adam32", grad="fp32", out="fp16",
             tensors="gpt2_vectors", loss_scale=1.0, step=1000),
        # one transformer block (an FSDP unit that is not flattened), bf16 gradients
        dict(name="adam32_llama3_block", op="adam32", grad="bf16", out="bf16",
             tensors="llama3_block", loss_scale=1.0, step=20),
        # all of GPT-2 1.5B from loss-scaled fp16 gradients: the longest list
        dict(name="adam32_gpt2", op="adam32", grad="fp16", out="fp16", tensors="gpt2",
             loss_scale=1024.0, step=100000),
        # the tiny workload's list (the last tensor has three elements), first step
        dict(name="adam8_tiny", op="adam8", grad="fp32", out="fp16", tensors="tiny",
             loss_scale=1.0, step=1),
        # the block again, its moments in 8 bits
        dict(name="adam8_llama3_block", op="adam8", grad="bf16", out="bf16",
             tensors="llama3_block", loss_scale=1.0, step=2000),
        # GPT-2 1.5B from fp32 gradients accumulated over micro-batches
        dict(name="adam8_gpt2", op="adam8", grad="fp32", out="fp16", tensors="gpt2",
             loss_scale=1.0, step=30),
        # one token of a reply: the weights are read once
        dict(name="ffn_llama3_1", op="ffn", dtype="bf16", act="silu", tokens=1, hidden=4096,
             inner=14336),
        # a batch of replies on a small model
        dict(name="ffn_gpt2_37", op="ffn", dtype="fp16", act="gelu_tanh", tokens=37, hidden=1600,
             inner=6400),
        # a long prompt (odd length) through the widest block
        dict(name="ffn_llama2_2047", op="ffn", dtype="bf16", act="silu", tokens=2047,
             hidden=8192, inner=28672),
        # a unit-test-sized model: launches and latency count
        dict(name="train_small_50", op="train", dtype="fp16", act="gelu", tokens=50, hidden=72,
             inner=200),
        # one full GPT-2 context
        dict(name="train_gpt2_1024", op="train", dtype="fp16", act="gelu_tanh", tokens=1024,
             hidden=1600, inner=6400),
        # a training micro-batch of Llama-3-8B: the largest products
        dict(name="train_llama3_4096", op="train", dtype="bf16", act="silu", tokens=4096,
             hidden=4096, inner=14336),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["adam32", "adam8", "ffn", "train"])
    if op in ("ffn", "train"):
        # the repository's widths or anything between; tokens from one to a long document, held
        # to the largest listed case's cost
        if rng.random() < 0.4:
            hidden, inner = rng.choice([(1600, 6400), (4096, 14336), (8192, 28672)])
        else:
            hidden = 8 * _log_int(rng, 8, 1024)
            inner = 8 * _log_int(rng, 8, 3584)
            if rng.random() < 0.25:
                hidden += rng.randrange(1, 8)  # widths that no 16-byte row fits
                inner += rng.randrange(0, 8)
        most = 4096 * 4096 * 14336 * (3 if op == "ffn" else 1) / (hidden * inner)
        tokens = _log_int(rng, 1, max(1, min(8192, int(most))))
        return dict(op=op, dtype=rng.choice(["fp16", "bf16"]),
                    act=rng.choice(["silu", "gelu", "gelu_tanh", "relu"]), tokens=tokens,
                    hidden=hidden, inner=inner)
    count = _log_int(rng, 1, 600)
    high = _log_int(rng, 64, max(64, min(200_000_000, 1_000_000_000 // count)))
    return dict(op=op, grad=rng.choice(["fp16", "bf16", "fp32"]),
                out=rng.choice(["fp16", "bf16", "fp32", "none"]), tensors="random", count=count,
                low=rng.choice([1, 1, 32]), high=high, size_seed=rng.randrange(1 << 30),
                loss_scale=rng.choice([1.0, 128.0, 1024.0]),
                step=rng.choice([1, 2, 10, 1000, 100000]))


def work(case):
    if case["op"] in ("ffn", "train"):
        t, h, f = case["tokens"], case["hidden"], case["inner"]
        if case["op"] == "ffn":
            return {"bytes": 2 * (3 * h * f + 2 * t * h), "flops": 6 * t * h * f}
        # x, dy, the weights read; y, dx and the weights' gradients written
        return {"bytes": 2 * (6 * h * f + 4 * t * h), "flops": 18 * t * h * f}
    n = sum(_sizes(case))
    per = SIZE[case["grad"]] + 8 + SIZE.get(case["out"], 0)
    # 8-bit moments: read, written, and read back as 16-bit values
    per += 16 if case["op"] == "adam32" else 4 + 4 / BLOCK + 4
    return {"bytes": n * per, "flops": 18 * n}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ffn_inputs(case, seed):
    """Hidden states after a norm, weights that keep the variance, and a gradient of the
    output as a (scaled) loss leaves it."""
    g = _generator(seed)
    t, h, f = case["tokens"], case["hidden"], case["inner"]
    dt = DTYPES[case["dtype"]]

    def normal(rows, cols, std):
        return (torch.randn(rows, cols, generator=g, device="cuda") * std).to(dt)

    out = {"x": normal(t, h, 1.0), "w_gate": normal(f, h, h ** -0.5),
           "w_up": normal(f, h, h ** -0.5), "w_down": normal(h, f, f ** -0.5)}
    if case["op"] == "train":
        out["dy"] = normal(t, h, 0.05)
    return out


def _decay(i, n):
    """Weight decay of tensor i: none for vectors, as usual."""
    return 0.0 if n <= 6400 else 0.1


def _encode(x, octaves, bits):
    """Values as 8-bit moments, cut off: codes and exponents (the inputs of a later step)."""
    p = (x.abs().view(torch.int32) >> 20).view(-1, BLOCK)
    e = p.amax(1, keepdim=True) >> 3
    code = (p - 8 * (e - (octaves - 1)).clamp(min=0)).clamp(min=0)
    code = code.view(-1)
    if bits == 7:
        code = code | ((x < 0).to(torch.int32) << 7)
    return code.to(torch.uint8), e.view(-1).to(torch.uint8)


def _adam_inputs(case, seed):
    """Gradients, master weights and moments as views of flat buffers, each tensor with its
    own magnitude; the moments are those of a run that is under way (zero at its first step)."""
    g = _generator(seed)
    sizes = _sizes(case)
    n = sum(sizes)
    offsets, total = _offsets(sizes)
    grad = torch.empty(n, dtype=DTYPES[case["grad"]], device="cuda")
    grad.normal_(0.0, 1e-3 * case["loss_scale"], generator=g)
    master = torch.empty(n, dtype=torch.float32, device="cuda").normal_(0.0, 0.02, generator=g)
    m = torch.zeros(total, dtype=torch.float32, device="cuda")
    v = torch.zeros(total, dtype=torch.float32, device="cuda")
    first = case["step"] == 1
    mags = (torch.rand(len(sizes), generator=torch.Generator().manual_seed(seed)) * 4 - 2).tolist()
    at = 0
    for size, off, mag in zip(sizes, offsets, mags):
        s = 2.0 ** mag
        grad[at:at + size].mul_(s)
        if not first:
            m[off:off + size].normal_(0.0, 3e-4 * s, generator=g)
            v[off:off + size].normal_(0.0, 1e-3 * s, generator=g).square_()
        at += size
    out = {"sizes": sizes, "offsets": offsets, "grad": grad, "master": master}
    if case["op"] == "adam32":
        out["m"], out["v"] = m, v
    else:
        out["m"], out["m_exp"] = _encode(m, 16, 7)
        out["v"], out["v_exp"] = _encode(v, 32, 8)
    out["out"] = None
    if case["out"] != "none":
        out["out"] = torch.zeros(n, dtype=DTYPES[case["out"]], device="cuda")
    return out


def prepare(case, seed):
    state = {"case": case}
    if case["op"] in ("ffn", "train"):
        state.update(_ffn_inputs(case, seed))
        if own:
            from zero_sharded_optimizer_rank_amd.ffn import GatedFFN
            state["ffn"] = GatedFFN(case["tokens"], case["hidden"], case["inner"],
                                    DTYPES[case["dtype"]], act=case["act"],
                                    device=state["x"].device, grad=case["op"] == "train")
        return state
    state.update(_adam_inputs(case, seed))
    state["seed"] = seed & 0x7FFFFFFF
    if own:
        from zero_sharded_optimizer_rank_amd.adam import AdamList, AdamState
        sizes = state["sizes"]
        moments = AdamState(sizes, bits=32 if case["op"] == "adam32" else 8,
                            device=state["grad"].device)
        for name in ("m", "v", "m_exp", "v_exp"):
            if name in state:
                getattr(moments, name).copy_(state.pop(name))
        out = state["out"]
        state["moments"] = moments
        state["list"] = AdamList(list(torch.split(state["grad"], sizes)),
                                 list(torch.split(state["master"], sizes)), moments,
                                 params=None if out is None else list(torch.split(out, sizes)),
                                 weight_decay=[_decay(i, n) for i, n in enumerate(sizes)])
    return state


# ------------------------------------------------------------------ the feed-forward block
def _act(name, g):
    if name == "silu":
        return g / (1.0 + torch.exp(-g))
    if name == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * 0.5 ** 0.5))
    if name == "gelu_tanh":
        return 0.5 * g * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (g + 0.044715 * g * g * g)))
    return torch.clamp(g, min=0.0)


def _act_slope(name, g):
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    if name == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g * 0.5 ** 0.5))
        return cdf + g * torch.exp(-0.5 * g * g) * (0.5 / math.pi) ** 0.5
    if name == "gelu_tanh":
        k = (2.0 / math.pi) ** 0.5
        t = torch.tanh(k * (g + 0.044715 * g * g * g))
        return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * g * g)
    return (g > 0).to(g.dtype)


def _plain_ffn(state):
    case = state["case"]
    x, wg, wu, wd = (state[k].float() for k in ("x", "w_gate", "w_up", "w_down"))
    g, u = x @ wg.t(), x @ wu.t()
    a = _act(case["act"], g)
    h = a * u
    out = {"y": h @ wd.t()}
    if case["op"] == "train":
        dy = state["dy"].float()
        dh = dy @ wd
        du = dh * a
        dg = dh * u * _act_slope(case["act"], g)
        out["dx"] = dg @ wg + du @ wu
        out["dw_gate"] = dg.t() @ x
        out["dw_up"] = du.t() @ x
        out["dw_down"] = dy.t() @ h
    return {k: t.to(state["x"].dtype) for k, t in out.items()}


# ------------------------------------------------------------------ AdamW
def _mix(x):
    """A 32-bit mixing function (two multiplications, three shifts) on int64 tensors or
    numbers of 32 bits."""
    x = (x ^ (x >> 16)) * 0x7FEB352D & 0xFFFFFFFF
    x = (x ^ (x >> 15)) * (0x846CA68B - (1 << 32)) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _dither(seed, tensor, n, device):
    """Element i's 32 random bits: those of its 4096-element chunk's key and its place there."""
    i = torch.arange(n, device=device)
    key = _mix((_mix((_mix(seed) + tensor) & 0xFFFFFFFF) + (i >> 12)) & 0xFFFFFFFF)
    return _mix((key + (i & 4095)) & 0xFFFFFFFF)


def _decoded(code, exp, octaves, bits):
    c = code.to(torch.int32)
    sign = (c >> 7) if bits == 7 else torch.zeros_like(c)
    c = c & ((1 << bits) - 1)
    base = 8 * (exp.to(torch.int32) - (octaves - 1)).clamp(min=0)
    base = base.repeat_interleave(BLOCK)[:c.numel()]
    x = torch.where(c > 0, (c + base) << 20, torch.zeros_like(c)).view(torch.float32)
    return torch.where(sign > 0, -x, x)


def _rounded(x, dither16, octaves, bits):
    """Stochastic rounding to 3 mantissa bits: the pattern plus random bits below them."""
    n = x.numel()
    p = ((x.abs().view(torch.int32) + (dither16 << 4) + 8) >> 20).to(torch.int32)
    blocks = (n + BLOCK - 1) // BLOCK
    e = torch.nn.functional.pad(p, (0, blocks * BLOCK - n)).view(-1, BLOCK).amax(1) >> 3
    base = (8 * (e - (octaves - 1)).clamp(min=0)).repeat_interleave(BLOCK)[:n]
    code = (p - base).clamp(min=0)
    if bits == 7:
        code = code | ((x < 0).to(torch.int32) << 7)
    else:
        code = torch.where(x > 0, code.clamp(min=1), code)  # no second moment becomes zero
    return code.to(torch.uint8), e.to(torch.uint8)


def _updated(case, i, n, g, p, m, v, device):
    """The formulas in fp32, one rounding an operation."""
    t, lr = case["step"], 1e-3
    g = g.float() * (1.0 / case["loss_scale"])
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * g) * (1.0 - BETA2)
    root = torch.tensor(math.sqrt(1.0 - BETA2 ** t), dtype=torch.float32, device=device)
    den = torch.sqrt(v) / root + EPS
    p = p * (1.0 - lr * _decay(i, n)) - (m / den) * (lr / (1.0 - BETA1 ** t))
    return p, m, v


def _plain_adam(state):
    case = state["case"]
    wide = case["op"] == "adam32"
    device = state["grad"].device
    if not wide:
        read_m = torch.zeros(state["m"].numel(), dtype=torch.bfloat16, device=device)
        read_v = torch.zeros_like(read_m)
    at = 0
    for i, (n, off) in enumerate(zip(state["sizes"], state["offsets"])):
        here, mom = slice(at, at + n), slice(off, off + n)
        exps = slice(off // BLOCK, (off + n + BLOCK - 1) // BLOCK)
        m, v = state["m"][mom], state["v"][mom]
        if not wide:
            m = _decoded(m, state["m_exp"][exps], 16, 7)
            v = _decoded(v, state["v_exp"][exps], 32, 8)
        p, m, v = _updated(case, i, n, state["grad"][here], state["master"][here], m, v, device)
        state["master"][here] = p
        if state["out"] is not None:
            state["out"][here] = p.to(state["out"].dtype)
        if wide:
            state["m"][mom], state["v"][mom] = m, v
        else:
            d = _dither(state["seed"], i, n, device)
            m, me = _rounded(m, (d & 0xFFFF).to(torch.int32), 16, 7)
            v, ve = _rounded(v, (d >> 16).to(torch.int32), 32, 8)
            state["m"][mom], state["v"][mom] = m, v
            state["m_exp"][exps], state["v_exp"][exps] = me, ve
            read_m[mom] = _decoded(m, me, 16, 7).to(torch.bfloat16)
            read_v[mom] = _decoded(v, ve, 32, 8).to(torch.bfloat16)
        at += n
    out = {"master": state["master"], "m": state["m"] if wide else read_m,
           "v": state["v"] if wide else read_v}
    if state["out"] is not None:
        out["param"] = state["out"]
    return out


def run(state):
    case = state["case"]
    if not own:
        return _plain_ffn(state) if case["op"] in ("ffn", "train") else _plain_adam(state)
    if case["op"] in ("ffn", "train"):
        f, weights = state["ffn"], (state["w_gate"], state["w_up"], state["w_down"])
        if case["op"] == "ffn":
            return {"y": f.forward(state["x"], *weights).y}
        r = f.forward(state["x"], *weights, save=True)
        d = f.backward(state["dy"], state["x"], *weights, r.saved)
        return {"y": r.y, "dx": d.dx, "dw_gate": d.dw_gate, "dw_up": d.dw_up,
                "dw_down": d.dw_down}
    lst, moments = state["list"], state["moments"]
    lst.step(lr=1e-3, beta1=BETA1, beta2=BETA2, eps=EPS, step=case["step"],
             loss_scale=case["loss_scale"], seed=state["seed"])
    m, v = (moments.m, moments.v) if case["op"] == "adam32" else lst.moments()
    out = {"master": state["master"], "m": m, "v": v}
    if state["out"] is not None:
        out["param"] = state["out"]
    return out


# ------------------------------------------------------------------ exact values
def _exact_ffn(case, seed):
    s = _ffn_inputs(case, seed)
    x, wg, wu, wd = (s[k].double() for k in ("x", "w_gate", "w_up", "w_down"))
    g, u = torch.matmul(x, wg.t()), torch.matmul(x, wu.t())
    name = case["act"]
    if name == "silu":
        sig = torch.sigmoid(g)
        a, slope = g * sig, sig + g * sig * (1 - sig)
    elif name == "gelu":
        cdf = torch.special.ndtr(g)
        a, slope = g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    elif name == "gelu_tanh":
        # (1 + tanh z) / 2 is the logistic function of 2 z
        z = math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)
        sig = torch.sigmoid(z)
        dz = math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * g ** 2)
        a, slope = g * sig, sig + g * sig * (1 - sig) * dz
    else:
        slope = torch.where(g > 0, 1.0, 0.0).double()
        a = g * slope
    h = a * u
    out = {"y": torch.matmul(h, wd.t())}
    if case["op"] == "train":
        dy = s["dy"].double()
        out["dw_down"] = torch.matmul(dy.t(), h)
        del h
        dh = torch.matmul(dy, wd)
        dg, du = slope * u * dh, a * dh
        out["dx"] = torch.matmul(dg, wg) + torch.matmul(du, wu)
        out["dw_gate"] = torch.matmul(dg.t(), x)
        out["dw_up"] = torch.matmul(du.t(), x)
    return out


def _exact_moment(code, exp, octaves, signed):
    """The value of 8-bit moments in fp64, from sign, exponent and fraction."""
    c = code.double()
    neg = torch.zeros_like(c)
    if signed:
        neg = torch.floor(c / 128)
        c = c - 128 * neg
    lift = torch.clamp(exp.double() - (octaves - 1), min=0).repeat_interleave(BLOCK)[:c.numel()]
    field = torch.floor(c / 8) + lift          # fp32's biased exponent
    frac = c - 8 * torch.floor(c / 8)
    x = torch.where(field > 0, (1 + frac / 8) * torch.exp2(field - 127), frac / 8 * 2.0 ** -126)
    return torch.where(c > 0, x, 0.0) * (1 - 2 * neg)


def _exact_rounded(x, share, octaves, signed):
    """The 8-bit value of an fp64 moment: `share` of the gap to the next value above decides
    (up where the part of the gap that x has passed and the share make a whole)."""
    n = x.numel()
    mant, ex = torch.frexp(x.abs())
    normal = ex > -126
    field = torch.where(normal, ex.double() + 126, 0.0)
    frac = torch.where(normal, 2 * mant - 1, x.abs() * 2.0 ** 126)
    steps = torch.where(x == 0, 0.0, torch.floor(8 * (field + frac) + share))
    blocks = (n + BLOCK - 1) // BLOCK
    top = torch.nn.functional.pad(steps, (0, blocks * BLOCK - n)).view(-1, BLOCK).amax(1)
    exp = torch.floor(top / 8)
    lift = torch.clamp(exp - (octaves - 1), min=0).repeat_interleave(BLOCK)[:n]
    code = torch.clamp(steps - 8 * lift, min=0)
    if signed:
        code = code + torch.where(x < 0, 128.0, 0.0)
    else:
        code = torch.where((x > 0) & (code < 1), 1.0, code)
    return _exact_moment(code, exp, octaves, signed)


def _exact_adam(case, seed):
    s = _adam_inputs(case, seed)
    t, lr = case["step"], 1e-3
    dev = s["grad"].device
    new_p = torch.empty(s["grad"].numel(), dtype=torch.float64, device=dev)
    new_m = torch.zeros(s["m"].numel(), dtype=torch.float64, device=dev)
    new_v = torch.zeros_like(new_m)
    at = 0
    for i, (n, off) in enumerate(zip(s["sizes"], s["offsets"])):
        m, v = s["m"][off:off + n], s["v"][off:off + n]
        if case["op"] == "adam8":
            e0, e1 = off // BLOCK, (off + n + BLOCK - 1) // BLOCK
            m = _exact_moment(m, s["m_exp"][e0:e1], 16, True)
            v = _exact_moment(v, s["v_exp"][e0:e1], 32, False)
        g = s["grad"][at:at + n].double() / case["loss_scale"]
        m = BETA1 * m.double() + (1 - BETA1) * g
        v = BETA2 * v.double() + (1 - BETA2) * g * g
        mhat, vhat = m / (1 - BETA1 ** t), v / (1 - BETA2 ** t)
        p = s["master"][at:at + n].double()
        new_p[at:at + n] = p - lr * (mhat / (torch.sqrt(vhat) + EPS) + _decay(i, n) * p)
        if case["op"] == "adam8":
            d = _dither(seed & 0x7FFFFFFF, i, n, dev)  # random numbers: an input
            m = _exact_rounded(m, ((d & 0xFFFF).double() + 0.5) / 65536, 16, True)
            v = _exact_rounded(v, ((d >> 16).double() + 0.5) / 65536, 32, False)
        new_m[off:off + n], new_v[off:off + n] = m, v
        at += n
    out = {"master": new_p, "m": new_m, "v": new_v}
    if s["out"] is not None:
        out["param"] = new_p.clone()
    return out


def exact(case, seed):
    """The values of the first pass over the inputs of this seed."""
    if case["op"] in ("ffn", "train"):
        return _exact_ffn(case, seed)
    return _exact_adam(case, seed)
