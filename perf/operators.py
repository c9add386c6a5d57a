"""Cases of the language-model head's loss and of the many-tensor gradient norm
and clip: what is measured, the operators in plain torch, and the exact values.

Operators (the "op" of a case):
  loss   softmax cross entropy of a language-model head, loss alone
  grad   the same with the gradients of the hidden states and of the weight
  norm   global gradient norm over many tensors, with each tensor's own squares
  clip   that norm, and the tensors unscaled, clipped and cast into their rows

Shapes are those of the workloads in synth/workloads.py (GPT-2 1.5B: 50257 x
1600; Llama-3-8B: 128256 x 4096; Llama-2-70B: 32000 x 8192; the tiny list) and
generic small ones.
"""
import math

import torch

own = False

IGNORE = -100  # the label of a token that takes no part
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"fp16": 2, "bf16": 2, "fp32": 4}
CLIP_EPS = 1e-6


# ------------------------------------------------------------------ tensor lists
def _gpt2():
    h, f = 1600, 6400
    t = [50257 * h, 1024 * h]
    for _ in range(48):
        t += [h, h, h * 3 * h, 3 * h, h * h, h, h, h, h * f, f, f * h, h]
    return t + [h, h]


def _gpt2_vectors():
    return [n for n in _gpt2() if n <= 6400]


def _llama3_block():
    h, kv, f = 4096, 1024, 14336
    return [h * h, kv * h, kv * h, h * h, f * h, f * h, h * f, h, h]


def _tiny():
    return [1000 * 1000, 1000, 3]


def _random_sizes(seed, count, low, high):
    g = torch.Generator().manual_seed(seed)
    u = torch.rand(count, generator=g, dtype=torch.float64)
    return [int(round(low * (high / low) ** float(x))) for x in u]


def _sizes(case):
    kind = case["tensors"]
    if kind == "gpt2":
        return _gpt2()
    if kind == "gpt2_vectors":
        return _gpt2_vectors()
    if kind == "llama3_block":
        return _llama3_block()
    if kind == "tiny":
        return _tiny()
    if kind == "flat":
        return [case["count"]]
    return _random_sizes(case["size_seed"], case["count"], case["low"], case["high"])


# ------------------------------------------------------------------ cases
def listed():
    return [
        # evaluation of one short prompt: few rows, the weight is read once
        dict(name="loss_gpt2_37", op="loss", dtype="fp16", tokens=37, vocab=50257, hidden=1600,
             ignored=0.0, mean=True),
        # perplexity of one long document; the prompt's part is not scored
        dict(name="loss_llama3_8192", op="loss", dtype="bf16", tokens=8192, vocab=128256,
             hidden=4096, ignored=0.1, mean=True),
        # a unit-test-sized model: launches and latency count
        dict(name="grad_small_50", op="grad", dtype="fp16", tokens=50, vocab=1000, hidden=72,
             ignored=0.0, mean=True, loss_scale=1024.0),
        # one full GPT-2 context under fp16 loss scaling (odd vocabulary)
        dict(name="grad_gpt2_1024", op="grad", dtype="fp16", tokens=1024, vocab=50257,
             hidden=1600, ignored=0.0, mean=True, loss_scale=65536.0),
        # a packed batch with next-token labels (odd count), wide hidden state, small vocabulary
        dict(name="grad_llama2_2047", op="grad", dtype="bf16", tokens=2047, vocab=32000,
             hidden=8192, ignored=0.0, mean=True, loss_scale=1.0),
        # a padded batch over the largest vocabulary: the largest case
        dict(name="grad_llama3_4096", op="grad", dtype="bf16", tokens=4096, vocab=128256,
             hidden=4096, ignored=0.2, mean=True, loss_scale=1.0),
        # the norm weights and biases of GPT-2: hundreds of short tensors, latency counts
        dict(name="norm_gpt2_vectors", op="norm", dtype="fp32", tensors="gpt2_vectors",
             loss_scale=1.0, max_norm=1.0),
        # every gradient of GPT-2 1.5B as the backward pass leaves it, loss-scaled fp16
        dict(name="norm_gpt2_fp16", op="norm", dtype="fp16", tensors="gpt2", loss_scale=1024.0,
             max_norm=1.0),
        # one rank's accumulated fp32 gradient of Llama-3-8B over 8 ranks, one flat tensor
        dict(name="norm_flat_fp32", op="norm", dtype="fp32", tensors="flat", count=1003782656,
             loss_scale=1.0, max_norm=1.0),
        # the tiny workload's list (the last tensor has three elements)
        dict(name="clip_tiny", op="clip", dtype="fp32", out="fp16", tensors="tiny",
             loss_scale=1.0, max_norm=1.0, out_scale=1024.0),
        # one transformer block's bf16 gradients (an FSDP unit) into its contribution row
        dict(name="clip_llama3_block", op="clip", dtype="bf16", out="bf16",
             tensors="llama3_block", loss_scale=1.0, max_norm=1.0, out_scale=1.0),
        # fp32 gradients accumulated over micro-batches, packed as fp16 contributions that
        # carry the loss scale again
        dict(name="clip_gpt2_pack", op="clip", dtype="fp32", out="fp16", tensors="gpt2",
             loss_scale=1.0, max_norm=1.0, out_scale=65536.0),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["loss", "grad", "norm", "clip"])
    if op in ("loss", "grad"):
        # vocabulary and width of the repository's models or anything between; tokens from one
        # to a long document, held to the largest listed case's cost
        vocab = rng.choice([50257, 128256, 32000, _log_int(rng, 300, 128256)])
        hidden = 8 * _log_int(rng, 8, 1024)
        if rng.random() < 0.25:
            hidden += rng.randrange(1, 8)  # a width that no 16-byte row fits
        most = 4096 * 128256 * 4096 / (vocab * hidden)
        tokens = _log_int(rng, 1, max(1, min(8192, int(most))))
        case = dict(op=op, dtype=rng.choice(["fp16", "bf16"]), tokens=tokens, vocab=vocab,
                    hidden=hidden, ignored=rng.choice([0.0, 0.1, 0.5]),
                    mean=rng.random() < 0.75)
        if op == "grad":
            # fp16 carries a loss scale that keeps the gradients in its range
            case["loss_scale"] = 1.0
            if case["dtype"] == "fp16":
                case["loss_scale"] = rng.choice([1.0, 8.0, 64.0])
                if case["mean"]:
                    case["loss_scale"] *= 2.0 ** int(math.log2(tokens))
        return case
    count = _log_int(rng, 1, 600)
    high = _log_int(rng, 64, max(64, min(200_000_000, 1_000_000_000 // count)))
    case = dict(op=op, dtype=rng.choice(["fp16", "bf16", "fp32"]), tensors="random", count=count,
                low=rng.choice([1, 1, 32]), high=high, size_seed=rng.randrange(1 << 30),
                loss_scale=rng.choice([1.0, 128.0, 1024.0]), max_norm=rng.choice([0.0, 0.5, 1.0]))
    if op == "clip":
        case["out"] = rng.choice(["fp16", "bf16", "fp32"])
        case["out_scale"] = 1024.0 if case["out"] == "fp16" else 1.0
    return case


def work(case):
    if case["op"] in ("loss", "grad"):
        t, v, h = case["tokens"], case["vocab"], case["hidden"]
        s = SIZE[case["dtype"]]
        valid = t - round(t * case["ignored"])
        if case["op"] == "loss":
            return {"bytes": s * h * (t + v) + 16 * t, "flops": 2 * valid * v * h}
        # the logits, the hidden states' gradient and the weight's: three products
        return {"bytes": 2 * s * h * (t + v) + 16 * t, "flops": 6 * valid * v * h}
    sizes = _sizes(case)
    n = sum(sizes)
    if case["op"] == "norm":
        return {"bytes": n * SIZE[case["dtype"]] + 8 * len(sizes), "flops": 2 * n}
    return {"bytes": n * (SIZE[case["dtype"]] + SIZE[case["out"]]), "flops": 4 * n}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _head_inputs(case, seed):
    """Hidden states after a final norm (unit variance), a weight of std 0.02, and labels
    that a partly trained model finds: each hidden state leans towards its label's row by
    a different amount, so some tokens are near certain and some near the uniform loss."""
    g = _generator(seed)
    t, v, h = case["tokens"], case["vocab"], case["hidden"]
    dt = DTYPES[case["dtype"]]
    w = (torch.randn(v, h, generator=g, device="cuda", dtype=torch.float32) * 0.02).to(dt)
    y = torch.randint(0, v, (t,), generator=g, device="cuda")
    x = torch.randn(t, h, generator=g, device="cuda", dtype=torch.float32)
    lean = torch.rand(t, 1, generator=g, device="cuda") * 16.0 / (0.0004 * h)
    x = (x + lean * w[y].float()).to(dt)
    gone = round(t * case["ignored"])
    if gone:
        y[torch.randperm(t, generator=g, device="cuda")[:gone]] = IGNORE
    return x, w, y


def _grad_inputs(case, seed):
    """Gradients as views of one flat buffer, each tensor with its own magnitude."""
    g = _generator(seed)
    sizes = _sizes(case)
    flat = torch.empty(sum(sizes), dtype=DTYPES[case["dtype"]], device="cuda")
    flat.normal_(0.0, 1e-3 * case["loss_scale"], generator=g)
    parts = list(torch.split(flat, sizes))
    mags = torch.rand(len(sizes), generator=torch.Generator().manual_seed(seed)) * 4 - 2
    for p, m in zip(parts, mags.tolist()):
        p.mul_(2.0 ** m)
    return sizes, flat, parts


def prepare(case, seed):
    state = {"case": case}
    if case["op"] in ("loss", "grad"):
        x, w, y = _head_inputs(case, seed)
        state.update(x=x, w=w, y=y)
        if own:
            from zero_sharded_optimizer_rank_amd.head import LossHead
            state["head"] = LossHead(case["tokens"], case["hidden"], case["vocab"],
                                     DTYPES[case["dtype"]], device=x.device,
                                     grad=case["op"] == "grad")
        return state
    sizes, flat, parts = _grad_inputs(case, seed)
    state.update(sizes=sizes, parts=parts)
    if case["op"] == "clip":
        state["row"] = torch.empty(flat.numel(), dtype=DTYPES[case["out"]], device="cuda")
    if own:
        from zero_sharded_optimizer_rank_amd.tensors import GradList
        out = list(torch.split(state["row"], sizes)) if case["op"] == "clip" else None
        state["list"] = GradList(parts, out=out)
    return state


# ------------------------------------------------------------------ one pass
def _plain_head(case, x, w, y):
    valid = y >= 0
    label = torch.where(valid, y, torch.zeros_like(y))
    xf, wf = x.float(), w.float()
    logits = xf @ wf.t()
    top = logits.amax(dim=1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(dim=1, keepdim=True)
    lse = torch.log(total) + top
    picked = logits.gather(1, label[:, None])
    zero = torch.zeros((), device=x.device)
    token = torch.where(valid, (lse - picked)[:, 0], zero)
    lse = torch.where(valid, lse[:, 0], zero)
    count = valid.sum()
    divisor = count.clamp(min=1).double() if case["mean"] else torch.ones(
        (), dtype=torch.float64, device=x.device)
    out = {"loss": (token.sum(dtype=torch.float64) / divisor).float(), "token_loss": token,
           "lse": lse, "valid": count}
    if case["op"] == "grad":
        d = e / total
        d.scatter_add_(1, label[:, None], torch.full_like(picked, -1.0))
        d *= (torch.where(valid, case["loss_scale"], 0.0) / divisor).float()[:, None]
        out["dx"] = (d @ wf).to(x.dtype)
        out["dw"] = (d.t() @ xf).to(w.dtype)
    return out


def _plain_norm(case, parts):
    inv = 1.0 / case["loss_scale"]
    squares = []
    for p in parts:
        f = p.double()  # the sum runs over up to a thousand million squares
        squares.append((f * f).sum())
    squares = torch.stack(squares)
    norm = torch.sqrt(squares.sum() * inv * inv)
    coef = torch.ones_like(norm)
    if case["max_norm"] > 0:
        coef = torch.clamp(case["max_norm"] / (norm + CLIP_EPS), max=1.0)
    return {"norm": norm, "clip_coef": coef.float(), "tensor_sq": squares * inv * inv}


def run(state):
    case = state["case"]
    if case["op"] in ("loss", "grad"):
        x, w, y = state["x"], state["w"], state["y"]
        if not own:
            return _plain_head(case, x, w, y)
        if case["op"] == "loss":
            r = state["head"].loss(x, w, y, mean=case["mean"])
            return {"loss": r.loss, "token_loss": r.token_loss, "lse": r.lse, "valid": r.valid}
        r = state["head"].loss_grad(x, w, y, mean=case["mean"], loss_scale=case["loss_scale"])
        return {"loss": r.loss, "token_loss": r.token_loss, "lse": r.lse, "valid": r.valid,
                "dx": r.dx, "dw": r.dw}
    if own:
        lst = state["list"]
        if case["op"] == "norm":
            r = lst.norm(max_grad_norm=case["max_norm"], loss_scale=case["loss_scale"])
            return {"norm": r.norm, "clip_coef": r.clip_coef, "tensor_sq": r.tensor_sq}
        r = lst.norm_clip(max_grad_norm=case["max_norm"], loss_scale=case["loss_scale"],
                          out_scale=case["out_scale"])
        return {"norm": r.norm, "clip_coef": r.clip_coef, "tensor_sq": r.tensor_sq,
                "row": state["row"]}
    out = _plain_norm(case, state["parts"])
    if case["op"] == "clip":
        inv = case["out_scale"] / case["loss_scale"]
        at = 0
        for p in state["parts"]:
            state["row"][at:at + p.numel()] = (p.float() * inv * out["clip_coef"]).to(
                state["row"].dtype)
            at += p.numel()
        out["row"] = state["row"]
    return out


# ------------------------------------------------------------------ exact values
def _exact_head(case, x, w, y):
    """The definition in 64 bits, the vocabulary taken in strips."""
    t, v, h = case["tokens"], case["vocab"], case["hidden"]
    keep = torch.nonzero(y >= 0)[:, 0]
    n = keep.numel()
    dev = x.device
    token = torch.zeros(t, dtype=torch.float64, device=dev)
    lse_all = torch.zeros(t, dtype=torch.float64, device=dev)
    xd = x[keep].double()
    label = y[keep]
    strip = max(1, min(v, (1 << 27) // max(n, 1)))
    big = torch.full((n,), -math.inf, dtype=torch.float64, device=dev)
    acc = torch.zeros(n, dtype=torch.float64, device=dev)
    at_label = torch.zeros(n, dtype=torch.float64, device=dev)
    for v0 in range(0, v, strip):
        l = xd @ w[v0:v0 + strip].double().t()
        new = torch.maximum(big, l.amax(1)) if n else big
        acc = acc * torch.exp(big - new) + torch.exp(l - new[:, None]).sum(1)
        big = new
        here = (label >= v0) & (label < v0 + strip)
        rows = torch.nonzero(here)[:, 0]
        at_label[rows] = l[rows, label[rows] - v0]
    lse = torch.log(acc) + big
    token[keep] = lse - at_label
    lse_all[keep] = lse
    div = float(max(n, 1)) if case["mean"] else 1.0
    out = {"loss": token.sum() / div, "token_loss": token, "lse": lse_all,
           "valid": torch.tensor(n, device=dev)}
    if case["op"] == "grad":
        c = case["loss_scale"] / div
        dx = torch.zeros(t, h, dtype=torch.float64, device=dev)
        dxk = torch.zeros(n, h, dtype=torch.float64, device=dev)
        dw = torch.empty(v, h, dtype=torch.float64, device=dev)
        for v0 in range(0, v, strip):
            ws = w[v0:v0 + strip].double()
            d = torch.exp(xd @ ws.t() - lse[:, None])
            rows = torch.nonzero((label >= v0) & (label < v0 + strip))[:, 0]
            d[rows, label[rows] - v0] -= 1.0
            d *= c
            dxk += d @ ws
            dw[v0:v0 + strip] = d.t() @ xd
        dx[keep] = dxk
        out["dx"], out["dw"] = dx, dw
    return out


def exact(case, seed):
    if case["op"] in ("loss", "grad"):
        return _exact_head(case, *_head_inputs(case, seed))
    sizes, _, parts = _grad_inputs(case, seed)
    squares = []
    for p in parts:
        s = torch.zeros((), dtype=torch.float64, device=p.device)
        for a in range(0, p.numel(), 1 << 26):
            d = p[a:a + (1 << 26)].double()
            s = s + torch.dot(d, d)
        squares.append(s / case["loss_scale"] ** 2)
    squares = torch.stack(squares)
    norm = squares.sum().sqrt()
    coef = 1.0
    if case["max_norm"] > 0:
        coef = torch.clamp(case["max_norm"] / (norm + CLIP_EPS), max=1.0)
    out = {"norm": norm, "clip_coef": torch.as_tensor(coef, dtype=torch.float64,
                                                      device=norm.device),
           "tensor_sq": squares}
    if case["op"] == "clip":
        row = torch.empty(sum(sizes), dtype=torch.float64, device=norm.device)
        at = 0
        for p in parts:
            for a in range(0, p.numel(), 1 << 26):
                d = p[a:a + (1 << 26)].double()
                row[at:at + d.numel()] = d * (coef * (case["out_scale"] / case["loss_scale"]))
                at += d.numel()
        out["row"] = row
    return out
