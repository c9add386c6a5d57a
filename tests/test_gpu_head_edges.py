"""The head's loss and gradients where sizes, strides and values meet their limits: each case
in both forms of the products (up to 64 tokens, and more), against 64 bits within the bounds of
tests/head_util.py unless stated otherwise."""
import pytest

torch = pytest.importorskip("torch")

from head_util import E, check, check_dw, reference  # noqa: E402
from test_gpu_head import TYPES, _check_loss, _head, _inputs  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _all(r, ref, base=None):
    _check_loss(r, ref)
    check(r.dx, *ref["dx"], "dx")
    check_dw(r.dw, ref, base)


@pytest.mark.parametrize("dtype", TYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("T", [1, 16, 33, 64, 65, 200])
@pytest.mark.parametrize("H,ldx,ldw,shift", [
    (65, 72, 72, 0),     # odd rows that start on 16-byte boundaries, NaN behind each
    (65, 65, 65, 0),     # odd rows, packed: every alignment of 2 bytes
    (64, 64, 64, 1), (136, 144, 139, 4), (8, 8, 8, 0), (1, 1, 1, 3), (7, 8, 16, 0),
])
def test_rows(T, H, ldx, ldw, shift, dtype):
    V = 531
    x, w, y = _inputs(T, V, H, dtype, seed=T + H, ldx=ldx, ldw=ldw, shift=shift)
    _all(_head(T, V, H, dtype).loss_grad(x, w, y), reference(x, w, y))


@pytest.mark.parametrize("dtype", TYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("T", [1, 20, 64])
@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradient_forms_few_tokens(dtype, T, out, accumulate):
    V, H = 600, 107
    x, w, y = _inputs(T, V, H, dtype, seed=3)
    ref = reference(x, w, y, loss_scale=32.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    base = torch.randn(V, H, generator=g, device="cuda").to(
        torch.float32 if out == "f32" else dtype)
    dw = base.clone()
    _head(T, V, H, dtype).loss_grad(x, w, y, loss_scale=32.0, dw=dw, accumulate=accumulate)
    check_dw(dw, ref, base if accumulate else None)


@pytest.mark.parametrize("dtype", TYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("T", [9, 64, 150])
def test_ignored_and_separate_calls(dtype, T):
    V, H = 700, 136
    x, w, y = _inputs(T, V, H, dtype, seed=5)
    y[1::3] = -100
    x[y < 0] = float("nan")
    ref = reference(x, w, y, mean=False)
    h = _head(T, V, H, dtype)
    r = h.loss_grad(x, w, y, mean=False)
    _all(r, ref)
    lse = r.lse.clone()
    assert torch.equal(h.loss(x, w, y, mean=False).lse, lse)
    dx, dw = _head(T, V, H, dtype).grad(x, w, y, lse, mean=False)
    check(dx, *ref["dx"], "dx")
    check_dw(dw, ref)


@pytest.mark.parametrize("dtype", TYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("T", [5, 130])
def test_equal_labels(dtype, T):
    """Every token has the same label: its row of dw takes every token's part."""
    V, H = 300, 72
    x, w, y = _inputs(T, V, H, dtype, seed=12)
    y[:] = 299
    _all(_head(T, V, H, dtype).loss_grad(x, w, y), reference(x, w, y))


@pytest.mark.parametrize("dtype", TYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("T", [30, 130])
@pytest.mark.parametrize("kind", ["label", "inf", "nan"])
def test_bad_values(dtype, T, kind):
    """A bad token spoils the sums and its own rows, never another token's."""
    V, H = 300, 72
    x, w, y = _inputs(T, V, H, dtype, seed=13)
    if kind == "label":
        y[4] = 2 ** 40
    else:
        x[4, 70] = float(kind)
    r = _head(T, V, H, dtype).loss_grad(x, w, y)
    assert r.loss.isnan() and r.token_loss[4].isnan() and r.dw.isnan().any()
    assert r.bad.item() == (kind == "label")
    others = torch.arange(T, device="cuda") != 4
    assert r.token_loss[others].isfinite().all()
    if kind != "label":  # a bad label makes the mean's divisor, so every gradient, NaN
        assert r.dx[4].isnan().all() and r.dx[others].isfinite().all()
    w[17, 3] = float("nan")  # a spoiled weight reaches every token
    assert _head(T, V, H, dtype).loss(x, w, y).token_loss.isnan().all()


@pytest.mark.parametrize("dtype", TYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("T", [20, 130])
def test_infinite_weight_rows(dtype, T):
    """Masked vocabulary entries: rows whose logit is -inf have probability 0 and do not
    disturb the others' loss; as a label such a row costs infinity."""
    V, H = 400, 64
    x, w, y = _inputs(T, V, H, dtype, seed=14)
    x[:, 0] = 1.0
    w[::5] = 0.0
    w[::5, 0] = float("-inf")
    y = y // 5 * 5 + 1  # never a masked one
    keep = torch.arange(V, device="cuda") % 5 != 0
    new = torch.cumsum(keep, 0) - 1
    ref = reference(x, w[keep].contiguous(), new[y])
    h = _head(T, V, H, dtype)
    r = h.loss(x, w, y)
    _check_loss(r, ref)
    y[2] = 10
    r = h.loss(x, w, y)
    assert r.token_loss[2].item() == float("inf") and r.loss.item() == float("inf")
    check(r.lse, *ref["lse"], "lse")


@pytest.mark.parametrize("dtype", TYPES, ids=["f16", "bf16"])
def test_large_logits_many_tokens(dtype):
    T, V, H = 150, 400, 128
    x, w, y = _inputs(T, V, H, dtype, seed=10, lean=400.0)
    _all(_head(T, V, H, dtype).loss_grad(x, w, y), reference(x, w, y))


@pytest.mark.parametrize("T", [3, 70])
@pytest.mark.parametrize("V", [2 ** 21, 2 ** 21 + 1, 3_000_001])
def test_long_vocabulary(T, V):
    """Both sides of the length where few tokens leave their own form."""
    H, dtype = 24, torch.bfloat16
    x, w, y = _inputs(T, V, H, dtype, seed=15)
    y[-1] = V - 1
    _all(_head(T, V, H, dtype).loss_grad(x, w, y), reference(x, w, y))
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T", [7, 64, 256])
def test_replays_with_changing_masks(T):
    """A captured loss_grad that accumulates: every replay adds what an eager call adds."""
    V, H, dtype = 1000, 264, torch.bfloat16
    x, w, y = _inputs(T, V, H, dtype, seed=11)
    h, eager = _head(T, V, H, dtype), _head(T, V, H, dtype)
    dw, want_dw = (torch.zeros(V, H, device="cuda") for _ in range(2))
    h.loss_grad(x, w, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        r = h.loss_grad(x, w, y, dw=dw, accumulate=True)
    for k in range(4):
        x2, _, y2 = _inputs(T, V, H, dtype, seed=60 + k, ignored=0.3 * k)
        if k == 2:
            y2[:] = -100  # no token at all
        x.copy_(x2), y.copy_(y2)
        want = eager.loss_grad(x2, w, y2, dw=want_dw, accumulate=True)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h.res, eager.res) and torch.equal(r.dx, want.dx)
        assert torch.equal(dw, want_dw)


# -------------------------------------------------- offsets past 32 bits

def _rows_of_dw(x, lse64, w_rows, labels_match, c):
    """fp64 gradient rows and the sums of absolute terms they are bounded with."""
    g = torch.exp(x @ w_rows.t() - lse64[:, None]) - labels_match
    return c * (g.t() @ x), c * (g.abs().t() @ x.abs())


@pytest.mark.parametrize("T", [6, 80])
def test_weight_past_32_bits(T):
    """V x H of more than 2^32 elements.  Checked: every loss, dx, and rows of dw from the
    start, the labels and the end.  Bounds: the logits are off by at most H e (|x| |w|^T), all
    else of one probability by less than a tenth of u, its g is rounded at most twice (2 u), the
    output once."""
    V, H, dtype = 1_049_003, 4096, torch.bfloat16
    u = torch.finfo(dtype).eps / 2
    g = torch.Generator(device="cuda").manual_seed(16)
    w = torch.empty(V, H, dtype=dtype, device="cuda")
    for s in range(0, V, 1 << 17):
        w[s:s + (1 << 17)] = torch.randn(min(1 << 17, V - s), H, generator=g,
                                         device="cuda") * H ** -0.5
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y[0], y[-1] = V - 1, 2 ** 32 // H + 1
    x = (torch.randn(T, H, generator=g, device="cuda") + 8 * w[y].float()).to(dtype)
    r = _head(T, V, H, dtype).loss_grad(x, w, y)
    x64 = x.double()
    logits = torch.cat([x64 @ w[s:s + 65536].double().t() for s in range(0, V, 65536)], 1)
    dl = H * E * float(x64.abs().sum(1).max()) * float(w.abs().max())
    assert dl < 2.0  # loose: the largest |w| in every place
    dl = max(H * E * float((x64.abs() @ w[s:s + 65536].double().abs().t()).max())
             for s in range(0, V, 65536))
    lse = torch.logsumexp(logits, 1)
    tok = lse - logits[torch.arange(T, device="cuda"), y]
    dlse = dl + (V + 64) * E + 64 * E * (lse.abs() + 2)
    check(r.lse, lse, 1.01 * dlse, "lse")
    check(r.token_loss, tok, 1.01 * (dlse + dl + 64 * E), "token_loss")
    rel = 2 * u + 0.1 * u + 1.01 * float((dl + dlse).max())
    c = 1.0 / T
    for rows in (torch.arange(0, 700), y.cpu().sort().values, torch.arange(V - 900, V)):
        rows = rows.cuda()
        want, terms = _rows_of_dw(x64, lse, w[rows].double(),
                                  (y[:, None] == rows[None]).double(), c)
        check(r.dw[rows], want, rel * terms + (T * E) * terms + 1.01 * u * want.abs() + 1e-38,
              "dw")
    want, terms = torch.zeros(T, H, dtype=torch.float64, device="cuda"), 0.0
    for s in range(0, V, 65536):
        ws = w[s:s + 65536].double()
        p = torch.exp(logits[:, s:s + 65536] - lse[:, None])
        p -= (y[:, None] == torch.arange(s, s + ws.shape[0], device="cuda")[None]).double()
        want += c * (p @ ws)
        terms = terms + c * (p.abs() @ ws.abs())
    check(r.dx, want, (rel + V * E) * terms + 1.01 * u * want.abs() + 1e-38, "dx")
    del logits, w, r
    torch.cuda.empty_cache()


def test_tokens_past_32_bits():
    """The most tokens a head takes, T x H of more than 2^32 elements: losses and dx of tokens
    from the start, the middle and the end, and the whole dw.  Bounds as above."""
    T, V, H, dtype = 1 << 20, 130, 4104, torch.bfloat16
    u = torch.finfo(dtype).eps / 2
    g = torch.Generator(device="cuda").manual_seed(17)
    x = torch.empty(T, H, dtype=dtype, device="cuda")
    for s in range(0, T, 1 << 16):
        x[s:s + (1 << 16)] = torch.randn(1 << 16, H, generator=g, device="cuda")
    w = (torch.randn(V, H, generator=g, device="cuda") * H ** -0.5).to(dtype)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y[::5] = -100
    dw = torch.empty(V, H, device="cuda")
    r = _head(T, V, H, dtype).loss_grad(x, w, y, mean=False, dw=dw)
    w64, lo = w.double(), w.double().abs()
    want_dw, terms_dw, total = 0.0, 0.0, 0.0
    dl_max = 0.0
    for s in range(0, T, 1 << 16):
        x64 = x[s:s + (1 << 16)].double()
        ys = y[s:s + (1 << 16)]
        keep = (ys >= 0)[:, None]
        l = x64 @ w64.t()
        dl = H * E * float((x64.abs() @ lo.t()).max())
        dl_max = max(dl, dl_max)
        lse = torch.logsumexp(l, 1)
        dlse = dl + (V + 64) * E + 64 * E * (lse.abs() + 2)
        hot = (ys[:, None] == torch.arange(V, device="cuda")[None]).double()
        d = (torch.exp(l - lse[:, None]) - hot) * keep
        tok = (lse - (l * hot).sum(1)) * keep[:, 0]
        total += float(tok.sum())
        check(r.token_loss[s:s + (1 << 16)], tok, 1.01 * (dlse + dl + 64 * E), "token_loss")
        rel = 2.1 * u + 1.01 * (dl + float(dlse.max()))
        want, terms = d @ w64, d.abs() @ lo
        check(r.dx[s:s + (1 << 16)], want, (rel + V * E) * terms + 1.01 * u * want.abs() + 1e-38,
              "dx")
        want_dw = want_dw + d.t() @ x64
        terms_dw = terms_dw + d.abs().t() @ x64.abs()
    n = int((y >= 0).sum())
    assert r.valid.item() == n
    assert abs(r.loss.item() - total) <= n * 3 * dl_max + 1e-5 * total
    check(dw, want_dw, (rel + n * E) * terms_dw + E * want_dw.abs(), "dw")
    del x, r
    torch.cuda.empty_cache()


def test_long_vocabulary_laid_out_again():
    """Rows of w that start anywhere, more of them than one launch has workgroups."""
    T, V, H, dtype = 70, 2 ** 20 + 300, 24, torch.bfloat16
    x, w, y = _inputs(T, V, H, dtype, seed=18, ldw=25)
    y[-1] = V - 1
    _all(_head(T, V, H, dtype).loss_grad(x, w, y), reference(x, w, y))
    torch.cuda.empty_cache()


def test_workspace_grows_on_another_stream():
    """A w that has to be laid out again, after calls on a stream of the caller's."""
    T, V, H, dtype = 100, 900, 264, torch.bfloat16
    x, w, y = _inputs(T, V, H, dtype, seed=19)
    _, odd, _ = _inputs(T, V, H, dtype, seed=19, ldw=265)
    ref = reference(x, w, y)
    h = _head(T, V, H, dtype)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    small = h.ws.numel()
    for m in (w, odd, w):
        r = h.loss_grad(x, m, y, stream=s)
        torch.empty(small, dtype=torch.uint8, device="cuda").fill_(0xFF)
    torch.cuda.synchronize()
    assert h.ws.numel() > small
    _all(r, ref)


@pytest.mark.parametrize("V", [50, 2 ** 21 + 1])
def test_empty_batch(V):
    """No tokens at all, on both sides of the length where few tokens leave their own form."""
    H, dtype = 8, torch.bfloat16
    w = torch.ones(V, H, dtype=dtype, device="cuda")
    x = torch.empty(0, H, dtype=dtype, device="cuda")
    y = torch.empty(0, dtype=torch.int64, device="cuda")
    h = _head(0, V, H, dtype)
    r = h.loss(x, w, y)
    assert r.loss.item() == 0.0 and r.valid.item() == 0 and r.bad.item() == 0
    r = h.loss_grad(x, w, y)
    assert r.loss.item() == 0.0 and (r.dw == 0).all()
    r.dw.fill_(3.0)
    h.loss_grad(x, w, y, dw=r.dw, accumulate=True)
    assert (r.dw == 3.0).all()
    _, dw = h.grad(x, w, y, torch.empty(0, device="cuda"))
    assert (dw == 0).all()


@pytest.mark.parametrize("T,fewer,V,H", [
    (4608, (4352, 4096, 4097, 64), 128256, 64),  # g's piece: one to 4096 tokens, then two
    (2048, (1792, 1), 32000, 8192),              # dx's splits: 1024 tiles, 896 twice over
])
def test_smaller_batches_of_a_large_head(T, fewer, V, H):
    """Counts whose room for g or for dx's sums is larger than that of more tokens."""
    dtype = torch.bfloat16
    h = _head(T, V, H, dtype)
    for t in (T,) + fewer:
        x, w, y = _inputs(t, V, H, dtype, seed=t)
        ref = reference(x, w, y)
        _all(h.loss_grad(x, w, y), ref)
        del ref
        torch.cuda.empty_cache()


def test_captured_call_keeps_its_workspace():
    """A graph is captured, then a w that has to be laid out again makes the head's workspace
    grow: replays still have the memory that they were captured with to themselves."""
    T, V, H, dtype = 200, 900, 264, torch.bfloat16
    x, w, y = _inputs(T, V, H, dtype, seed=20)
    _, odd, _ = _inputs(T, V, H, dtype, seed=20, ldw=265)
    ref = reference(x, w, y)
    h = _head(T, V, H, dtype)
    h.loss_grad(x, w, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        r = h.loss_grad(x, w, y)
    old = h.ws.data_ptr(), h.ws.numel()
    _all(h.loss_grad(x[:50], odd, y[:50]), reference(x[:50], w, y[:50]))
    assert h.ws.numel() == old[1]  # a few tokens read w in place
    _all(h.loss_grad(x[:70], odd, y[:70]), reference(x[:70], w, y[:70]))
    grown = h.ws.data_ptr()
    assert grown != old[0]
    others = [torch.full((old[1],), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(4)]
    for o in others:
        assert o.data_ptr() + o.numel() <= old[0] or o.data_ptr() >= old[0] + old[1]
    for _ in range(3):
        r.dx.zero_(), r.dw.zero_()
        graph.replay()
        _all(r, ref)
        _all(h.loss_grad(x, odd, y), ref)  # the larger batch: no further growth
        assert h.ws.data_ptr() == grown
        torch.cuda.synchronize()
    assert all((o == 0xA5).all() for o in others)


def test_buffers_made_in_a_call_are_its_streams():
    """The first dw and a grown workspace are made while the current stream still writes to
    memory that it has given back: the call on a stream of the caller's takes none of that."""
    from zero_sharded_optimizer_rank_amd import abi
    T, V, H, dtype = 100, 4000, 264, torch.bfloat16
    x, _, y = _inputs(T, V, H, dtype, seed=21)
    _, odd, _ = _inputs(T, V, H, dtype, seed=21, ldw=265)
    ref = reference(x, odd, y)
    h = _head(T, V, H, dtype)
    grown = abi.zero_head_workspace_bytes(
        abi.zero_head_t(T, H, V, 0, H, odd.data_ptr(), 265, 0, abi.ZERO_BF16, 1, 1.0), True)
    assert grown > h.ws.numel()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    given_back = []
    busy = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (2 * V * H, grown)]
    torch.cuda._sleep(20_000_000)
    for b in busy:
        b.fill_(0xFF)
        given_back.append((b.data_ptr(), b.data_ptr() + b.numel()))
    del b, busy
    r = h.loss_grad(x, odd, y, stream=s)
    assert h.ws.numel() == grown
    for t in (r.dw, h.ws):
        a, b = t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()
        assert all(b <= lo or a >= hi for lo, hi in given_back)
    torch.cuda.synchronize()
    _all(r, ref)


@pytest.mark.parametrize("dtype", TYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("T", [1, 30, 130])
@pytest.mark.parametrize("alone", [True, False])
def test_a_bad_label_reaches_every_gradient(dtype, T, alone):
    """NaN in dw and in dx of the bad token and of every valid one; ignored tokens stay 0.
    With one call, and with the gradients alone."""
    V, H = 300, 72
    x, w, y = _inputs(T, V, H, dtype, seed=22)
    y[1::3] = -100
    if alone:
        y[:] = -100
    y[0] = V
    h = _head(T, V, H, dtype)
    r = h.loss_grad(x, w, y)
    apart = h.grad(x, w, y, r.lse, dx=torch.zeros_like(r.dx), dw=torch.zeros_like(r.dw))
    for dx, dw in ((r.dx, r.dw), apart):
        assert dw.isnan().all() and dx[y >= 0].isnan().all() and (dx[y < 0] == 0).all()
    assert r.lse[0].isnan() and r.token_loss[0].isnan() and r.loss.isnan()


@pytest.mark.parametrize("dtype", TYPES, ids=["f16", "bf16"])
@pytest.mark.parametrize("label", [5, 128255])
def test_confident_tokens_in_every_piece(dtype, label):
    """Two pieces of the vocabulary, every token nearly certain of a label in the first or the
    last: the label's element of g, alone in column 0 of dx (w is 0 there but for the label's
    row, x is 0), keeps its digits.

    dx[t, 0] = c (e^-loss - 1), c a power of two.  With o the others' sum over the label's
    exponential, loss = log(1 + o) is off by as much, relatively, as o: the two logits' errors
    dl, 300 e for the exponentials (at most 4e + 2e |l - m| + e/8 |l| < 100 e at |l| < 40) and
    their sums (34 additions, then 33 joins of at most 4 roundings); g is rounded once (u).  The
    gradient alone takes its lse in fp32: 8 |lse| 2^-24 of the element, absolutely, on top."""
    T, V, H = 4352, 128256, 64
    g = torch.Generator(device="cuda").manual_seed(23)
    w = torch.randn(V, H, generator=g, device="cuda") * H ** -0.5
    w[:, 0] = 0.0
    w[label] /= w[label].norm()
    x = w[label] * (torch.rand(T, 1, generator=g, device="cuda") * 12.0 + 20.0)
    w[label, 0] = 1.0
    x, w = x.to(dtype), w.to(dtype)
    y = torch.full((T,), label, device="cuda")
    l = x.double() @ w.double().t()
    assert float(l.abs().max()) < 40
    dl = 2 * H * E * float((x.double().abs() @ w.double().abs().t()).max())
    lse = torch.logsumexp(l, 1)
    loss = lse - l[:, label]
    del l
    assert loss.min() < 3e-5 and loss.max() < 1.0
    c = 1024.0
    want = c * torch.expm1(-loss)
    u = torch.finfo(dtype).eps / 2
    bound = 1.01 * (u + dl + 300 * E) * want.abs()
    h = _head(T, V, H, dtype)
    r = h.loss_grad(x, w, y, mean=False, loss_scale=c)
    check(r.dx[:, 0], want, bound, "label's element")
    dx, _ = h.grad(x, w, y, r.lse.clone(), mean=False, loss_scale=c)
    check(dx[:, 0], want, bound + c * 4 * E * lse.abs(), "label's element, lse alone")
    torch.cuda.empty_cache()


def test_last_token_of_a_long_sequence():
    """x [1, H] out of a sequence of hidden states, whose stride is far past a row's."""
    S, V, H, dtype = 1100, 500, 1024, torch.bfloat16
    x, w, y = _inputs(S, V, H, dtype, seed=24)
    last = x.reshape(1, S, H)[:, -1]
    assert last.stride(0) > 1 << 20
    _all(_head(1, V, H, dtype).loss_grad(last, w, y[-1:]), reference(last, w, y[-1:]))
