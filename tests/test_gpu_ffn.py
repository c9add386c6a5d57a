"""The gated feed-forward block (zero_ffn_*) on the GPU against 64-bit values, every element within
the bounds that ffn_util derives from the roundings."""
import pytest

import ffn_util as fu

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]
ACTS = ["silu", "gelu", "gelu_tanh", "relu"]
NAMES = ("dw_gate", "dw_up", "dw_down")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _ffn(*a, **k):
    from zero_sharded_optimizer_rank_amd.ffn import GatedFFN
    return GatedFFN(*a, **k)


def _inputs(T, H, F, dt, seed=0, scale=1.0, dy=0.05):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(r, c, s):
        return (torch.randn(r, c, generator=g, device="cuda") * s).to(dt)
    return (normal(T, H, scale), normal(F, H, H ** -0.5), normal(F, H, H ** -0.5),
            normal(H, F, F ** -0.5), normal(T, H, dy))


def _guarded(rows, cols, dtype, extra=0):
    """A matrix whose rows lie `extra` apart more, between guard values."""
    buf = torch.full((rows + 2, cols + extra), 3.0, dtype=dtype, device="cuda")
    return buf, buf[1:1 + rows, :cols]


def _guards_intact(buf, rows, cols):
    assert (buf[0] == 3).all() and (buf[1 + rows] == 3).all() and (buf[:, cols:] == 3).all()


def _dirty(f):
    """What lies in the workspace before a call does not matter: NaN patterns."""
    f.ws.fill_(0xFF)


def _run(T, H, F, dt, act, seed=0, tokens=None, views=None, dw_type=None, extra=0, scale=1.0):
    x, wg, wu, wd, dy = _inputs(T, H, F, dt, seed, scale)
    if views:
        x, wg, wu, wd, dy = (views(t) for t in (x, wg, wu, wd, dy))
    ref = fu.reference(x, wg, wu, wd, act, dy)
    f = _ffn(tokens or T, H, F, dt, act=act)
    u = ref["u"]
    saved = f.new_saved(T)
    for t in saved:
        t.fill_(float("nan"))
    yb, y = _guarded(T, H, dt, extra)
    _dirty(f)
    r = f.forward(x, wg, wu, wd, y=y, save=saved)
    fu.check(r.y, *ref["y"], "y")
    _guards_intact(yb, T, H)
    if T * H >= 1000:
        fu.check_norm(r.y, ref["y"][0], 2.5 * u, "y")
    alone = f.forward(x, wg, wu, wd).y
    assert torch.equal(alone, y)  # the same bits without keeping
    bufs = {"dx": _guarded(T, H, dt, extra), "dw_gate": _guarded(F, H, dw_type or dt, extra),
            "dw_up": _guarded(F, H, dw_type or dt, extra),
            "dw_down": _guarded(H, F, dw_type or dt, extra)}
    _dirty(f)
    d = f.backward(dy, x, wg, wu, wd, saved, **{k: b[1] for k, b in bufs.items()})
    fu.check(d.dx, *ref["dx"], "dx")
    for name in NAMES:
        fu.check_dw(getattr(d, name), ref, name)
    for k, (b, m) in bufs.items():
        _guards_intact(b, *m.shape)
    if T * H >= 1000:
        fu.check_norm(d.dx, ref["dx"][0], 6 * u, "dx")
        for name in NAMES:
            fu.check_norm(getattr(d, name), ref[name][0], 6 * u, name)
    return f, (x, wg, wu, wd, dy), ref, r, d


SHAPES = [(1, 1, 1), (1, 8, 8), (2, 7, 3), (5, 16, 40), (16, 64, 64), (17, 72, 200),
          (33, 131, 77), (48, 264, 264), (63, 136, 1000), (64, 512, 130), (65, 64, 64),
          (100, 131, 77), (130, 8, 500), (255, 256, 256), (256, 256, 256), (257, 264, 520),
          (300, 1000, 136), (513, 72, 129), (70, 300, 5000), (1, 1600, 640), (64, 1601, 70),
          # few tiles of long contractions: every product in parts
          (200, 4000, 40), (2000, 24, 40), (5000, 8, 8), (130, 2051, 9), (1030, 515, 260)]


@pytest.mark.parametrize("dt", TYPES, ids=["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_sizes(shape, dt):
    _run(*shape, dt, "silu", seed=1)


@pytest.mark.parametrize("dt", TYPES, ids=["bf16", "f16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [9, 96])
def test_activations(act, dt, T):
    _run(T, 136, 328, dt, act, seed=2, scale=3.0)  # g of several units: the tails too


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 64, 65, 128, 129])
def test_tokens(T):
    """Every form for few tokens, on a block made for more; the last rows stay."""
    f, (x, wg, wu, wd, dy), ref, r, d = _run(T, 256, 384, torch.bfloat16, "silu", seed=3,
                                             tokens=200)
    f._y.fill_(3.0)
    f._dx.fill_(3.0)
    y = f.forward(x, wg, wu, wd, save=True)
    g = f.backward(dy, x, wg, wu, wd, y.saved)
    assert torch.equal(y.y, r.y) and torch.equal(g.dx, d.dx)
    assert (f._y[T:] == 3).all() and (f._dx[T:] == 3).all()


@pytest.mark.parametrize("dt", TYPES, ids=["bf16", "f16"])
@pytest.mark.parametrize("T,H,F", [(1, 24, 4000), (4, 40, 1001), (7, 16, 2048), (8, 2056, 8200),
                                   (9, 24, 2000), (13, 67, 515), (16, 40, 8200)])
def test_few_tokens_round_once(T, H, F, dt):
    """Up to 16 tokens h's own rounding does not reach y."""
    x, wg, wu, wd, _ = _inputs(T, H, F, dt, seed=24)
    h, want, bound = fu.few_bound(x, wg, wu, wd, "gelu")
    f = _ffn(T, H, F, dt, act="gelu")
    saved = f.new_saved()
    for t in saved:
        t.fill_(float("nan"))
    _dirty(f)
    r = f.forward(x, wg, wu, wd, save=saved)
    fu.check(r.y, want, bound, "y")
    # |round(y + d) - y| <= |round(y) - y| + 2 |d|: d are fp32 sums' errors, which add up as a
    # random walk does, to a relative (sqrt F + sqrt H + 16) E at twice their size
    limit = (want.to(dt).double() - want).norm() / want.norm()
    limit = float(limit) + 2 * 2 * (F ** 0.5 + H ** 0.5 + 16) * fu.E
    fu.check_norm(r.y, want, limit, "y")
    if dt == torch.bfloat16 and T * H >= 200:  # it tells: h rounded once more is outside
        once = (h.to(dt).double() @ wd.double().t()).to(dt).double()
        assert float((once - want).norm() / want.norm()) > limit


@pytest.mark.parametrize("T", [5, 12])
def test_few_tokens_past_16_bits(T):
    """Where h passes fp16's range y is what infinities give, as for more tokens."""
    H, F, dt = 64, 64, torch.float16
    x, wg, wu = (torch.zeros(r, H, dtype=dt, device="cuda") for r in (T, F, F))
    x[:, 0] = 300.0
    wg[3, 0] = wu[3, 0] = 1.0  # h = 90000 in one column
    wd = torch.eye(H, F, device="cuda").to(dt)
    y = _ffn(T, H, F, dt, act="relu").forward(x, wg, wu, wd).y
    many = _ffn(40, H, F, dt, act="relu").forward(x.repeat(40, 1)[:40], wg, wu, wd).y
    assert torch.isinf(y[:, 3]).all()
    assert torch.equal(torch.isnan(y), torch.isnan(many[:T]))
    assert torch.equal(y.nan_to_num(nan=7.0), many[:T].nan_to_num(nan=7.0))


def _strided(t):
    b = torch.full((t.shape[0], t.shape[1] + 24), float("nan"), dtype=t.dtype, device=t.device)
    b[:, 8:8 + t.shape[1]] = t
    return b[:, 8:8 + t.shape[1]]


def _odd(t):
    b = torch.full((t.shape[0], t.shape[1] + 5), float("nan"), dtype=t.dtype, device=t.device)
    b[:, 3:3 + t.shape[1]] = t
    return b[:, 3:3 + t.shape[1]]


@pytest.mark.parametrize("views", [_strided, _odd], ids=["aligned", "odd"])
@pytest.mark.parametrize("T,H,F", [(20, 64, 72), (20, 67, 75), (150, 64, 72), (150, 67, 75)])
@pytest.mark.parametrize("extra", [0, 3, 16])
def test_strides(views, T, H, F, extra):
    _run(T, H, F, torch.float16, "gelu", seed=4, views=views, extra=extra)


@pytest.mark.parametrize("dt", TYPES, ids=["bf16", "f16"])
@pytest.mark.parametrize("wide", [False, True], ids=["16", "f32"])
@pytest.mark.parametrize("T,H,F", [(40, 72, 136), (300, 136, 72), (0, 40, 24), (90, 67, 45)])
def test_accumulated(T, H, F, wide, dt):
    x, wg, wu, wd, dy = _inputs(T, H, F, dt, seed=5)
    ref = fu.reference(x, wg, wu, wd, "silu", dy)
    f = _ffn(max(T, 1), H, F, dt)
    wt = torch.float32 if wide else dt
    base = {k: torch.randn(*((H, F) if k == "dw_down" else (F, H)), device="cuda").to(wt)
            for k in NAMES}
    dw = {k: b.clone() for k, b in base.items()}
    saved = f.forward(x, wg, wu, wd, save=True).saved
    d = f.backward(dy, x, wg, wu, wd, saved, accumulate=True, **dw)
    for k in NAMES:
        if T == 0:
            assert torch.equal(dw[k], base[k])
        else:
            fu.check_dw(dw[k], ref, k, base[k])
    fu.check(d.dx, *ref["dx"], "dx")
    d = f.backward(dy, x, wg, wu, wd, saved, **dw)  # overwritten
    for k in NAMES:
        fu.check_dw(dw[k], ref, k)
        if T == 0:
            assert (dw[k] == 0).all()


def test_wide_gradients_of_a_16_bit_block():
    _run(200, 264, 136, torch.bfloat16, "silu", seed=6, dw_type=torch.float32)


def test_what_is_not_wanted_is_not_written():
    from zero_sharded_optimizer_rank_amd import abi
    T, H, F, dt = 130, 72, 136, torch.bfloat16
    x, wg, wu, wd, dy = _inputs(T, H, F, dt, seed=7)
    f = _ffn(T, H, F, dt)
    saved = f.forward(x, wg, wu, wd, save=True).saved
    full = f.backward(dy, x, wg, wu, wd, saved)
    full = type(full)(*(t.clone() for t in full))
    only = f.backward(dy, x, wg, wu, wd, saved, need_dw=False)
    assert torch.equal(only.dx, full.dx) and only.dw_gate is None
    f._dx.fill_(3.0)
    only = f.backward(dy, x, wg, wu, wd, saved, need_dx=False)
    assert only.dx is None and (f._dx == 3).all()
    for k in NAMES:
        assert torch.equal(getattr(only, k), getattr(full, k))
    for k in NAMES:  # one weight alone, through the C ABI
        out = torch.full_like(getattr(full, k), 3.0)
        g = f._grads_t(dy.data_ptr(), H)
        setattr(g, k, out.data_ptr())
        ffn = f._ffn(x, wg, wu, wd)
        abi.zero_ffn_backward(ffn, f._saved_t(saved, T), g, f.ws, f.ws.numel(),
                              torch.cuda.current_stream())
        assert torch.equal(out, getattr(full, k))


@pytest.mark.parametrize("T", [40, 300])
def test_a_token_of_nan_stays_alone(T):
    H, F, dt = 264, 520, torch.bfloat16
    x, wg, wu, wd, dy = _inputs(T, H, F, dt, seed=8)
    f = _ffn(T, H, F, dt)
    r = f.forward(x, wg, wu, wd, save=True)
    y, dx = r.y.clone(), f.backward(dy, x, wg, wu, wd, r.saved).dx.clone()
    keep = torch.arange(T, device="cuda") != 17
    for value in (float("nan"), float("inf")):
        bad = x.clone()
        bad[17, 5] = value
        r = f.forward(bad, wg, wu, wd, save=True)
        d = f.backward(dy, bad, wg, wu, wd, r.saved)
        assert torch.equal(r.y[keep], y[keep]) and torch.equal(d.dx[keep], dx[keep])
        assert torch.isnan(r.y[17]).any()
        for k in NAMES:
            assert torch.isnan(getattr(d, k)).any()
    bad = dy.clone()
    bad[17, 5] = float("nan")
    r = f.forward(x, wg, wu, wd, save=True)
    d = f.backward(bad, x, wg, wu, wd, r.saved)
    assert torch.equal(d.dx[keep], dx[keep]) and torch.isnan(d.dx[17]).all()


def test_equal_calls_give_equal_bits():
    """Another address, another stream, a workspace that another call has used."""
    T, H, F, dt = 200, 520, 1000, torch.float16
    x, wg, wu, wd, dy = _inputs(T, H, F, dt, seed=9)
    f = _ffn(512, H, F, dt, act="gelu_tanh")
    r = f.forward(x, wg, wu, wd, save=True)
    d = f.backward(dy, x, wg, wu, wd, r.saved)
    want = [t.clone() for t in (r.y, *d)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = _inputs(512, H, F, dt, seed=10)
    f.forward(*other[:4])
    side.wait_stream(torch.cuda.current_stream())
    x2, wg2, wu2, wd2, dy2 = (_strided(t) for t in (x, wg, wu, wd, dy))
    side.wait_stream(torch.cuda.current_stream())
    r = f.forward(x2, wg2, wu2, wd2, save=True, stream=side)
    d = f.backward(dy2, x2, wg2, wu2, wd2, r.saved, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, (r.y, *d)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [20, 200])
def test_captured_and_replayed(T):
    H, F, dt = 264, 520, torch.bfloat16
    x, wg, wu, wd, dy = _inputs(T, H, F, dt, seed=11)
    f = _ffn(T, H, F, dt)
    f.backward(dy, x, wg, wu, wd, f.forward(x, wg, wu, wd, save=True).saved)  # its buffers
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        r = f.forward(x, wg, wu, wd, save=True)
        d = f.backward(dy, x, wg, wu, wd, r.saved)
    for i in range(3):
        new = _inputs(T, H, F, dt, seed=20 + i)
        for a, b in zip((x, wg, wu, wd, dy), new):
            a.copy_(b)
        torch.cuda.synchronize()
        graph.replay()
        got = [t.clone() for t in (r.y, *d)]
        e = f.forward(x, wg, wu, wd, save=True)  # eager work between the replays
        g = f.backward(dy, x, wg, wu, wd, e.saved)
        for a, b in zip(got, (e.y, *g)):
            assert torch.equal(a, b)


def test_two_layers_keep_their_own():
    T, H, F, dt = 80, 72, 136, torch.bfloat16
    f = _ffn(T, H, F, dt)
    layers = []
    for s in (12, 13):
        x, wg, wu, wd, dy = _inputs(T, H, F, dt, seed=s)
        layers.append((x, wg, wu, wd, dy, f.forward(x, wg, wu, wd, save=f.new_saved()).saved))
    for x, wg, wu, wd, dy, saved in reversed(layers):
        ref = fu.reference(x, wg, wu, wd, "silu", dy)
        d = f.backward(dy, x, wg, wu, wd, saved)
        fu.check(d.dx, *ref["dx"], "dx")
        for k in NAMES:
            fu.check_dw(getattr(d, k), ref, k)


def test_workspace_grows_once_for_odd_rows():
    T, H, F, dt = 150, 64, 72, torch.float16
    x, wg, wu, wd, dy = _inputs(T, H, F, dt, seed=14)
    f = _ffn(T, H, F, dt)
    first = f.ws
    saved = f.forward(x, wg, wu, wd, save=True).saved
    assert f.ws is first
    want = [t.clone() for t in f.backward(dy, x, wg, wu, wd, saved)]
    o = [_odd(t) for t in (x, wg, wu, wd, dy)]
    saved = f.forward(*o[:4], save=True).saved
    got = f.backward(o[4], *o[:4], saved)
    grown = f.ws
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    f.backward(o[4], *o[:4], f.forward(*o[:4], save=True).saved)
    assert f.ws is grown and first in f._old_ws


@pytest.mark.parametrize("T", [3, 70])
def test_offsets_past_32_bits(T):
    """Weights of 2^32 elements and more; every output against sums in strips."""
    H, F, dt = 65536 + 64, 65536 + 8, torch.bfloat16
    if torch.cuda.mem_get_info()[0] < 9 * 2 * H * F:
        pytest.skip("not enough memory")
    g = torch.Generator(device="cuda").manual_seed(15)

    def normal(r, c, s):
        t = torch.empty(r, c, dtype=dt, device="cuda")
        return t.normal_(0.0, s, generator=g)
    x, dy = normal(T, H, 1.0), normal(T, H, 0.05)
    wg, wu, wd = normal(F, H, H ** -0.5), normal(F, H, H ** -0.5), normal(H, F, F ** -0.5)
    f = _ffn(T, H, F, dt)
    r = f.forward(x, wg, wu, wd, save=True)
    # the bounds hold for parts too: all tokens, strips of the inner axis
    X, Y = x.double(), dy.double()
    y, dx = (torch.zeros(T, H, dtype=torch.float64, device="cuda") for _ in range(2))
    strips = []
    for f0 in range(0, F, 8192):
        s = slice(f0, min(F, f0 + 8192))
        G, U, D = wg[s].double(), wu[s].double(), wd[:, s].double()
        gg, uu = X @ G.t(), X @ U.t()
        a, slope = fu.act("silu", gg)
        dh = Y @ D
        y += (a * uu) @ D.t()
        dg, du = dh * uu * slope, dh * a
        dx += dg @ G + du @ U
        if f0 in (0, 57344, 65536):
            strips.append((s, dg, du, a * uu))
        del G, U, D
    u = torch.finfo(dt).eps / 2
    fu.check_norm(r.y, y, 2.5 * u, "y")
    d = f.backward(dy, x, wg, wu, wd, r.saved)
    fu.check_norm(d.dx, dx, 6 * u, "dx")
    for s, dg, du, h in strips:
        fu.check_norm(d.dw_gate[s], dg.t() @ X, 6 * u, "dw_gate")
        fu.check_norm(d.dw_up[s], du.t() @ X, 6 * u, "dw_up")
        fu.check_norm(d.dw_down[:, s], Y.t() @ h, 6 * u, "dw_down")
