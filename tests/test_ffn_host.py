"""Argument checks of the feed-forward block (zero_ffn_*) on the CPU: every refusal happens before
anything touches the GPU; and the 64-bit reference against differences."""
import pytest

from zero_sharded_optimizer_rank_amd import abi

X, WG, WU, WD, Y, DY, DX = (0x1000000 * i for i in range(1, 8))  # never dereferenced
DG, DU, DD, ACT, SLOPE, LOW, MID, WS = (0x1000000 * i for i in range(8, 16))
T, H, F = 100, 64, 96


def _ffn(**kw):
    f = dict(tokens=T, hidden=H, inner=F, x=X, ldx=H, w_gate=WG, ld_gate=H, w_up=WU, ld_up=H,
             w_down=WD, ld_down=F, dtype=abi.ZERO_BF16, act=abi.ZERO_ACT_SILU)
    f.update(kw)
    return abi.zero_ffn_t(**f)


def _saved(**kw):
    s = dict(act=ACT, slope=SLOPE, low=LOW, h=MID, ld=F)
    s.update(kw)
    return abi.zero_ffn_saved_t(**s)


def _grads(**kw):
    g = dict(dy=DY, lddy=H, dx=DX, lddx=H, dw_gate=DG, lddw_gate=H, dw_up=DU, lddw_up=H,
             dw_down=DD, lddw_down=F, dw_dtype=abi.ZERO_BF16, accumulate=0)
    g.update(kw)
    return abi.zero_ffn_grads_t(**g)


BIG = 1 << 40


def _forward(f=None, y=Y, ldy=H, saved=None, ws=WS, n=BIG):
    abi.zero_ffn_forward(f or _ffn(), y, ldy, saved, ws, n)


def _backward(f=None, saved=None, g=None, ws=WS, n=BIG):
    abi.zero_ffn_backward(f or _ffn(), saved or _saved(), g or _grads(), ws, n)


@pytest.mark.parametrize("call,code", [
    (lambda: _forward(_ffn(tokens=-1)), abi.ZERO_EINVAL),
    (lambda: _forward(_ffn(tokens=(1 << 20) + 1)), abi.ZERO_EINVAL),
    (lambda: _forward(_ffn(hidden=0)), abi.ZERO_EINVAL),
    (lambda: _forward(_ffn(inner=0)), abi.ZERO_EINVAL),
    (lambda: _forward(_ffn(inner=(1 << 20) + 1, ld_down=1 << 21)), abi.ZERO_EINVAL),
    (lambda: _forward(_ffn(hidden=1 << 20, inner=1 << 20, ldx=1 << 20, ld_gate=1 << 20,
                           ld_up=1 << 20, ld_down=1 << 20)), abi.ZERO_EINVAL),
    (lambda: _forward(_ffn(ldx=H - 1)), abi.ZERO_EINVAL),
    (lambda: _forward(_ffn(ld_gate=H - 1)), abi.ZERO_EINVAL),
    (lambda: _forward(_ffn(ld_up=H - 1)), abi.ZERO_EINVAL),
    (lambda: _forward(_ffn(ld_down=F - 1)), abi.ZERO_EINVAL),
    (lambda: _forward(_ffn(ld_down=(1 << 20) + 1)), abi.ZERO_EINVAL),
    (lambda: _forward(_ffn(dtype=abi.ZERO_F32)), abi.ZERO_EINVAL),
    (lambda: _forward(_ffn(act=4)), abi.ZERO_EINVAL),
    (lambda: _forward(_ffn(act=-1)), abi.ZERO_EINVAL),
    (lambda: _forward(_ffn(x=None)), abi.ZERO_EINVAL),
    (lambda: _forward(_ffn(w_down=None)), abi.ZERO_EINVAL),
    (lambda: _forward(_ffn(x=X + 1)), abi.ZERO_EALIGN),
    (lambda: _forward(_ffn(w_up=WU + 1)), abi.ZERO_EALIGN),
    (lambda: _forward(y=None), abi.ZERO_EINVAL),
    (lambda: _forward(y=Y + 1), abi.ZERO_EALIGN),
    (lambda: _forward(ldy=H - 1), abi.ZERO_EINVAL),
    (lambda: _forward(y=X + 2), abi.ZERO_EINVAL),
    (lambda: _forward(y=WD + 2), abi.ZERO_EINVAL),
    (lambda: _forward(y=WS), abi.ZERO_EINVAL),
    (lambda: _forward(ws=None), abi.ZERO_EINVAL),
    (lambda: _forward(ws=WS + 128), abi.ZERO_EALIGN),
    (lambda: _forward(n=16), abi.ZERO_ENOSPC),
    (lambda: _forward(saved=_saved(ld=F + 4)), abi.ZERO_EINVAL),
    (lambda: _forward(saved=_saved(ld=F - 8)), abi.ZERO_EINVAL),
    (lambda: _forward(_ffn(inner=F - 3), saved=_saved(ld=F - 3)), abi.ZERO_EINVAL),
    (lambda: _forward(saved=_saved(act=None)), abi.ZERO_EINVAL),
    (lambda: _forward(saved=_saved(slope=SLOPE + 8)), abi.ZERO_EALIGN),
    (lambda: _forward(saved=_saved(low=None)), abi.ZERO_EINVAL),
    (lambda: _forward(saved=_saved(low=LOW + 8)), abi.ZERO_EALIGN),
    (lambda: _forward(saved=_saved(h=ACT + 16)), abi.ZERO_EINVAL),
    (lambda: _forward(saved=_saved(h=WG)), abi.ZERO_EINVAL),
    (lambda: _backward(_ffn(x=None)), abi.ZERO_EINVAL),
    (lambda: _backward(saved=_saved(act=None)), abi.ZERO_EINVAL),
    (lambda: _backward(g=_grads(dy=None)), abi.ZERO_EINVAL),
    (lambda: _backward(g=_grads(dy=DY + 1)), abi.ZERO_EALIGN),
    (lambda: _backward(g=_grads(lddy=H - 1)), abi.ZERO_EINVAL),
    (lambda: _backward(g=_grads(lddx=H - 1)), abi.ZERO_EINVAL),
    (lambda: _backward(g=_grads(lddw_gate=H - 1)), abi.ZERO_EINVAL),
    (lambda: _backward(g=_grads(lddw_down=F - 1)), abi.ZERO_EINVAL),
    (lambda: _backward(g=_grads(dw_dtype=abi.ZERO_F16)), abi.ZERO_EINVAL),
    (lambda: _backward(g=_grads(dw_dtype=abi.ZERO_F32, dw_up=DU + 2)), abi.ZERO_EALIGN),
    (lambda: _backward(g=_grads(dw_up=DG + 2)), abi.ZERO_EINVAL),
    (lambda: _backward(g=_grads(dx=DY)), abi.ZERO_EINVAL),
    (lambda: _backward(g=_grads(dw_down=LOW)), abi.ZERO_EINVAL),
    (lambda: _backward(g=_grads(dx=WS + 64)), abi.ZERO_EINVAL),
    (lambda: _backward(ws=None), abi.ZERO_EINVAL),
    (lambda: _backward(n=16), abi.ZERO_ENOSPC),
])
def test_refusals(call, code):
    with pytest.raises(abi.ZeroError) as e:
        call()
    assert e.value.code == code
    assert abi.zero_last_error()


def test_null_structures():
    lib = abi.lib()
    assert lib.zero_ffn_forward(None, Y, H, None, WS, BIG, None) == abi.ZERO_EINVAL
    assert lib.zero_ffn_backward(None, None, None, WS, BIG, None) == abi.ZERO_EINVAL
    assert lib.zero_ffn_workspace_bytes(None, None) == 0


def test_workspace_bytes():
    def ws(g=None, **kw):
        return abi.zero_ffn_workspace_bytes(_ffn(**kw), g)
    assert ws(tokens=-1) == 0 and ws(g=_grads(lddy=1)) == 0
    assert ws(tokens=0) > 0
    # what holds for so many tokens holds for every batch of fewer
    for kw in (dict(), dict(hidden=1600, inner=6400, ldx=1600, ld_gate=1600, ld_up=1600,
                            ld_down=6400), dict(x=X + 2), dict(inner=F - 3, ld_down=F)):
        h = kw.get("hidden", H)
        for g in (None, _grads(lddy=h)):
            most = ws(g, tokens=3000, **kw)
            for t in list(range(0, 700, 7)) + [63, 64, 65, 255, 256, 257, 1024, 2999]:
                assert ws(g, tokens=t, **kw) <= most
    # rows that start between 16-byte boundaries are laid out again
    assert ws(x=X + 2) > ws() and ws(ld_down=F + 1) > ws()
    assert ws(tokens=20, x=X + 2) == ws(tokens=20)


def test_classes_refuse_on_the_host():
    torch = pytest.importorskip("torch")
    from zero_sharded_optimizer_rank_amd.ffn import GatedFFN
    with pytest.raises(TypeError, match="float16"):
        GatedFFN(4, 8, 8, torch.float32)
    with pytest.raises(ValueError, match="activation"):
        GatedFFN(4, 8, 8, torch.float16, act="swish")
    with pytest.raises(ValueError, match="not a GPU"):
        GatedFFN(4, 8, 8, torch.float16, device="cpu")
    with pytest.raises(ValueError, match="out of range"):
        GatedFFN(4, 8, 0, torch.float16, device="cuda:0")


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh", "relu"])
def test_reference_against_differences(name):
    """Central differences in 64 bits of sum(y * dy), h = 1e-5: off by h^2 / 6 times a third
    derivative of a few units and 2^-53 / h: under 1e-8 relative to the largest."""
    torch = pytest.importorskip("torch")
    import ffn_util as fu
    g = torch.Generator().manual_seed(0)
    t, h, f = 3, 4, 5
    m = [torch.randn(*s, generator=g, dtype=torch.float64)
         for s in ((t, h), (f, h), (f, h), (h, f), (t, h))]

    def loss(x, wg, wu, wd, dy):
        return float(((fu.act(name, x @ wg.t())[0] * (x @ wu.t())) @ wd.t() * dy).sum())
    r = fu.reference(*m[:4], name, m[4])
    for k, out in enumerate(("dx", "dw_gate", "dw_up", "dw_down")):
        for i in range(m[k].numel()):
            d = []
            for s in (1e-5, -1e-5):
                moved = [a.clone() for a in m]
                moved[k].view(-1)[i] += s
                d.append(loss(*moved))
            got = (d[0] - d[1]) / 2e-5
            assert abs(got - float(r[out][0].reshape(-1)[i])) < 1e-7 * (1 + abs(got))
