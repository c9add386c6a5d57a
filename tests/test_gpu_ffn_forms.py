"""The gated feed-forward block's kernels by their forms (the shapes of ffn_shapes, which a host
test holds to them): 256 x 256 tiles in every launch, with and without parts, and every kernel for
up to 64 tokens; every element within ffn_util's bounds.

2-norms: each output takes two roundings to 16 bits on its way (h, dg or du, and its own), each at
most u of a value and, spread evenly over a step, u / sqrt(3) of it in the mean square; sums of
mean zero keep that ratio.  sqrt(2 / 3) u = 0.82 u; what is kept in 24 bits (2^-16, 2^-5 u at most)
and fp32 sums add under 0.1 u: 1 u."""
import pytest

import ffn_util as fu
import test_gpu_ffn as tg
from ffn_shapes import FEW, LARGE

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

NAMES = ("dw_gate", "dw_up", "dw_down")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _id(shape):
    return "x".join(map(str, shape))


def _norms(y, d, ref):
    for name, got in (("y", y), ("dx", d.dx), *((k, getattr(d, k)) for k in NAMES)):
        fu.check_norm(got, ref[name][0], ref["u"], name)


# all types and activations on the first, two of them on the others
CASES = [(s, dt, act) for s in LARGE for dt in tg.TYPES for act in tg.ACTS
         if s == next(iter(LARGE)) or (dt, act) in ((torch.bfloat16, "silu"),
                                                    (torch.float16, "gelu_tanh"))]


@pytest.mark.parametrize("shape,dt,act", CASES,
                         ids=[f"{_id(s)}-{str(d)[6:]}-{a}" for s, d, a in CASES])
def test_large_tiles(shape, dt, act):
    """Kept and not, outputs between guards, a workspace of NaNs."""
    f, inputs, ref, r, d = tg._run(*shape, dt, act, seed=31, extra=8)
    _norms(r.y, d, ref)


@pytest.mark.parametrize("wide", [False, True], ids=["16", "f32"])
@pytest.mark.parametrize("dt", tg.TYPES, ids=["bf16", "f16"])
@pytest.mark.parametrize("shape", list(LARGE), ids=_id)
def test_large_tiles_accumulate(shape, dt, wide):
    T, H, F = shape
    x, wg, wu, wd, dy = tg._inputs(T, H, F, dt, seed=32)
    ref = fu.reference(x, wg, wu, wd, "silu", dy)
    f = tg._ffn(T, H, F, dt)
    gen = torch.Generator(device="cuda").manual_seed(33)
    saved = f.forward(x, wg, wu, wd, save=True).saved
    dw, base = {}, {}
    for k in NAMES:
        rows, cols = (H, F) if k == "dw_down" else (F, H)
        base[k] = torch.randn(rows, cols, generator=gen, device="cuda").to(
            torch.float32 if wide else dt)
        dw[k] = torch.full((rows, cols + 3), 3.0, dtype=base[k].dtype, device="cuda")
        dw[k][:, :cols] = base[k]
    views = {k: t[:, :t.shape[1] - 3] for k, t in dw.items()}
    d = f.backward(dy, x, wg, wu, wd, saved, accumulate=True, **views)
    for k in NAMES:
        fu.check_dw(getattr(d, k), ref, k, base[k])
    fu.check(d.dx, *ref["dx"], "dx")
    f.backward(dy, x, wg, wu, wd, saved, **views)  # overwritten
    for k in NAMES:
        fu.check_dw(views[k], ref, k)
        assert (dw[k][:, -3:] == 3).all()


@pytest.mark.parametrize("shape", list(FEW), ids=_id)
def test_few_tokens(shape):
    dt = tg.TYPES[shape[0] % 2]
    f, inputs, ref, r, d = tg._run(*shape, dt, "silu", seed=34)
    _norms(r.y, d, ref)


@pytest.mark.parametrize("T,H,F", [(20, 72, 136), (100, 264, 520), (1030, 4104, 4099)])
@pytest.mark.parametrize("dt,power", [(torch.bfloat16, -40), (torch.bfloat16, 40),
                                      (torch.float16, -8), (torch.float16, 8)],
                         ids=["bf16-down", "bf16-up", "f16-down", "f16-up"])
def test_gradients_carry_a_loss_scale(T, H, F, dt, power):
    """dy times a power of two gives the gradients times it, bit for bit, in bf16, whose range
    they stay in.  In fp16 some of dg and du lie below the normal range, more or fewer by the scale:
    there each pass is held to the 64-bit values (fp16's smallest step is in the bounds)."""
    x, wg, wu, wd, dy = tg._inputs(T, H, F, dt, seed=35)
    f = tg._ffn(T, H, F, dt)
    saved = f.forward(x, wg, wu, wd, save=True).saved
    if dt == torch.bfloat16:
        a = [t.clone() for t in f.backward(dy, x, wg, wu, wd, saved)]
        b = f.backward((dy.double() * 2.0 ** power).to(dt), x, wg, wu, wd, saved)
        for s, t in zip(a, b):
            assert torch.equal(s.double() * 2.0 ** power, t.double())
        return
    dy = (dy.double() * 2.0 ** power).to(dt)
    ref = fu.reference(x, wg, wu, wd, "silu", dy)
    d = f.backward(dy, x, wg, wu, wd, saved)
    fu.check(d.dx, *ref["dx"], "dx")
    for k in NAMES:
        fu.check_dw(getattr(d, k), ref, k)
