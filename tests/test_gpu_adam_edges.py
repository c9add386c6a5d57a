"""AdamW over tensor lists at the ends of fp32's range: the largest second moments, and NaNs of
every sign and payload; with bounds from adam_util.update64."""
import numpy as np
import pytest

import adam_util as au

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _list(grad, master, bits):
    from zero_sharded_optimizer_rank_amd.adam import AdamList, AdamState
    return AdamList([grad], [master], AdamState([grad.numel()], bits=bits))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [0.0, 1e-8])
def test_first_step_is_lr_up_to_the_largest_moments(bits, eps):
    """g up to 2^63, so that v = g^2 / 2 goes up to 2^125: the first step moves every element by
    lr.  The roundings of the step are update64's 14 E < 2^-20 of it, half a step of beta's 1/2 none
    (a power of two); from g = 2 on, eps = 1e-8 is under 2^-26 of the root."""
    n = 500
    g = torch.from_numpy(np.exp2(np.linspace(1, 63, n)).astype(np.float32)).cuda()
    g[::3] *= -1
    w = torch.zeros_like(g)
    _list(g, w, bits).step(lr=2.0 ** -10, eps=eps, step=1, beta2=0.5)
    want = -torch.sign(g).double() * 2.0 ** -10
    assert ((w.double() - want).abs() <= 2.0 ** -10 * (2.0 ** -20 + 2.0 ** -26)).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_large_gradients_within_the_roundings(bits, gt):
    """Random gradients around 2^30 .. 2^62, a block of 128 of each magnitude, second step too."""
    rng = np.random.default_rng(0)
    mags = np.exp2(np.repeat(np.arange(30, 63, 2), au.BLOCK))
    x = torch.from_numpy((rng.standard_normal(mags.size) * 0.5 * mags).astype(np.float32)).to(gt)
    p = (rng.standard_normal(mags.size) * 0.02).astype(np.float32)
    w = torch.from_numpy(p).cuda()
    lst = _list(x.cuda(), w, bits)
    m, v = (np.zeros(mags.size, dtype=np.float32) for _ in range(2))
    for step in (1, 2):
        s = au.scalars(1e-3, 0.9, 0.999, 1e-8, step, 1.0, 0.0, 1.0, 1.0)
        want, far = au.update64(x.float().numpy(), p, m, v, s, bits)
        lst.step(lr=1e-3, step=step)
        p = w.cpu().numpy()
        assert (np.abs(p.astype(np.float64) - want[0]) <= far[0]).all()
        m, v = (t[:mags.size].float().cpu().numpy() for t in lst.moments())
