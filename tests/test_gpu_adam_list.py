"""AdamW over tensor lists (zero_tensors_adam) on the GPU: against the same fp32 operations on
the CPU, bit for bit, 8-bit moments and their random rounding included; against 64-bit values
within the bounds of adam_util.update64 (the roundings counted there; the parameters of 8-bit
moments go by it alone); and against the shard update (zero_adam_apply)."""
import math

import numpy as np
import pytest

import adam_util as au

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]
SIZES = [0, 1, 2, 3, 4, 5, 127, 128, 129, 1000, 4095, 4096, 4097, 0, 8192, 12345, 64]
GUARD = 7.0


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _mods():
    from zero_sharded_optimizer_rank_amd.adam import AdamList, AdamState
    return AdamList, AdamState


def _guarded(n, dtype, shift):
    buf = torch.full((n + 16,), GUARD, dtype=dtype, device="cuda")
    return buf, buf[shift:shift + n]


class Run:
    """A list on the GPU and the same state on the CPU."""

    def __init__(self, sizes, grad_types, out_types, bits, shift=0, seed=0, sigma=1e-3, warm=True,
                 weight_decay=0.0, lr_scale=1.0):
        AdamList, AdamState = _mods()
        rng = np.random.default_rng(seed)
        self.sizes, self.bits = sizes, bits
        self.state = AdamState(sizes, bits=bits, device="cuda")
        self.bufs, grads, masters, params = [], [], [], []
        self.g, self.p, self.m, self.v = [], [], [], []
        for i, n in enumerate(sizes):
            gt = grad_types[i % len(grad_types)]
            ot = out_types[i % len(out_types)] if out_types else None
            mag = 2.0 ** rng.integers(-3, 4)
            g = torch.from_numpy((rng.standard_normal(n) * sigma * mag).astype(np.float32)).to(gt)
            p = (rng.standard_normal(n) * 0.02).astype(np.float32)
            b, t = _guarded(n, gt, shift)
            t.copy_(g)
            grads.append(t)
            self.bufs.append((b, shift, n))
            b, t = _guarded(n, torch.float32, shift)
            t.copy_(torch.from_numpy(p))
            masters.append(t)
            self.bufs.append((b, shift, n))
            if ot is not None:
                b, t = _guarded(n, ot, shift)
                params.append(t)
                self.bufs.append((b, shift, n))
            self.g.append(g.float().numpy())
            self.p.append(p)
            m = (rng.standard_normal(n) * sigma * mag * 0.3).astype(np.float32)
            v = np.square(rng.standard_normal(n) * sigma * mag).astype(np.float32)
            if not warm:
                m, v = np.zeros_like(m), np.zeros_like(v)
            self._set(i, m, v)
        self.grads, self.masters, self.params = grads, masters, params
        self.wd = weight_decay if isinstance(weight_decay, list) else [weight_decay] * len(sizes)
        self.ls = lr_scale if isinstance(lr_scale, list) else [lr_scale] * len(sizes)
        self.list = AdamList(grads, masters, self.state, params=params if out_types else None,
                             weight_decay=weight_decay, lr_scale=lr_scale)

    def _set(self, i, m, v):
        """Moments of tensor i, on both sides (8 bits: cut off)."""
        n, at = self.sizes[i], self.state.offsets[i]
        if self.bits == 8:
            zero = np.zeros(n, dtype=np.uint32)
            mc, me = au.encode(m, zero, 16, 7)
            vc, ve = au.encode(v, zero, 32, 8)
            e = slice(at // au.BLOCK, at // au.BLOCK + me.size)
            for dst, src, where in ((self.state.m, mc, slice(at, at + n)), (self.state.m_exp, me, e),
                                    (self.state.v, vc, slice(at, at + n)), (self.state.v_exp, ve, e)):
                dst[where].copy_(torch.from_numpy(src))
            m, v = au.decode(mc, me, 16, 7), au.decode(vc, ve, 32, 8)
        else:
            self.state.m[at:at + n].copy_(torch.from_numpy(m))
            self.state.v[at:at + n].copy_(torch.from_numpy(v))
        self.m.append(m)
        self.v.append(v)

    def scalars(self, i, coef=1.0, **kw):
        return au.scalars(kw["lr"], kw.get("beta1", 0.9), kw.get("beta2", 0.999),
                          kw.get("eps", 1e-8), kw["step"], kw.get("loss_scale", 1.0), self.wd[i],
                          self.ls[i], coef)

    def expect(self, coef=1.0, **kw):
        """The CPU side takes the step; codes and exponents stay in self.codes."""
        seed = kw.get("seed", kw["step"])
        self.codes, self.near = [], []
        for i, n in enumerate(self.sizes):
            if self.bits == 8:
                want, far = au.update64(self.g[i], self.p[i], self.m[i], self.v[i],
                                        self.scalars(i, coef, **kw), bits=8)
                self.near.append((want[0], far[0]))
            self.p[i], m, v = au.update32(self.g[i], self.p[i], self.m[i], self.v[i],
                                          self.scalars(i, coef, **kw))
            if self.bits == 8:
                r = au.random_bits(seed, i, 0, n)
                mc, me = au.encode(m, r & np.uint32(0xFFFF), 16, 7)
                vc, ve = au.encode(v, r >> np.uint32(16), 32, 8)
                self.codes.append((mc, me, vc, ve))
                m, v = au.decode(mc, me, 16, 7), au.decode(vc, ve, 32, 8)
            self.m[i], self.v[i] = m, v

    def check(self):
        m, v = self.list.moments()
        for i, n in enumerate(self.sizes):
            at = self.state.offsets[i]
            if self.bits == 8:
                want, far = self.near[i]
                self.p[i] = self.masters[i].cpu().numpy()  # the next step goes on from here
                assert (np.abs(self.p[i].astype(np.float64) - want) <= far).all(), f"master {i}"
            assert _same(self.masters[i], self.p[i]), f"master {i}"
            assert _same(m[at:at + n].float(), self.m[i]), f"m {i}"
            assert _same(v[at:at + n].float(), self.v[i]), f"v {i}"
            if self.bits == 8:
                mc, me, vc, ve = self.codes[i]
                e = slice(at // au.BLOCK, at // au.BLOCK + me.size)
                for got, want in ((self.state.m[at:at + n], mc), (self.state.m_exp[e], me),
                                  (self.state.v[at:at + n], vc), (self.state.v_exp[e], ve)):
                    assert np.array_equal(got.cpu().numpy(), want), f"codes of {i}"
            if self.params:
                want = torch.from_numpy(self.p[i]).to(self.params[i].dtype)
                assert torch.equal(self.params[i].cpu(), want), f"parameter {i}"
        self.check_guards()

    def check_guards(self):
        for b, shift, n in self.bufs:
            b = b.cpu()
            assert (b[:shift] == GUARD).all() and (b[shift + n:] == GUARD).all()
        for flat in (self.state.m, self.state.v):  # between the tensors
            for at, n in zip(self.state.offsets, self.sizes):
                end = -(-n // au.BLOCK) * au.BLOCK
                assert (flat[at + n:at + end] == 0).all()


def _same(t, a):
    return np.array_equal(t.cpu().numpy().view(np.uint32), a.view(np.uint32))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gt", TYPES, ids=["gf32", "gf16", "gbf16"])
@pytest.mark.parametrize("out", [None] + TYPES, ids=["none", "f32", "f16", "bf16"])
@pytest.mark.parametrize("shift", [0, 1])
def test_step_matches_single_roundings(bits, gt, out, shift):
    r = Run(SIZES, [gt], [out] if out else None, bits, shift=shift, seed=1, weight_decay=0.1)
    kw = dict(lr=1e-3, step=7, loss_scale=3.0, seed=123456789)
    for _ in range(2):  # the second from what the first has left
        r.expect(**kw)
        r.list.step(**kw)
        r.check()


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_from_zero(bits):
    r = Run(SIZES, TYPES, TYPES, bits, seed=2, warm=False)
    for step in (1, 2, 3):
        r.expect(lr=1e-2, step=step)
        r.list.step(lr=1e-2, step=step)
        r.check()


@pytest.mark.parametrize("bits", [32, 8])
def test_a_decay_and_a_rate_a_tensor(bits):
    n = len(SIZES)
    r = Run(SIZES, TYPES, TYPES, bits, seed=3, weight_decay=[0.01 * i for i in range(n)],
            lr_scale=[0.5 + 0.125 * i if i % 3 else 0.0 for i in range(n)])
    kw = dict(lr=3e-3, beta1=0.8, beta2=0.95, eps=1e-6, step=11)
    r.expect(**kw)
    r.list.step(**kw)
    r.check()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 128, 129, 1000, 4096, 4097])
def test_many_tensors(n, bits):
    """Tables of one part and several, searched in one step, two and three."""
    sizes = [(37 * i) % 61 if i % 50 else 5000 for i in range(n)]
    r = Run(sizes, TYPES, TYPES, bits, seed=4)
    r.expect(lr=1e-3, step=5)
    r.list.step(lr=1e-3, step=5)
    r.check()


def test_empty_lists():
    AdamList, AdamState = _mods()
    for sizes in ([], [0], [0, 0, 0]):
        for bits in (8, 32):
            t = [torch.empty(0, device="cuda") for _ in sizes]
            lst = AdamList(t, t, AdamState(sizes, bits=bits))
            lst.step(lr=1e-3, step=1)
            assert [x.numel() for x in lst.moments()] == [0, 0]
    torch.cuda.synchronize()


@pytest.mark.parametrize("bits", [32, 8])
def test_within_the_roundings_of_64_bits(bits):
    r = Run([50_000], [torch.float32], None, bits, seed=5, weight_decay=0.1)
    g, p, m, v = (x[0].copy() for x in (r.g, r.p, r.m, r.v))
    kw = dict(lr=1e-3, step=20, loss_scale=7.0)
    r.list.step(**kw)
    want, far = au.update64(g, p, m, v, r.scalars(0, **kw), bits)
    assert (np.abs(r.masters[0].double().cpu().numpy() - want[0]) <= far[0]).all()
    got = [t[:50_000].double().cpu().numpy() for t in r.list.moments()]
    for x, y, d, octaves in zip(got, want[1:], far[1:], (16, 32)):
        if bits == 8:
            # a step of the pattern: an eighth of the power of two below the value; what lies
            # `octaves` below the block's largest value may go to zero or to the smallest code
            step = 2.0 ** np.floor(np.log2(np.maximum(np.abs(y) + d, 2.0 ** -126))) / 8
            pad = np.zeros(-(-y.size // au.BLOCK) * au.BLOCK)
            pad[:y.size] = np.abs(y)
            least = np.repeat(pad.reshape(-1, au.BLOCK).max(1), au.BLOCK)[:y.size]
            d = d + np.maximum(step, least * 2.0 ** (2 - octaves))
        assert (np.abs(x - y) <= d).all()


def test_rounding_is_unbiased():
    """40000 elements of one value v: with f the part of the gap passed, the mean of the rounded
    values is v within five standard deviations, gap sqrt(f (1 - f) / n)."""
    n = 40_000
    AdamList, AdamState = _mods()
    for seed in range(4):
        for value in (1.0, 1.01, 1.06, 1.12, 1.5 + 0.125 * 0.3):
            g = torch.full((n,), value, device="cuda")
            w = torch.zeros(n, device="cuda")
            lst = AdamList([g], [w], AdamState([n], bits=8))
            # beta = 0: m = g, v = g^2
            lst.step(lr=0.0, beta1=0.0, beta2=0.0, step=1, seed=seed)
            for got, x in zip(lst.moments(), (np.float32(value), np.float32(value) ** 2)):
                got, x = got[:n].double(), float(x)
                gap = 2.0 ** math.floor(math.log2(x)) / 8
                f = x / gap - math.floor(x / gap)
                bound = 5 * gap * math.sqrt(f * (1 - f) / n) + gap * 2.0 ** -17
                assert abs(got.mean().item() - x) <= bound
                assert set(((got / gap).round() * gap - got).tolist()) == {0.0}


def test_seeds_and_tensors_round_apart():
    n = 8192
    AdamList, AdamState = _mods()
    g = torch.full((n,), 1.06, device="cuda")

    def values(seed):
        w = [torch.zeros(n, device="cuda") for _ in range(2)]
        state = AdamState([n, n], bits=8)
        lst = AdamList([g, g.clone()], w, state)
        lst.step(lr=0.0, beta1=0.0, beta2=0.0, step=1, seed=seed)
        return state.m.clone(), state.v.clone()
    a, b, c = values(1), values(1), values(2)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # rounded up with probability f, independently: equal with f^2 + (1 - f)^2 (m: f = 0.48,
    # 0.501; v = 1.06^2: f = 0.989, 0.978), within five standard deviations
    for x, y, value in ((a[0], c[0], 1.06), (a[1], c[1], 1.06 ** 2),
                        (a[0][:n], a[0][n:], 1.06), (a[1][:n], a[1][n:], 1.06 ** 2),
                        (a[0][:4096], a[0][4096:n], 1.06)):
        f = (value - 1.0) * 8
        same = f * f + (1 - f) * (1 - f)
        far = 5 * math.sqrt(same * (1 - same) / x.numel())
        assert abs((x == y).float().mean().item() - same) < far


@pytest.mark.parametrize("bits", [32, 8])
def test_small_roots_without_eps(bits):
    """eps = 0 and v down to the smallest fp32: the first step is lr in every element that moves
    (v below 2^-149 is zero, and m / 0 infinite, in fp32 too)."""
    AdamList, AdamState = _mods()
    g = torch.from_numpy(np.exp2(np.linspace(-64, 40, 500)).astype(np.float32)).cuda()
    w = torch.zeros_like(g)
    AdamList([g], [w], AdamState([500], bits=bits)).step(lr=2.0 ** -10, eps=0.0, step=1,
                                                         beta2=0.5)
    # v = g^2 / 2 from 2^-129, of which fp32 keeps 20 bits at least: 2^-21 of it, half of that
    # in the root, and 14 E < 2^-20
    assert ((w.double() + 2.0 ** -10).abs() <= 2.0 ** -10 * (2.0 ** -22 + 2.0 ** -20)).all()


def test_wide_blocks():
    """Values from the smallest fp32 to the largest in one block."""
    n = 256
    x = np.exp2(np.linspace(-149, 126, n)).astype(np.float32)
    x[::3] *= -1
    AdamList, AdamState = _mods()
    g = torch.from_numpy(x).cuda()
    w = torch.zeros(n, device="cuda")
    state = AdamState([n], bits=8)
    lst = AdamList([g], [w], state)
    lst.step(lr=0.0, beta1=0.0, beta2=0.5, step=1, seed=3)
    with np.errstate(over="ignore"):
        v = np.float32(0.5) * (x * x)
    r = au.random_bits(3, 0, 0, n)
    mc, me = au.encode(x, r & np.uint32(0xFFFF), 16, 7)
    vc, ve = au.encode(v, r >> np.uint32(16), 32, 8)
    for got, want in ((state.m, mc), (state.m_exp, me), (state.v, vc), (state.v_exp, ve)):
        assert np.array_equal(got.cpu().numpy(), want)
    assert (vc[v > 0] > 0).all()


def test_nan_and_inf_without_a_norm():
    """What a step without skip makes of them: the element's own values, its block's codes."""
    n = 300
    AdamList, AdamState = _mods()
    for bits in (8, 32):
        g = torch.full((n,), 1e-3, device="cuda")
        g[130], g[131] = float("nan"), float("inf")
        w = torch.ones(n, device="cuda")
        lst = AdamList([g], [w], AdamState([n], bits=bits))
        lst.step(lr=1e-3, step=1)
        bad = ~torch.isfinite(w)
        assert torch.nonzero(bad)[:, 0].tolist() == [130, 131]
        m, v = (t[:n].float() for t in lst.moments())
        assert torch.isnan(m[130]) and torch.isnan(v[130])
        assert torch.isinf(m[131]) and torch.isinf(v[131])
        for t in (m, v):
            assert torch.isfinite(t[:128]).all() and (t[:128] != 0).all()
            assert torch.isfinite(t[256:n]).all() and (t[256:n] != 0).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_clip_and_skip_of_a_norm(bits):
    from zero_sharded_optimizer_rank_amd.tensors import GradList
    r = Run(SIZES, TYPES, TYPES, bits, seed=6)
    norm = GradList(r.grads)
    with pytest.raises(RuntimeError, match="norm"):
        r.list.step(lr=1e-3, step=1, norm=norm)
    res = norm.norm(max_grad_norm=0.05, loss_scale=4.0)
    assert res.clip_coef.item() < 1
    kw = dict(lr=1e-3, step=9, loss_scale=4.0)
    r.expect(coef=res.clip_coef.item(), **kw)
    r.list.step(norm=norm, **kw)
    r.check()
    r.grads[5][2] = float("inf")
    before = [t.clone() for t in (r.state.m, r.state.v, *r.masters, *r.params)]
    norm.norm(max_grad_norm=0.05, loss_scale=4.0)
    r.list.step(norm=norm, **kw)
    for a, b in zip(before, (r.state.m, r.state.v, *r.masters, *r.params)):
        assert torch.equal(a, b)


def test_same_bits_as_the_shard_update():
    from zero_sharded_optimizer_rank_amd import abi
    n = 100_003
    g = torch.Generator().manual_seed(7)
    grad = (torch.randn(n, generator=g) * 1e-3).cuda()
    master = (torch.randn(n, generator=g) * 0.02).cuda()
    AdamList, AdamState = _mods()
    for step in (1, 2, 999):
        a = [master.clone(), torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"),
             torch.zeros(n, dtype=torch.float16, device="cuda")]
        plan, _ = abi.zero_plan([n], 1)
        res = torch.zeros(abi.RESULT_BYTES, dtype=torch.uint8, device="cuda")
        res.view(torch.float32)[10] = 0.75
        args = abi.step_args(lr=2e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1,
                             max_grad_norm=1.0, loss_scale=1.0, step=step)
        abi.zero_adam_apply(plan, 0, grad, *a, args, res, torch.cuda.current_stream())
        state = AdamState([n])
        w, out = master.clone(), torch.zeros(n, dtype=torch.float16, device="cuda")
        lst = AdamList([grad], [w], state, params=[out], weight_decay=0.1)
        abi.zero_tensors_adam(lst.list, args, 0, res, torch.cuda.current_stream())
        for x, y in zip(a, (w, state.m[:n], state.v[:n], out)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("bits", [32, 8])
def test_other_streams_and_graphs(bits):
    r = Run(SIZES, TYPES, TYPES, bits, seed=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r.expect(lr=1e-3, step=1)
    r.list.step(lr=1e-3, step=1, stream=side)
    r.list.moments(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    r.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.list.step(lr=1e-3, step=2)
        m, v = r.list.moments()
    for _ in range(3):  # a replay is that step again
        graph.replay()
        r.expect(lr=1e-3, step=2)
        r.check()
        for t in r.grads:  # eager work between the replays
            t.mul_(0.5)
        r.g = [t.float().cpu().numpy() for t in r.grads]
        torch.cuda.synchronize()


def test_moments_in_fp32_and_kept_places():
    from zero_sharded_optimizer_rank_amd import abi
    AdamList, AdamState = _mods()
    sizes = [130, 5, 4097]
    r = Run(sizes, [torch.float32], None, 8, seed=9)
    n = r.state.elements
    m, v = (torch.full((n,), GUARD, device="cuda") for _ in range(2))
    abi.zero_tensors_adam_moments(r.list.list, m, v, abi.ZERO_F32, torch.cuda.current_stream())
    a, b = r.list.moments()
    at = 0
    for i, k in enumerate(sizes):
        off = r.state.offsets[i]
        for x, y in ((m, a), (v, b)):
            assert (x[at:off] == GUARD).all()
            assert torch.equal(x[off:off + k], y[off:off + k].float())
        at = off + k
    assert (m[at:] == GUARD).all() and (v[at:] == GUARD).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_offsets_past_32_bits(bits):
    """A tensor of 2^32 + 20003 elements behind another; windows of it against the CPU."""
    n = (1 << 32) + 20003
    free = torch.cuda.mem_get_info()[0]
    if free < n * (2 + 4 + (8 if bits == 32 else 6.1)) + (4 << 30):
        pytest.skip("not enough memory")
    AdamList, AdamState = _mods()
    small = torch.full((10,), 0.5, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(n, device="cuda")
    state = AdamState([10, n], bits=bits)
    lst = AdamList([small, g], [torch.zeros(10, device="cuda"), w], state)
    rng = np.random.default_rng(10)
    k = 5000
    windows = [0, (1 << 31) - 2432, (1 << 32) - 2432, n - k]  # multiples of a block, or the end
    windows[-1] -= windows[-1] % au.BLOCK
    data = []
    for at in windows:
        x = torch.from_numpy(rng.standard_normal(k).astype(np.float32)).bfloat16()
        g[at:at + k].copy_(x)
        data.append(x.float().numpy())
    lst.step(lr=1e-2, step=1, seed=77)
    m, v = lst.moments()
    s = au.scalars(1e-2, 0.9, 0.999, 1e-8, 1, 1.0, 0.0, 1.0, 1.0)
    zero = np.zeros(k, dtype=np.float32)
    off = state.offsets[1]
    for at, x in zip(windows, data):
        p1, m1, v1 = au.update32(x, zero, zero, zero, s)
        if bits == 32:
            assert _same(w[at:at + k], p1)
        else:
            want, far = au.update64(x, zero, zero, zero, s, bits)
            assert (np.abs(w[at:at + k].double().cpu().numpy() - want[0]) <= far[0]).all()
        if bits == 8:
            r = au.random_bits(77, 1, at, k)
            m1 = au.decode(*au.encode(m1, r & np.uint32(0xFFFF), 16, 7), 16, 7)
            v1 = au.decode(*au.encode(v1, r >> np.uint32(16), 32, 8), 32, 8)
        assert _same(m[off + at:off + at + k].float(), m1)
        assert _same(v[off + at:off + at + k].float(), v1)
    assert int((w != 0).sum()) <= 4 * k
