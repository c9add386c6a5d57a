"""The training operators as a program runs them, one after another: two gated feed-forward blocks
with residuals and a language-model head forward and backward, the norm of all gradients, and the
AdamW step whose 16-bit weights the next forward pass reads.

Every operator has its own tests against 64-bit values; here each is checked on what the ones
before it have left: outputs and gradients against 64-bit values of the same 16-bit inputs, within
the bounds of ffn_util and head_util; norm, clip and update against the fp32 sequence on those
gradients (bit for bit with 32-bit moments, within adam_util.update64's bounds with 8)."""
import math

import numpy as np
import pytest

import adam_util as au
import ffn_util as fu
import head_util as hu

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

T, H, F, V = 96, 136, 264, 501
DT = torch.bfloat16
LAYERS = 2
NAMES = ("w_gate", "w_up", "w_down")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Program:
    """What a training program holds: fp32 masters, 16-bit weights, gradients, moments."""

    def __init__(self, bits, seed=0):
        from zero_sharded_optimizer_rank_amd.adam import AdamList, AdamState
        from zero_sharded_optimizer_rank_amd.ffn import GatedFFN
        from zero_sharded_optimizer_rank_amd.head import LossHead
        from zero_sharded_optimizer_rank_amd.tensors import GradList
        g = torch.Generator(device="cuda").manual_seed(seed)
        shapes = []
        for _ in range(LAYERS):
            shapes += [(F, H), (F, H), (H, F)]
        shapes.append((V, H))
        self.master = [torch.randn(*s, generator=g, device="cuda") * s[1] ** -0.5 for s in shapes]
        self.w = [m.to(DT) for m in self.master]
        # the head's gradient is accumulated in fp32, the blocks' leave in 16 bits
        self.grad = [torch.zeros(*s, dtype=DT, device="cuda") for s in shapes[:-1]]
        self.grad.append(torch.zeros(V, H, device="cuda"))
        self.ffn = GatedFFN(T, H, F, DT)
        self.saved = [self.ffn.new_saved() for _ in range(LAYERS)]
        self.head = LossHead(T, H, V, DT)
        self.norm = GradList(self.grad)
        self.state = AdamState([m.numel() for m in self.master], bits=bits)
        self.decay = [0.1] * (len(shapes) - 1) + [0.0]
        self.opt = AdamList(self.grad, self.master, self.state, params=self.w,
                            weight_decay=self.decay)
        self.x = torch.randn(T, H, generator=g, device="cuda").to(DT)
        self.y = torch.randint(0, V, (T,), generator=g, device="cuda")
        self.bits = bits

    def step(self, step, lr=1e-2, scale=4.0, max_norm=0.05):
        """One training step; nothing waits for the GPU.  The activations stay in self.a."""
        self.a = [self.x]
        for i in range(LAYERS):
            y = self.ffn.forward(self.a[-1], *self.w[3 * i:3 * i + 3], save=self.saved[i]).y
            self.a.append(self.a[-1] + y)
        self.grad[-1].zero_()
        r = self.head.loss_grad(self.a[-1], self.w[-1], self.y, loss_scale=scale,
                                dw=self.grad[-1], accumulate=True)
        self.d = [r.dx.clone()]
        for i in reversed(range(LAYERS)):
            gw = self.grad[3 * i:3 * i + 3]
            b = self.ffn.backward(self.d[0], self.a[i], *self.w[3 * i:3 * i + 3], self.saved[i],
                                  dw_gate=gw[0], dw_up=gw[1], dw_down=gw[2])
            self.d.insert(0, self.d[0] + b.dx)
        n = self.norm.norm(max_grad_norm=max_norm, loss_scale=scale)
        self.opt.step(lr=lr, step=step, loss_scale=scale, norm=self.norm, seed=step)
        return r, n


@pytest.mark.parametrize("bits", [32, 8])
def test_training_steps(bits):
    p = Program(bits)
    losses, clipped = [], []
    for step in (1, 2, 3):
        w = [t.clone() for t in p.w]
        master = [t.clone() for t in p.master]
        m0, v0 = (t.float().clone() for t in p.opt.moments())
        r, n = p.step(step)
        losses.append(r.loss.item())
        # forward and backward, on the weights that the last step has written
        for i in range(LAYERS):
            ref = fu.reference(p.a[i], *w[3 * i:3 * i + 3], "silu", p.d[i + 1])
            y = p.ffn.forward(p.a[i], *w[3 * i:3 * i + 3]).y
            fu.check(y, *ref["y"], "y")
            assert torch.equal(p.a[i] + y, p.a[i + 1])
            for name, g in zip(("dw_gate", "dw_up", "dw_down"), p.grad[3 * i:3 * i + 3]):
                fu.check_dw(g, ref, name)
        ref = hu.reference(p.a[-1], w[-1], p.y, loss_scale=4.0)
        assert abs(r.loss.item() - ref["loss"][0]) <= ref["loss"][1]
        hu.check(p.d[LAYERS], *ref["dx"], "dx")
        hu.check_dw(p.grad[-1], ref)
        # norm and clip of what lies there
        sq = math.fsum(float((g.double() ** 2).sum()) for g in p.grad)
        assert abs(n.norm.item() - math.sqrt(sq) / 4.0) <= 1e-9 * n.norm.item()
        coef = np.float32(min(1.0, 0.05 / (n.norm.item() + 1e-6)))
        assert n.clip_coef.item() == coef and n.skip.item() == 0
        clipped.append(coef < 1)
        # the update
        m1, v1 = (t.float() for t in p.opt.moments())
        for i, (g, k) in enumerate(zip(p.grad, p.state.numels)):
            at = p.state.offsets[i]
            old = [t.reshape(-1).float().cpu().numpy() for t in
                   (g, master[i], m0[at:at + k], v0[at:at + k])]
            s = au.scalars(1e-2, 0.9, 0.999, 1e-8, step, 4.0, p.decay[i], 1.0,
                           n.clip_coef.item())
            got = p.master[i].reshape(-1).cpu().numpy()
            want = au.update32(*old, s)
            if bits == 32:
                assert np.array_equal(got, want[0])
                for x, y in zip((m1, v1), want[1:]):
                    assert np.array_equal(x[at:at + k].cpu().numpy(), y)
            else:
                want64, far = au.update64(*old, s, bits=8)
                assert (np.abs(got - want64[0]) <= far[0]).all()
                rnd = au.random_bits(step, i, 0, k)
                for x, y, u, o, b in ((m1, want[1], rnd & np.uint32(0xFFFF), 16, 7),
                                      (v1, want[2], rnd >> np.uint32(16), 32, 8)):
                    assert np.array_equal(x[at:at + k].cpu().numpy(),
                                          au.decode(*au.encode(y, u, o, b), o, b))
            assert torch.equal(p.w[i], p.master[i].to(DT))
    assert all(math.isfinite(x) for x in losses) and any(clipped)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_bad_label_skips_the_step(bits):
    p = Program(bits, seed=1)
    p.step(1)
    kept = [t.clone() for t in (*p.w, *p.master, p.state.m, p.state.v)]
    good = p.y[3].item()
    p.y[3] = V  # outside the vocabulary: the loss and its gradients become NaN
    r, n = p.step(2)
    assert n.skip.item() == 1 and math.isnan(r.loss.item())
    for a, b in zip(kept, (*p.w, *p.master, p.state.m, p.state.v)):
        assert torch.equal(a, b)
    p.y[3] = good
    r, n = p.step(2)  # the same step again, as if it had not been
    assert n.skip.item() == 0 and math.isfinite(r.loss.item())
    assert not torch.equal(kept[0], p.w[0])


@pytest.mark.parametrize("bits", [32, 8])
def test_a_whole_step_in_a_graph(bits):
    """Captured once, replayed with eager work between, against an eager twin."""
    a, b = Program(bits, seed=2), Program(bits, seed=2)
    for p in (a, b):
        p.step(1)  # makes what is made on first use
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        a.step(2)
    for i in range(3):
        graph.replay()
        b.step(2)
        torch.cuda.synchronize()
        for x, y in zip((*a.w, *a.master, a.state.m, a.state.v, *a.grad),
                        (*b.w, *b.master, b.state.m, b.state.v, *b.grad)):
            assert torch.equal(x, y)
        for p in (a, b):  # other tokens for the next one
            p.x.mul_(0.5).add_(0.25)
            p.y.add_(7).remainder_(V)


def test_two_programs_on_two_streams():
    """Blocks, lists and states of their own do not meet."""
    progs = [Program(32, seed=3), Program(8, seed=4)]
    twins = [Program(32, seed=3), Program(8, seed=4)]
    streams = [torch.cuda.Stream() for _ in progs]
    torch.cuda.synchronize()
    for step in (1, 2, 3):
        for p, s in zip(progs, streams):
            with torch.cuda.stream(s):
                p.step(step)
    torch.cuda.synchronize()
    for p, q in zip(progs, twins):
        for step in (1, 2, 3):
            q.step(step)
        torch.cuda.synchronize()
        for x, y in zip((*p.w, *p.master, p.state.m, p.state.v),
                        (*q.w, *q.master, q.state.m, q.state.v)):
            assert torch.equal(x, y)
