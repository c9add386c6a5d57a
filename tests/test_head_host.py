"""The head's loss (zero_head_*) on the CPU: argument checks, the workspace's
size, and the 64-bit reference's gradients against differences."""
import ctypes

import pytest

from zero_sharded_optimizer_rank_amd import abi

torch = pytest.importorskip("torch")

X, W, Y, DX, DW, WS, RES = (0x10000000 * (i + 1) for i in range(7))  # never dereferenced
GOOD = dict(tokens=5, hidden=64, vocab=100, x=X, ldx=64, w=W, ldw=64, labels=Y,
            dtype=abi.ZERO_BF16, mean=1, loss_scale=1.0)


def _head(**kw):
    a = dict(GOOD)
    a.update(kw)
    return abi.zero_head_t(*(a[n] for n, _ in abi.zero_head_t._fields_))


def _grads(**kw):
    a = dict(dx=DX, lddx=64, dw=DW, lddw=64, dw_dtype=abi.ZERO_BF16, accumulate=0)
    a.update(kw)
    return abi.zero_head_grads_t(*(a[n] for n, _ in abi.zero_head_grads_t._fields_))


def _loss(head, token_loss=None, lse=None, ws=WS, n=1 << 30, res=RES):
    abi.zero_head_loss(head, token_loss, lse, ws, n, res)


def _grad(head=None, lse=0x90000000, grads=None, ws=WS, n=1 << 30):
    abi.zero_head_grad(head or _head(), lse, grads or _grads(), ws, n)


INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("call,code", [
    (lambda: _loss(_head(tokens=-1)), abi.ZERO_EINVAL),
    (lambda: _loss(_head(tokens=(1 << 20) + 1)), abi.ZERO_EINVAL),
    (lambda: _loss(_head(hidden=0)), abi.ZERO_EINVAL),
    (lambda: _loss(_head(hidden=1 << 21, ldx=1 << 21, ldw=1 << 21)), abi.ZERO_EINVAL),
    (lambda: _loss(_head(vocab=0)), abi.ZERO_EINVAL),
    (lambda: _loss(_head(vocab=(1 << 30) + 1)), abi.ZERO_EINVAL),
    (lambda: _loss(_head(ldx=63)), abi.ZERO_EINVAL),
    (lambda: _loss(_head(ldw=63)), abi.ZERO_EINVAL),
    (lambda: _loss(_head(dtype=abi.ZERO_F32)), abi.ZERO_EINVAL),
    (lambda: _loss(_head(loss_scale=0.0)), abi.ZERO_EINVAL),
    (lambda: _loss(_head(loss_scale=NAN)), abi.ZERO_EINVAL),
    (lambda: _loss(_head(loss_scale=INF)), abi.ZERO_EINVAL),
    (lambda: _loss(_head(x=0)), abi.ZERO_EINVAL),
    (lambda: _loss(_head(w=0)), abi.ZERO_EINVAL),
    (lambda: _loss(_head(labels=0)), abi.ZERO_EINVAL),
    (lambda: _loss(_head(x=X + 1)), abi.ZERO_EALIGN),
    (lambda: _loss(_head(w=W + 1)), abi.ZERO_EALIGN),
    (lambda: _loss(_head(labels=Y + 4)), abi.ZERO_EALIGN),
    (lambda: _loss(_head(), token_loss=RES + 2), abi.ZERO_EALIGN),
    (lambda: _loss(_head(), lse=RES + 2), abi.ZERO_EALIGN),
    (lambda: _loss(_head(), res=None), abi.ZERO_EINVAL),
    (lambda: _loss(_head(), res=RES + 4), abi.ZERO_EALIGN),
    (lambda: _loss(_head(), ws=None), abi.ZERO_EINVAL),
    (lambda: _loss(_head(), ws=WS + 128), abi.ZERO_EALIGN),
    (lambda: _loss(_head(), n=1000), abi.ZERO_ENOSPC),
    (lambda: _grad(lse=None), abi.ZERO_EINVAL),
    (lambda: _grad(lse=0x90000002), abi.ZERO_EALIGN),
    (lambda: _grad(grads=_grads(dx=0)), abi.ZERO_EINVAL),
    (lambda: _grad(grads=_grads(dw=0)), abi.ZERO_EINVAL),
    (lambda: _grad(grads=_grads(lddx=63)), abi.ZERO_EINVAL),
    (lambda: _grad(grads=_grads(lddw=63)), abi.ZERO_EINVAL),
    (lambda: _grad(grads=_grads(dw_dtype=abi.ZERO_F16)), abi.ZERO_EINVAL),
    (lambda: _grad(grads=_grads(dw=DW + 2, dw_dtype=abi.ZERO_F32)), abi.ZERO_EALIGN),
    (lambda: _grad(grads=_grads(dx=X)), abi.ZERO_EINVAL),
    (lambda: _grad(grads=_grads(dw=W + 128)), abi.ZERO_EINVAL),
    (lambda: _grad(grads=_grads(dw=DX)), abi.ZERO_EINVAL),
    (lambda: _grad(grads=_grads(dx=Y)), abi.ZERO_EINVAL),
    (lambda: _grad(n=1000), abi.ZERO_ENOSPC),
])
def test_refusals(call, code):
    with pytest.raises(abi.ZeroError) as e:
        call()
    assert e.value.code == code
    assert abi.zero_last_error()


def test_null_structures():
    so = abi.lib()
    assert so.zero_head_loss(None, None, None, WS, 1 << 30, RES, None) == abi.ZERO_EINVAL
    assert so.zero_head_grad(ctypes.byref(_head()), 0x90000000, None, WS, 1 << 30, None) == \
        abi.ZERO_EINVAL
    assert so.zero_head_workspace_bytes(None, 1) == 0
    assert abi.zero_head_workspace_bytes(_head(hidden=0), True) == 0


def test_workspace_bytes():
    need = lambda grad, **kw: abi.zero_head_workspace_bytes(_head(**kw), grad)
    big = dict(tokens=8192, hidden=4096, vocab=128256, ldx=4096, ldw=4096)
    # far less than the logits (fp32 4.2 GB, 16-bit 2.1 GB)
    assert need(False, **big) < 0.2e9
    assert need(True, **big) < 1.6e9
    # a w whose rows do not start on 16-byte boundaries is laid out once more
    copy = 2 * 128256 * 4096
    assert copy <= need(False, **dict(big, w=W + 2)) - need(False, **big) <= copy + 256
    assert need(False, **dict(big, ldw=4097)) > copy


@pytest.mark.parametrize("mean", [True, False])
def test_reference_gradients_against_differences(mean):
    from head_util import reference
    g = torch.Generator().manual_seed(0)
    x = torch.randn(4, 6, generator=g, dtype=torch.float64)
    w = torch.randn(5, 6, generator=g, dtype=torch.float64)
    y = torch.tensor([2, -100, 0, 4])
    ref = reference(x, w, y, loss_scale=8.0, mean=mean)

    def loss(x, w):
        return reference(x, w, y, mean=mean)["loss"][0] * 8.0

    h = 1e-6  # central differences: error ~ h^2 and 1e-16 / h, both under 1e-8 here
    for name, t in (("dx", x), ("dw", w)):
        got = torch.zeros_like(t)
        for i in range(t.numel()):
            a, b = t.clone(), t.clone()
            a.view(-1)[i] += h
            b.view(-1)[i] -= h
            got.view(-1)[i] = (loss(*((a, w) if name == "dx" else (x, a)))
                               - loss(*((b, w) if name == "dx" else (x, b)))) / (2 * h)
        assert (got - ref[name][0]).abs().max() < 1e-7, name


def test_loss_head_refusals():
    from zero_sharded_optimizer_rank_amd.head import LossHead
    with pytest.raises(TypeError):
        LossHead(4, 8, 16, torch.float32)
    with pytest.raises(ValueError):
        LossHead(4, 8, 16, torch.float16, device="cpu")
    with pytest.raises(ValueError):
        LossHead(4, 0, 16, torch.float16)


def test_tiles_of_one_launch():
    """The logits' tiles fit one launch, or the call is refused."""
    ok = dict(tokens=1 << 20, hidden=8, ldx=8, ldw=8)
    limit = 2 ** 23 // (2 ** 20 // 256) * 256
    assert abi.zero_head_workspace_bytes(_head(vocab=limit - 256, **ok), False) > 0
    for vocab in (limit - 255, limit, 1 << 30):
        assert abi.zero_head_workspace_bytes(_head(vocab=vocab, **ok), False) == 0
        with pytest.raises(abi.ZeroError) as e:
            _loss(_head(vocab=vocab, **ok), n=1 << 62)
        assert e.value.code == abi.ZERO_EINVAL
    assert abi.zero_head_workspace_bytes(
        _head(vocab=1 << 30, tokens=65, hidden=8, ldx=8, ldw=8), False) > 0


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("vocab", [100, 1 << 21, (1 << 21) + 1, 1 << 30])
def test_workspace_of_an_empty_batch(grad, vocab):
    """No token needs the room of one: the join writes its sum whatever the count."""
    need = [abi.zero_head_workspace_bytes(_head(tokens=t, hidden=8, vocab=vocab, ldx=8, ldw=8),
                                          grad) for t in (0, 1)]
    assert need[0] == need[1] > 0


SHAPES = [(4096, 128256), (1600, 50257), (8192, 32000), (3, 39070), (72, 9001), (64, 700),
          (8, (1 << 21) + 1)]


@pytest.mark.parametrize("hidden,vocab", SHAPES)
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("w", [W, W + 2])
def test_workspace_holds_every_smaller_batch(hidden, vocab, grad, w):
    """A head for T tokens takes batches of 0 to T: the plan changes at 64 tokens and by
    the tile of 256, and its room for g and dx's sums does not grow with each."""
    counts = [0, 1, 64, 65] + [256 * k + d for k in range(1, 160) for d in (0, 1)]
    most = 0
    for t in counts:
        need = abi.zero_head_workspace_bytes(
            _head(tokens=t, hidden=hidden, vocab=vocab, ldx=hidden, w=w, ldw=hidden), grad)
        assert need >= most, (t, need, most)
        most = need


@pytest.mark.parametrize("hidden,vocab,most,fewer", [
    (4096, 128256, 5000, 4096), (4096, 128256, 16384, 12000), (1600, 50257, 12000, 10496),
    (8192, 32000, 2048, 1792), (4096, 128256, 5000, 64)])
@pytest.mark.parametrize("grad", [False, True])
def test_smaller_batches_are_not_refused(hidden, vocab, most, fewer, grad):
    """What a call of `fewer` tokens asks for (a refusal names it) is there in the workspace of
    a head for `most`."""
    size = dict(hidden=hidden, vocab=vocab, ldx=hidden, ldw=hidden)
    far = [1 << (40 + k) for k in range(4)]  # apart for any of these sizes
    head = _head(tokens=fewer, x=far[0], w=far[1], **size)
    with pytest.raises(abi.ZeroError) as e:
        if grad:
            _grad(head, grads=_grads(dx=far[2], lddx=hidden, dw=far[3], lddw=hidden), n=1)
        else:
            _loss(head, n=1)
    assert e.value.code == abi.ZERO_ENOSPC
    need = int(str(e.value).split("<")[1])
    assert 0 < need <= abi.zero_head_workspace_bytes(_head(tokens=most, **size), grad)


def test_one_row_of_a_far_strided_tensor():
    """The stride of a single row means nothing: the last token of one long sequence."""
    from zero_sharded_optimizer_rank_amd.head import LossHead
    h = LossHead.__new__(LossHead)
    h.hidden, h.device = 8, torch.device("cpu")
    for far in (8, 1 << 21, 3):
        assert h._matrix(torch.zeros(8).as_strided((1, 8), (far, 1)), 1, "x") == 8
    assert h._matrix(torch.zeros(0, 8), 0, "x") == 8
    assert h._matrix(torch.zeros(24).as_strided((2, 8), (16, 1)), 2, "x") == 16
    with pytest.raises(ValueError, match="overlap"):
        h._matrix(torch.zeros(24).as_strided((2, 8), (3, 1)), 2, "x")
