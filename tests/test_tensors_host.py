"""Argument checks of the tensor-list calls (zero_tensors_*) on the CPU: every
refusal happens before anything touches the GPU."""
import pytest

from zero_sharded_optimizer_rank_amd import abi

SRC, DST, WS, RES = 0x10000, 0x80000, 0x200000, 0x300000  # never dereferenced
F32, F16, BF16 = abi.ZERO_F32, abi.ZERO_F16, abi.ZERO_BF16


def _args(**kw):
    a = dict(lr=0.0, beta1=0.0, beta2=0.0, eps=0.0, weight_decay=0.0, max_grad_norm=1.0,
             loss_scale=1.0, step=1)
    a.update(kw)
    return abi.step_args(**a)


def _norm(entries, args=None, sq=None, ws=WS, ws_bytes=1 << 20, res=RES, n=None):
    abi.zero_tensors_norm(abi.tensor_table(entries), len(entries) if n is None else n,
                          args or _args(), sq, ws, ws_bytes, res)


def _clip(entries, args=None, out_scale=1.0, res=RES):
    abi.zero_tensors_clip(abi.tensor_table(entries), len(entries), args or _args(), out_scale,
                          res)


GOOD = (SRC, F32, DST, F16, 100)


@pytest.mark.parametrize("call,code", [
    (lambda: _norm([GOOD], n=-1), abi.ZERO_EINVAL),
    (lambda: _norm([(SRC, F32, DST, F16, -1)]), abi.ZERO_EINVAL),
    (lambda: _norm([(SRC, 3, DST, F16, 4)]), abi.ZERO_EINVAL),
    (lambda: _norm([(None, F32, DST, F16, 4)]), abi.ZERO_EINVAL),
    (lambda: _norm([(SRC + 2, F32, DST, F16, 4)]), abi.ZERO_EALIGN),
    (lambda: _norm([(SRC + 1, BF16, DST, F16, 4)]), abi.ZERO_EALIGN),
    (lambda: _norm([GOOD], args=_args(loss_scale=0.0)), abi.ZERO_EINVAL),
    (lambda: _norm([GOOD], args=_args(loss_scale=float("nan"))), abi.ZERO_EINVAL),
    (lambda: _norm([GOOD], args=_args(max_grad_norm=float("nan"))), abi.ZERO_EINVAL),
    (lambda: _norm([GOOD], args=_args(other_sq=-1.0)), abi.ZERO_EINVAL),
    (lambda: _norm([GOOD], args=_args(other_q=5)), abi.ZERO_EINVAL),
    (lambda: _norm([GOOD], sq=RES + 4), abi.ZERO_EALIGN),
    (lambda: _norm([GOOD], ws=None), abi.ZERO_EINVAL),
    (lambda: _norm([GOOD], ws=WS + 8), abi.ZERO_EALIGN),
    (lambda: _norm([GOOD], ws_bytes=64), abi.ZERO_ENOSPC),
    (lambda: _norm([GOOD], res=None), abi.ZERO_EINVAL),
    (lambda: _norm([GOOD], res=RES + 4), abi.ZERO_EALIGN),
    (lambda: _clip([(SRC, F32, DST, 7, 4)]), abi.ZERO_EINVAL),
    (lambda: _clip([(SRC, F32, None, F16, 4)]), abi.ZERO_EINVAL),
    (lambda: _clip([(SRC, F32, DST + 1, F16, 4)]), abi.ZERO_EALIGN),
    (lambda: _clip([(SRC, F32, SRC + 4, F32, 4)]), abi.ZERO_EINVAL),
    (lambda: _clip([(SRC, F32, SRC, F16, 4)]), abi.ZERO_EINVAL),
    (lambda: _clip([GOOD], out_scale=0.0), abi.ZERO_EINVAL),
    (lambda: _clip([GOOD], out_scale=float("inf")), abi.ZERO_EINVAL),
    (lambda: _clip([GOOD], out_scale=1e-30, args=_args(loss_scale=1e30)), abi.ZERO_EINVAL),
    (lambda: _clip([GOOD], res=None), abi.ZERO_EINVAL),
])
def test_refusals(call, code):
    with pytest.raises(abi.ZeroError) as e:
        call()
    assert e.value.code == code
    assert abi.zero_last_error()


def test_norm_clip_checks_both_halves_first():
    bad_clip = [(SRC, F32, None, F16, 4)]
    with pytest.raises(abi.ZeroError) as e:
        abi.zero_tensors_norm_clip(abi.tensor_table(bad_clip), 1, _args(), 1.0, None, WS, 1 << 20,
                                   RES)
    assert e.value.code == abi.ZERO_EINVAL


def test_workspace_bytes():
    def ws(*numels):
        return abi.zero_tensors_workspace_bytes(
            abi.tensor_table([(SRC, F32, DST, F32, n) for n in numels]), len(numels))
    assert ws() > 0
    assert ws(-1) == 0
    # a chunk's partial is 16 bytes; an empty tensor has one chunk
    assert ws(0) == ws(1) == ws(16384)
    assert ws(16385) == ws(1) + 16
    # long lists take longer chunks: the partials stay near 32768 for any length
    for n in (1 << 28, (1 << 28) + 1, 1 << 33, 1 << 40):
        assert ws(n) <= ws(1) + 16 * 32768
    assert abi.lib().zero_tensors_workspace_bytes(None, 1) == 0
    assert abi.lib().zero_tensors_workspace_bytes(None, -1) == 0


def test_grad_list_refusals_on_the_host():
    torch = pytest.importorskip("torch")
    from zero_sharded_optimizer_rank_amd.tensors import GradList
    dev = torch.device("cuda", 0)
    with pytest.raises(ValueError, match="is on cpu"):
        GradList([torch.zeros(3)], device=dev)
    with pytest.raises(TypeError, match="dtype"):
        GradList([torch.zeros(3, dtype=torch.float64)], device=dev)
    with pytest.raises(TypeError, match="not a tensor"):
        GradList([3.0], device=dev)
    with pytest.raises(ValueError, match="outputs for"):
        GradList([torch.zeros(3)], out=[], device=dev)


@pytest.mark.parametrize("device", ["cpu", "cpu:0", "meta"])
@pytest.mark.parametrize("tensors", [0, 1])
def test_grad_list_is_on_a_gpu(device, tensors):
    """An empty list too: its kernels write the list's own results."""
    torch = pytest.importorskip("torch")
    from zero_sharded_optimizer_rank_amd.tensors import GradList
    with pytest.raises(ValueError, match="not a GPU"):
        GradList([torch.zeros(3, device=device)] * tensors, device=device)


def test_entries_that_share_memory():
    torch = pytest.importorskip("torch")
    from zero_sharded_optimizer_rank_amd.tensors import _check_apart
    b = torch.zeros(100)
    a, c, d = b[:40], b[40:60], b[60:]
    empty = b[10:10]
    _check_apart([a, c, d, empty, empty], [a, c, d, empty, empty])
    _check_apart([a, c], [torch.zeros(40), torch.zeros(20)])
    for tensors, out in (([a, a], [a, a]),                    # twice, in place
                         ([a, c, b[:1]], [a, c, b[:1]]),
                         ([a, c], [d, d[:20]]),               # outputs over each other
                         ([a, c], [c, a]),                    # outputs over other inputs
                         ([b[:90], c], [torch.zeros(90), torch.zeros(20)])):
        with pytest.raises(ValueError, match="share memory"):
            _check_apart(tensors, out)


def test_stream_of_another_device():
    torch = pytest.importorskip("torch")
    from types import SimpleNamespace
    from zero_sharded_optimizer_rank_amd.tensors import stream_of
    here = SimpleNamespace(device_index=1, cuda_stream=77)
    assert stream_of(torch.device("cuda", 1), here) == 77
    with pytest.raises(ValueError, match="the stream is on cuda:1"):
        stream_of(torch.device("cuda", 0), here)
