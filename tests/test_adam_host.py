"""Argument checks of the list update (zero_tensors_adam*) on the CPU: every refusal happens
before anything touches the GPU; and the 8-bit moments' arithmetic on its own."""
import numpy as np
import pytest

import adam_util as au
from zero_sharded_optimizer_rank_amd import abi

BASE, STEP = 0x100000, 0x10000  # never dereferenced
TABLE, RES = 0x900000, 0xA00000


def _entry(**kw):
    names = ("grad", "master", "m", "v", "m_exp", "v_exp", "param")
    e = {k: BASE + i * STEP for i, k in enumerate(names)}
    e.update(numel=100, grad_dtype=abi.ZERO_BF16, param_dtype=abi.ZERO_F16, moment_bits=8)
    e.update(kw)
    return e


def _args(**kw):
    a = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, max_grad_norm=0.0,
             loss_scale=1.0, step=1)
    a.update(kw)
    return abi.step_args(**a)


def _prepare(entries, n=None, table=TABLE, table_bytes=1 << 20):
    abi.zero_tensors_adam_prepare(abi.adam_table(entries), len(entries) if n is None else n,
                                  table, table_bytes)


LIST = abi.zero_adam_list_t(TABLE, 0, 1, 128, 1, 0)


def _step(adam_list=LIST, args=None, res=None):
    abi.zero_tensors_adam(adam_list, args or _args(), 0, res)


def _read(m=BASE, v=BASE + STEP, dtype=abi.ZERO_F32, adam_list=LIST):
    abi.zero_tensors_adam_moments(adam_list, m, v, dtype)


@pytest.mark.parametrize("call,code", [
    (lambda: _prepare([_entry()], n=-1), abi.ZERO_EINVAL),
    (lambda: _prepare([_entry()], table=None), abi.ZERO_EINVAL),
    (lambda: _prepare([_entry()], table=TABLE + 4), abi.ZERO_EALIGN),
    (lambda: _prepare([_entry()], table_bytes=32), abi.ZERO_ENOSPC),
    (lambda: _prepare([_entry(numel=-1)]), abi.ZERO_EINVAL),
    (lambda: _prepare([_entry(numel=(1 << 39) + 1)]), abi.ZERO_EINVAL),
    (lambda: _prepare([_entry(grad_dtype=3)]), abi.ZERO_EINVAL),
    (lambda: _prepare([_entry(param_dtype=-1)]), abi.ZERO_EINVAL),
    (lambda: _prepare([_entry(moment_bits=16)]), abi.ZERO_EINVAL),
    (lambda: _prepare([_entry(weight_decay=float("nan"))]), abi.ZERO_EINVAL),
    (lambda: _prepare([_entry(lr_scale=-1.0)]), abi.ZERO_EINVAL),
    (lambda: _prepare([_entry(lr_scale=float("inf"))]), abi.ZERO_EINVAL),
    (lambda: _prepare([_entry(grad=None)]), abi.ZERO_EINVAL),
    (lambda: _prepare([_entry(master=None)]), abi.ZERO_EINVAL),
    (lambda: _prepare([_entry(m=None)]), abi.ZERO_EINVAL),
    (lambda: _prepare([_entry(v=None, moment_bits=32)]), abi.ZERO_EINVAL),
    (lambda: _prepare([_entry(m_exp=None)]), abi.ZERO_EINVAL),
    (lambda: _prepare([_entry(v_exp=None)]), abi.ZERO_EINVAL),
    (lambda: _prepare([_entry(grad=BASE + 1)]), abi.ZERO_EALIGN),
    (lambda: _prepare([_entry(master=BASE + STEP + 2)]), abi.ZERO_EALIGN),
    (lambda: _prepare([_entry(m=BASE + 2 * STEP + 1)]), abi.ZERO_EALIGN),
    (lambda: _prepare([_entry(param=BASE + 6 * STEP + 1)]), abi.ZERO_EALIGN),
    (lambda: _prepare([_entry(param=BASE + 8)]), abi.ZERO_EINVAL),           # over the gradient
    (lambda: _prepare([_entry(v=BASE + 2 * STEP + 96)]), abi.ZERO_EINVAL),   # over m's last codes
    (lambda: _prepare([_entry(), _entry(m_exp=BASE + 5 * STEP)]), abi.ZERO_EINVAL),
    (lambda: _step(abi.zero_adam_list_t()), abi.ZERO_EINVAL),
    (lambda: _step(abi.zero_adam_list_t(TABLE, 1 << 33, 0, 1, 1, 0)), abi.ZERO_EINVAL),
    (lambda: _step(args=_args(lr=-1.0)), abi.ZERO_EINVAL),
    (lambda: _step(args=_args(beta1=1.0)), abi.ZERO_EINVAL),
    (lambda: _step(args=_args(step=0)), abi.ZERO_EINVAL),
    (lambda: _step(args=_args(loss_scale=0.0)), abi.ZERO_EINVAL),
    (lambda: _step(args=_args(loss_scale=1e60)), abi.ZERO_EINVAL),
    (lambda: _step(args=_args(eps=float("nan"))), abi.ZERO_EINVAL),
    (lambda: _step(res=RES + 4), abi.ZERO_EALIGN),
    (lambda: _read(m=None), abi.ZERO_EINVAL),
    (lambda: _read(dtype=abi.ZERO_F16), abi.ZERO_EINVAL),
    (lambda: _read(m=BASE + 2), abi.ZERO_EALIGN),
    (lambda: _read(v=BASE + 4), abi.ZERO_EINVAL),
    (lambda: _read(adam_list=abi.zero_adam_list_t()), abi.ZERO_EINVAL),
])
def test_refusals(call, code):
    with pytest.raises(abi.ZeroError) as e:
        call()
    assert e.value.code == code
    assert abi.zero_last_error()


def test_table_bytes():
    assert abi.zero_adam_table_bytes(-1) == 0
    assert 0 < abi.zero_adam_table_bytes(0) <= abi.zero_adam_table_bytes(1)
    assert abi.zero_adam_table_bytes(600) == 600 * abi.zero_adam_table_bytes(1)


def test_classes_refuse_on_the_host():
    torch = pytest.importorskip("torch")
    from zero_sharded_optimizer_rank_amd.adam import AdamState, _check_buffers_apart, _each
    with pytest.raises(ValueError, match="not a GPU"):
        AdamState([3], device="cpu")
    with pytest.raises(ValueError, match="bits"):
        AdamState([3], bits=4, device="cuda:0")
    with pytest.raises(ValueError, match=">= 0"):
        AdamState([-3], device="cuda:0")
    assert _each(0.5, 2, "x") == [0.5, 0.5] and _each([1, 2], 2, "x") == [1.0, 2.0]
    with pytest.raises(ValueError, match="for 3 tensors"):
        _each([1, 2], 3, "x")
    _check_buffers_apart([(0, 4, "a"), (8, 9, "c"), (4, 8, "b")])
    for spans in ([(0, 4, "a"), (3, 8, "b")], [(0, 10, "a"), (2, 3, "b")],
                  [(0, 4, "a"), (0, 4, "b")]):
        with pytest.raises(ValueError, match="share memory"):
            _check_buffers_apart(spans)


class _Fake:
    """Stands where a list's tensors would: the constructor's checks need no GPU."""

    def __init__(self, n, bits=32):
        import torch
        self.numels, self.offsets, self.bits = [n], [0], bits
        self.device = torch.device("cuda", 0)
        self.m = self.v = torch.zeros(n)
        self.m_exp = self.v_exp = None


def test_list_refuses_on_the_host():
    torch = pytest.importorskip("torch")
    from zero_sharded_optimizer_rank_amd.adam import AdamList
    t = torch.zeros(3)
    with pytest.raises(ValueError, match="is on cpu"):
        AdamList([t], [t], _Fake(3))
    with pytest.raises(ValueError, match="1 gradients, 0 masters"):
        AdamList([t], [], _Fake(3))
    with pytest.raises(ValueError, match="2 parameters"):
        AdamList([t], [t], _Fake(3), params=[t, t])
    with pytest.raises(TypeError, match="dtype"):
        AdamList([t.double()], [t], _Fake(3))
    with pytest.raises(ValueError, match="weight_decay"):
        AdamList([t], [t], _Fake(3), weight_decay=[1.0, 2.0])


def test_codes_hold_what_they_say():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(1000) * 2.0 ** rng.uniform(-6, 6, 1000)).astype(np.float32)
    x[::17] = 0
    u = rng.integers(0, 1 << 16, 1000).astype(np.uint32)
    for octaves, bits, y in ((16, 7, x), (32, 8, x * x)):
        code, exp = au.encode(y, u, octaves, bits)
        z = au.decode(code, exp, octaves, bits)
        assert ((z == 0) == (y == 0)).all() or bits == 7
        gap = 2.0 ** np.floor(np.log2(np.maximum(np.abs(y), 1e-30))) / 8
        near = np.abs(z.astype(np.float64) - y) < gap
        pad = np.zeros(1024)
        pad[:1000] = np.abs(y)
        low = np.abs(y) < np.repeat(pad.reshape(-1, 128).max(1), 128)[:1000] * 2.0 ** (2 - octaves)
        assert (near | low).all() and near.mean() > 0.95
        # a value that the codes hold stays, whatever the random bits
        again = au.encode(z, u, octaves, bits)
        assert (again[0] == code).all() and (again[1] == exp).all()
