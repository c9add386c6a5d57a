"""AdamW over a list of torch tensors, moments in 32 or in 8 bits.

PyTorch supplies the memory and the stream; the work runs in libzero_shard.so
(zero_tensors_adam).  An ``AdamState`` holds the moments of a list, an ``AdamList``
the table of its tensors; gradients, master weights and parameters stay the
caller's.
"""
from __future__ import annotations

from typing import Optional, Sequence, Tuple, Union

import torch

from . import abi
from .tensors import DTYPES, GradList, _check_tensor, on_device, stream_of


def _device(device):
    device = torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise ValueError(f"device {device} is not a GPU")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return device


class AdamState:
    """Moments of tensors with the given element counts, zero at first, in flat buffers.

    bits: 32 (m and v are float32) or 8 (m and v are uint8 codes, m_exp and v_exp the exponents
    that 128 neighbouring elements share).  Tensor i's moments start at element offsets[i], a
    multiple of 128.  Save the buffers to save a run, and copy into them to resume it: a list made
    of the state holds them where they lie.
    """

    def __init__(self, numels: Sequence[int], bits: int = 32, device=None):
        if bits not in (8, 32):
            raise ValueError(f"moments of {bits} bits: 8 and 32 are supported")
        self.numels, self.bits, self.device = [int(n) for n in numels], bits, _device(device)
        if any(n < 0 for n in self.numels):
            raise ValueError("element counts must be >= 0")
        block = abi.ZERO_ADAM_BLOCK
        self.offsets, at = [], 0
        for n in self.numels:
            self.offsets.append(at)
            at += -(-n // block) * block
        self.elements = at

        def zeros(count, dtype):
            return torch.zeros(count, dtype=dtype, device=self.device)

        wide = torch.float32 if bits == 32 else torch.uint8
        self.m, self.v = zeros(at, wide), zeros(at, wide)
        self.m_exp = self.v_exp = None
        if bits == 8:
            self.m_exp, self.v_exp = (zeros(at // block, torch.uint8) for _ in range(2))


def _each(value, n, what):
    values = list(value) if isinstance(value, (list, tuple)) else [value] * n
    if len(values) != n:
        raise ValueError(f"{len(values)} values of {what} for {n} tensors")
    return [float(v) for v in values]


MOMENTS = ("m", "v", "m_exp", "v_exp")


def _moments_of(state):
    """The state's buffers, checked: they may have been exchanged since it was made."""
    block, small = abi.ZERO_ADAM_BLOCK, state.bits == 8
    blocks = sum(-(-n // block) for n in state.numels)
    dtype = torch.uint8 if small else torch.float32
    buffers = tuple(getattr(state, name) for name in MOMENTS)
    for t, name, count in zip(buffers, MOMENTS, (block * blocks,) * 2 + (blocks,) * 2):
        if not small and name.endswith("exp"):
            continue
        if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.numel() != count \
                or not t.is_contiguous():
            raise ValueError(f"the state's {name} must be {count} contiguous elements of {dtype}")
        if t.device != state.device:
            raise ValueError(f"the state's {name} is on {t.device}, the state on {state.device}")
    return buffers


def _check_buffers_apart(spans) -> None:
    reach, owner = 0, ""
    for start, end, what in sorted(spans):
        if start < reach:
            raise ValueError(f"{owner} and {what} share memory")
        reach, owner = end, what


class AdamList:
    """One AdamW step over many tensors at once.

    grads: contiguous float32 / float16 / bfloat16 tensors, mixed as they come; masters: float32
    weights of the same sizes, updated in place; state: the list's AdamState; params: tensors of
    any of the three types that receive the new weights, or None.  weight_decay (decoupled) and
    lr_scale (a factor on the step's lr): one number, or one a tensor.  No two buffers may share
    memory.  The list is made for these tensors where they lie, as a ``GradList`` is: gradients
    that a step makes anew need a new list, and so does a state whose buffers were exchanged
    (calls refuse it).  Calls run on the given stream (default: the current
    stream of the list's device), which has to wait for the stream that the list was made on, as
    for any tensor; calls on one list must not overlap.  The list has to outlive their work, and
    the graphs that hold them.  A graph replays the scalars of the step that it captured, its bias
    correction, rate and seed: 8-bit moments are rounded by the same random bits each time, so a
    run of many steps calls ``step`` and does not replay one.
    """

    def __init__(self, grads: Sequence[torch.Tensor], masters: Sequence[torch.Tensor],
                 state: AdamState, params: Optional[Sequence[torch.Tensor]] = None,
                 weight_decay: Union[float, Sequence[float]] = 0.0,
                 lr_scale: Union[float, Sequence[float]] = 1.0):
        self.grads, self.masters, self.state = list(grads), list(masters), state
        self.params = None if params is None else list(params)
        self.device = device = state.device
        n = self.n = len(self.grads)
        sizes = [len(self.masters), len(state.numels)]
        if self.params is not None:
            sizes.append(len(self.params))
        if any(k != n for k in sizes):
            raise ValueError(f"{n} gradients, {len(self.masters)} masters, moments of "
                             f"{len(state.numels)} tensors"
                             + ("" if params is None else f", {len(self.params)} parameters"))
        decay, scale = _each(weight_decay, n, "weight_decay"), _each(lr_scale, n, "lr_scale")
        entries, spans = [], []

        def span(t, what):
            if t.numel():
                spans.append((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), what))

        small, block = state.bits == 8, abi.ZERO_ADAM_BLOCK
        m, v = state.m.data_ptr(), state.v.data_ptr()
        me, ve = (state.m_exp.data_ptr(), state.v_exp.data_ptr()) if small else (0, 0)
        width = 1 if small else 4
        for i in range(n):
            g, w, numel, at = self.grads[i], self.masters[i], state.numels[i], state.offsets[i]
            _check_tensor(g, f"gradient {i}", device)
            _check_tensor(w, f"master {i}", device)
            if w.dtype != torch.float32:
                raise TypeError(f"master {i} is {w.dtype}: float32 is supported")
            p = None if self.params is None else self.params[i]
            if p is not None:
                _check_tensor(p, f"parameter {i}", device)
            for t, what in ((g, "gradient"), (w, "master"), (p, "parameter")):
                if t is not None and t.numel() != numel:
                    raise ValueError(f"{what} {i} has {t.numel()} elements, its moments {numel}")
                if t is not None:
                    span(t, f"{what} {i}")
            entries.append(dict(grad=g, master=w, m=m + width * at, v=v + width * at,
                                m_exp=me + at // block, v_exp=ve + at // block, param=p,
                                numel=numel, weight_decay=decay[i], lr_scale=scale[i],
                                grad_dtype=DTYPES[g.dtype],
                                param_dtype=abi.ZERO_F32 if p is None else DTYPES[p.dtype],
                                moment_bits=state.bits))
        self._moments = _moments_of(state)
        for t, what in zip(self._moments, MOMENTS):
            if t is not None:
                span(t, what)
        _check_buffers_apart(spans)
        size = abi.zero_adam_table_bytes(n)
        self.table = torch.empty(size, dtype=torch.uint8, device=device)
        with on_device(device):
            self.list = abi.zero_tensors_adam_prepare(abi.adam_table(entries), n, self.table, size,
                                                      stream_of(device, None))
        self._read, self._cleared = None, False
        # filled by each step: making it anew would take a third of a short list's time
        self._args = abi.step_args(lr=0.0, beta1=0.0, beta2=0.0, eps=0.0, weight_decay=0.0,
                                   max_grad_norm=0.0, loss_scale=1.0, step=1)

    def _check_state(self):
        s, (m, v, m_exp, v_exp) = self.state, self._moments
        if s.m is not m or s.v is not v or s.m_exp is not m_exp or s.v_exp is not v_exp:
            raise RuntimeError("the state's buffers were exchanged: make a new list")

    def step(self, *, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
             step: int, loss_scale: float = 1.0, norm: Optional[GradList] = None,
             seed: Optional[int] = None, stream=None) -> None:
        """The update number ``step`` (from 1), of gradients that carry loss_scale.

        norm: the GradList whose last norm gives the clip coefficient, and the skip (nothing is
        written then; the next step has the same number).  seed: 32 bits for the rounding of
        8-bit moments, default the step's number."""
        self._check_state()
        result = None
        if norm is not None:
            if norm.device != self.device:
                raise ValueError(f"the norm is on {norm.device}, the list on {self.device}")
            if not norm._normed:
                raise RuntimeError("the clip coefficient comes from a norm of that list")
            result = norm._res
        args = self._args
        args.lr, args.beta1, args.beta2, args.eps = lr, beta1, beta2, eps
        args.loss_scale, args.step = loss_scale, step
        seed = (step if seed is None else seed) & 0xFFFFFFFF
        handle = stream_of(self.device, stream)
        with on_device(self.device):
            abi.zero_tensors_adam(self.list, args, seed, result, handle)

    def moments(self, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """The values of m and v, flat as in the state, zero between the tensors: the state's own
        buffers for 32 bits, for 8 bits bfloat16 buffers of the list (exact), written again by the
        next call."""
        self._check_state()
        if self.state.bits == 32:
            return self.state.m, self.state.v
        handle = stream_of(self.device, stream)
        with on_device(self.device):
            if not self._cleared:
                with torch.cuda.stream(stream):
                    if self._read is None:  # the memory is the call's stream's from the start
                        self._read = tuple(torch.empty(self.state.elements, dtype=torch.bfloat16,
                                                       device=self.device) for _ in range(2))
                    for t in self._read:
                        t.zero_()
                    # (a call that is captured clears them when it is replayed)
                    self._cleared = not torch.cuda.is_current_stream_capturing()
            m, v = self._read
            abi.zero_tensors_adam_moments(self.list, m, v, abi.ZERO_BF16, handle)
        return m, v
