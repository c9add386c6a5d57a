"""Gradient norm and clipping over a list of torch tensors.

PyTorch supplies the memory and the stream; the work runs in libzero_shard.so
(zero_tensors_norm, zero_tensors_clip).  A ``GradList`` holds the table of one
list, its workspace and its results; the tensors stay the caller's.
"""
from __future__ import annotations

import contextlib
from typing import NamedTuple, Optional, Sequence

import torch

from . import abi

DTYPES = {torch.float32: abi.ZERO_F32, torch.float16: abi.ZERO_F16, torch.bfloat16: abi.ZERO_BF16}


class GradNorm(NamedTuple):
    """Views of the list's device results, written when its stream has passed the call; the
    next call on the same list writes them again."""
    norm: torch.Tensor        # 0-dim float64
    clip_coef: torch.Tensor   # 0-dim float32
    overflow: torch.Tensor    # 0-dim int32: some element is inf or NaN
    skip: torch.Tensor        # 0-dim int32: overflow here or on another rank
    own_sq: torch.Tensor      # 0-dim float64: this list's squared norm, unscaled
    total_sq: torch.Tensor    # 0-dim float64: with the other ranks'
    tensor_sq: torch.Tensor   # [n] float64: each tensor's squared norm, unscaled


_HERE = contextlib.nullcontext()


def on_device(device):
    """A guard that makes `device` the current one; nothing to do where it is."""
    return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def stream_of(device, stream) -> int:
    """The handle of the given stream, or of the device's current one."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif stream.device_index != device.index:
        raise ValueError(f"the stream is on cuda:{stream.device_index}, the call on {device}")
    return stream.cuda_stream


def _check_tensor(t, what: str, device) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} is not a tensor")
    if t.dtype not in DTYPES:
        raise TypeError(f"{what} has dtype {t.dtype}; float32, float16 and bfloat16 are supported")
    if t.device.type != "cuda" or t.device != device:
        raise ValueError(f"{what} is on {t.device}, the list on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{what} is not contiguous")


def _check_apart(tensors, out) -> None:
    """No tensor or output may share memory with another entry's."""
    spans = []
    for i, (t, o) in enumerate(zip(tensors, out)):
        for x in (t,) if o is t else (t, o):
            if x.numel():
                spans.append((x.data_ptr(), x.data_ptr() + x.numel() * x.element_size(), i))
    reach, owner = 0, -1
    for start, end, i in sorted(spans):
        if start < reach and i != owner:  # an entry's own pair is checked by the library
            raise ValueError(f"tensors {min(i, owner)} and {max(i, owner)} share memory")
        if end > reach:
            reach, owner = end, i


class GradList:
    """A list of gradient tensors on one GPU, and where its clipped copies go.

    tensors: contiguous float32 / float16 / bfloat16 tensors, mixed as they come; out: tensors
    of the same sizes (any of the three types) that ``clip`` writes, or None to clip in place.
    Different tensors must not share memory.  The list is made for these tensors where they lie
    (1.6 us a tensor): gradients that a step makes anew, or whose memory is exchanged, need a
    new list.  Calls run on the given stream (default: the current stream of the list's device),
    which has to wait for the stream that the list was made on, as for any tensor; calls on one
    list must not overlap.  The list has to outlive their work, and the graphs that hold them.
    """

    def __init__(self, tensors: Sequence[torch.Tensor],
                 out: Optional[Sequence[torch.Tensor]] = None, device=None):
        self.tensors = list(tensors)
        self.out = self.tensors if out is None else list(out)
        if len(self.out) != len(self.tensors):
            raise ValueError(f"{len(self.out)} outputs for {len(self.tensors)} tensors")
        if device is not None:
            device = torch.device(device)
        elif self.tensors and isinstance(self.tensors[0], torch.Tensor):
            device = self.tensors[0].device
        else:
            device = torch.device("cuda", torch.cuda.current_device())
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        if device.type != "cuda":
            raise ValueError(f"device {device} is not a GPU")
        self.device = device
        entries = []
        for i, (t, o) in enumerate(zip(self.tensors, self.out)):
            _check_tensor(t, f"tensor {i}", device)
            if o is not t:
                _check_tensor(o, f"output {i}", device)
                if o.numel() != t.numel():
                    raise ValueError(f"output {i} has {o.numel()} elements, its tensor "
                                     f"{t.numel()}")
            entries.append((t, DTYPES[t.dtype], o, DTYPES[o.dtype], t.numel()))
        _check_apart(self.tensors, self.out)
        self.n = len(entries)
        self._normed = False
        self.table = abi.tensor_table(entries)
        self.ws_bytes = abi.zero_tensors_workspace_bytes(self.table, self.n)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
        self.res = torch.zeros(abi.RESULT_BYTES, dtype=torch.uint8, device=device)
        sq = torch.zeros(self.n, dtype=torch.float64, device=device)
        # addresses, resolved once
        self._sq, self._ws, self._res = sq.data_ptr(), self.ws.data_ptr(), self.res.data_ptr()
        d, f, w = (self.res.view(t) for t in (torch.float64, torch.float32, torch.int32))
        self.result = GradNorm(norm=d[4], clip_coef=f[10], overflow=w[11], skip=w[12],
                               own_sq=d[2], total_sq=d[3], tensor_sq=sq)

    def args(self, max_grad_norm: float, loss_scale: float, other_sq: float = 0.0,
             other_overflow: bool = False):
        return abi.step_args(lr=0.0, beta1=0.0, beta2=0.0, eps=0.0, weight_decay=0.0,
                             max_grad_norm=max_grad_norm, loss_scale=loss_scale, step=1,
                             other_sq=other_sq, other_overflow=other_overflow)

    def _on(self, stream):
        return on_device(self.device), stream_of(self.device, stream)

    def norm(self, max_grad_norm: float = 0.0, loss_scale: float = 1.0, other_sq: float = 0.0,
             other_overflow: bool = False, stream=None) -> GradNorm:
        """The norm of the tensors divided by loss_scale, the coefficient that clips it to
        max_grad_norm (<= 0: 1) and the skip decision."""
        guard, stream = self._on(stream)
        with guard:
            abi.zero_tensors_norm(self.table, self.n,
                                  self.args(max_grad_norm, loss_scale, other_sq, other_overflow),
                                  self._sq, self._ws, self.ws_bytes, self._res, stream)
        self._normed = True
        return self.result

    def clip(self, loss_scale: float = 1.0, out_scale: float = 1.0, stream=None) -> None:
        """out = tensor / loss_scale * out_scale * clip_coef of the last norm; nothing is
        written if that norm found inf or NaN."""
        if not self._normed:
            raise RuntimeError("clip takes its coefficient from a norm of this list")
        guard, stream = self._on(stream)
        with guard:
            abi.zero_tensors_clip(self.table, self.n, self.args(0.0, loss_scale), out_scale,
                                  self._res, stream)

    def norm_clip(self, max_grad_norm: float, loss_scale: float = 1.0, out_scale: float = 1.0,
                  other_sq: float = 0.0, other_overflow: bool = False, stream=None) -> GradNorm:
        """``norm`` then ``clip``, enqueued together."""
        guard, stream = self._on(stream)
        with guard:
            abi.zero_tensors_norm_clip(self.table, self.n,
                                       self.args(max_grad_norm, loss_scale, other_sq,
                                                 other_overflow),
                                       out_scale, self._sq, self._ws, self.ws_bytes, self._res,
                                       stream)
        self._normed = True
        return self.result
