"""Gated feed-forward block and its gradients for torch tensors.

PyTorch supplies the memory and the stream; the work runs in libzero_shard.so
(zero_ffn_forward, zero_ffn_backward).  A ``GatedFFN`` holds the workspace and the
outputs for up to ``tokens`` tokens of blocks of one size; the weights stay the
caller's, so that one serves all layers.
"""
from __future__ import annotations

import warnings
from typing import NamedTuple, Optional

import torch

from . import abi
from .head import DTYPES
from .tensors import on_device, stream_of

ACTIVATIONS = {"silu": abi.ZERO_ACT_SILU, "gelu": abi.ZERO_ACT_GELU,
               "gelu_tanh": abi.ZERO_ACT_GELU_TANH, "relu": abi.ZERO_ACT_RELU}


class FFNSaved(NamedTuple):
    """What the gradients need of a forward pass, columns padded to a multiple of 8.  act and
    slope hold the upper 16 bits of fp32 values (bfloat16 patterns, whatever the block's type),
    low the next 8 of both: 24 bits each."""
    act: torch.Tensor     # act(x @ w_gate.T)
    slope: torch.Tensor   # (x @ w_up.T) * act'(x @ w_gate.T)
    low: torch.Tensor
    h: torch.Tensor       # act * (x @ w_up.T), in the block's type


class FFNOut(NamedTuple):
    y: torch.Tensor                  # [T, H]
    saved: Optional[FFNSaved]        # if asked for


class FFNGrads(NamedTuple):
    dx: Optional[torch.Tensor]       # [T, H], type of x
    dw_gate: Optional[torch.Tensor]  # [F, H]
    dw_up: Optional[torch.Tensor]    # [F, H]
    dw_down: Optional[torch.Tensor]  # [H, F]


class GatedFFN:
    """y = (act(x @ w_gate.T) * (x @ w_up.T)) @ w_down.T for up to ``tokens`` tokens.

    dtype: torch.float16 or torch.bfloat16, the type of x [T, hidden], w_gate and w_up [inner,
    hidden] and w_down [hidden, inner]; rows may be strided (up to 2^20 elements apart), elements
    of a row must be adjacent.  act: "silu", "gelu", "gelu_tanh" or "relu".  grad=False keeps the
    smaller workspace of the forward pass alone.  Outputs that are not given are the block's own
    buffers, which the next call writes again.  Calls run on the given stream (default: the
    current stream of the device), which has to wait for the stream that the block was made on, as
    for any tensor, and must not overlap on one block.  The block has to outlive the work of its
    calls, and the graphs that hold them.  Outputs carry no autograd graph: the gradients are what
    ``backward`` returns, and a forward pass of inputs that require gradients warns where autograd
    is on.
    """

    def __init__(self, tokens: int, hidden: int, inner: int, dtype: torch.dtype,
                 act: str = "silu", device="cuda:0", grad: bool = True):
        if dtype not in DTYPES:
            raise TypeError(f"dtype {dtype}: float16 and bfloat16 are supported")
        if act not in ACTIVATIONS:
            raise ValueError(f"activation {act!r}: one of {', '.join(ACTIVATIONS)}")
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError(f"device {self.device} is not a GPU")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.tokens, self.hidden, self.inner = tokens, hidden, inner
        self.dtype, self.act, self.has_grad = dtype, act, grad
        self._pad = -(-inner // 8) * 8
        need = self._need(self._sizes(tokens), grad)
        if need == 0:
            raise ValueError(f"sizes out of range: tokens {tokens}, hidden {hidden}, "
                             f"inner {inner}")
        dev = self.device
        self.ws = torch.empty(need, dtype=torch.uint8, device=dev)
        self._y = torch.empty(tokens, hidden, dtype=dtype, device=dev)
        self._saved = None  # made by the first save=True: 8 bytes an element of tokens x inner
        self._dx = torch.empty(tokens, hidden, dtype=dtype, device=dev) if grad else None
        self._dw = {}  # made by the first backward that is not given one
        self._needs = {}  # workspace by the matrices whose rows lie between 16-byte boundaries

    def _sizes(self, tokens):
        h, f = self.hidden, self.inner
        return abi.zero_ffn_t(tokens, h, f, 0, h, 0, h, 0, h, 0, f, DTYPES[self.dtype],
                              ACTIVATIONS[self.act])

    def _grads_t(self, dy=0, lddy=None):
        h, f = self.hidden, self.inner
        return abi.zero_ffn_grads_t(dy, h if lddy is None else lddy, 0, h, 0, h, 0, h, 0, f,
                                    DTYPES[self.dtype], 0)

    def _need(self, ffn, grad, grads=None):
        need = abi.zero_ffn_workspace_bytes(ffn)
        if need and grad:
            need = max(need, abi.zero_ffn_workspace_bytes(ffn, grads or self._grads_t()))
        return need

    def new_saved(self, tokens: Optional[int] = None) -> FFNSaved:
        """Buffers for a forward pass to keep what its gradients need: one set a layer whose
        gradients are still to come."""
        tokens = self.tokens if tokens is None else tokens
        return FFNSaved(*(torch.empty(tokens, self._pad, dtype=self.dtype, device=self.device)
                          for _ in range(4)))

    def _matrix(self, t, rows, cols, what, types=None):
        if not isinstance(t, torch.Tensor) or t.dim() != 2 or tuple(t.shape) != (rows, cols):
            raise ValueError(f"{what} must be a [{rows}, {cols}] tensor")
        if t.device != self.device:
            raise ValueError(f"{what} is on {t.device}, the block on {self.device}")
        if t.dtype not in (types or (self.dtype,)):
            raise TypeError(f"{what} is {t.dtype}, the block {self.dtype}")
        if cols > 1 and t.stride(1) != 1:
            raise ValueError(f"the elements of a row of {what} must be adjacent")
        ld = t.stride(0) if rows > 1 else cols  # one row has no next
        if ld < cols:
            raise ValueError(f"the rows of {what} overlap")
        return ld

    def _ffn(self, x, w_gate, w_up, w_down):
        h, f = self.hidden, self.inner
        t = x.shape[0] if isinstance(x, torch.Tensor) and x.dim() == 2 else -1
        if t > self.tokens:
            raise ValueError(f"{t} tokens on a block for {self.tokens}")
        ldx = self._matrix(x, t, h, "x")
        lg, lu = self._matrix(w_gate, f, h, "w_gate"), self._matrix(w_up, f, h, "w_up")
        ld = self._matrix(w_down, h, f, "w_down")
        return abi.zero_ffn_t(t, h, f, x.data_ptr(), ldx, w_gate.data_ptr(), lg, w_up.data_ptr(),
                              lu, w_down.data_ptr(), ld, DTYPES[self.dtype],
                              ACTIVATIONS[self.act])

    def _saved_t(self, saved, t):
        if not isinstance(saved, FFNSaved):
            raise TypeError("saved must be an FFNSaved")
        lds = set()
        for b, what in zip(saved, saved._fields):
            if not isinstance(b, torch.Tensor) or b.dim() != 2 or b.shape[0] < t:
                raise ValueError(f"saved.{what} must be a [{t}, {self._pad}] tensor")
            lds.add(self._matrix(b[:t], t, self._pad, "saved." + what))
        if len(lds) > 1:
            raise ValueError("the rows of act, slope, low and h lie differently")
        return abi.zero_ffn_saved_t(*(b.data_ptr() for b in saved), lds.pop())

    def _workspace(self, ffn, grads, stream):
        # rows that do not start on 16-byte boundaries take copies in the workspace
        rows = [(ffn.x, ffn.ldx), (ffn.w_gate, ffn.ld_gate), (ffn.w_up, ffn.ld_up),
                (ffn.w_down, ffn.ld_down)]
        if grads is not None:
            rows.append((grads.dy, grads.lddy))
        # (an empty batch has no address)
        lies = tuple([((p or 0) | 2 * ld) % 16 != 0 for p, ld in rows])
        if any(lies):
            # grown for every later batch that lies so; graphs captured before hold the old
            # one's address, so that stays too
            need = self._needs.get(lies)
            if need is None:  # sized once: all smaller batches are looked at
                full = abi.zero_ffn_t.from_buffer_copy(ffn)
                full.tokens = self.tokens
                need = self._needs[lies] = self._need(full, grads is not None, grads)
            if need > self.ws.numel():
                self._old_ws = getattr(self, "_old_ws", []) + [self.ws]
                with torch.cuda.stream(stream):  # the memory is the call's stream's from the start
                    self.ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        return self.ws

    def forward(self, x, w_gate, w_up, w_down, y=None, save=False, stream=None) -> FFNOut:
        """The block's output; save=True, or an FFNSaved, keeps what ``backward`` needs."""
        ffn = self._ffn(x, w_gate, w_up, w_down)
        if torch.is_grad_enabled() and (x.requires_grad or w_gate.requires_grad
                                        or w_up.requires_grad or w_down.requires_grad):
            warnings.warn("autograd does not record the block: call its backward (under "
                          "torch.no_grad() this is not said)", stacklevel=2)
        t = ffn.tokens
        y = self._y[:t] if y is None else y
        ldy = self._matrix(y, t, self.hidden, "y")
        handle = stream_of(self.device, stream)
        saved = saved_t = None
        if save is not False and save is not None:
            if save is True and not self.has_grad:
                raise ValueError("the block was made with grad=False")
            if save is True and self._saved is None:
                with torch.cuda.stream(stream):  # as a grown workspace
                    self._saved = self.new_saved()
            saved = FFNSaved(*(b[:t] for b in self._saved)) if save is True else save
            saved_t = self._saved_t(saved, t)
        with on_device(self.device):
            ws = self._workspace(ffn, None, stream)
            abi.zero_ffn_forward(ffn, y, ldy, saved_t, ws, ws.numel(), handle)
        return FFNOut(y, saved)

    def backward(self, dy, x, w_gate, w_up, w_down, saved: FFNSaved, dx=None, dw_gate=None,
                 dw_up=None, dw_down=None, accumulate: bool = False, need_dx: bool = True,
                 need_dw: bool = True, stream=None) -> FFNGrads:
        """The gradients, from what ``forward`` kept for the same x and weights.  They carry the
        loss scale that dy carries; in float16 it has to hold them, and the gradients of both
        projections, between 2^-14 (below, steps are 2^-24) and 65504.  dw_* may be given, all of
        one type, the block's or float32 (e.g. pieces of a flat contribution row); accumulate adds
        to them."""
        if not self.has_grad:
            raise ValueError("the block was made with grad=False")
        ffn = self._ffn(x, w_gate, w_up, w_down)
        t, h, f = ffn.tokens, self.hidden, self.inner
        saved_t = self._saved_t(saved, t)
        grads = self._grads_t(dy.data_ptr() if isinstance(dy, torch.Tensor) else 0,
                              self._matrix(dy, t, h, "dy"))
        handle = stream_of(self.device, stream)
        if need_dx:
            dx = self._dx[:t] if dx is None else dx
            grads.dx, grads.lddx = dx.data_ptr(), self._matrix(dx, t, h, "dx")
        given = {"dw_gate": dw_gate, "dw_up": dw_up, "dw_down": dw_down}
        out = dict.fromkeys(given)
        if need_dw:
            if accumulate and any(w is None for w in given.values()):
                raise ValueError("accumulate needs the dw_* to add to")
            for name, w in given.items():
                shape = (h, f) if name == "dw_down" else (f, h)
                if w is None:
                    if name not in self._dw:
                        with torch.cuda.stream(stream):  # as a grown workspace
                            self._dw[name] = torch.empty(*shape, dtype=self.dtype,
                                                         device=self.device)
                    w = self._dw[name]
                ld = self._matrix(w, *shape, name, (self.dtype, torch.float32))
                setattr(grads, name, w.data_ptr())
                setattr(grads, "ld" + name, ld)
                out[name] = w
            if len({w.dtype for w in out.values()}) > 1:
                raise TypeError("dw_gate, dw_up and dw_down must have one type")
            if out["dw_gate"].dtype == torch.float32:
                grads.dw_dtype = abi.ZERO_F32
        grads.accumulate = 1 if accumulate else 0
        with on_device(self.device):
            ws = self._workspace(ffn, grads, stream)
            abi.zero_ffn_backward(ffn, saved_t, grads, ws, ws.numel(), handle)
        return FFNGrads(dx=dx if need_dx else None, **out)
