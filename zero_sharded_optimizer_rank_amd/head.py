"""Loss of a language-model head and its gradients for torch tensors.

PyTorch supplies the memory and the stream; the work runs in libzero_shard.so
(zero_head_loss, zero_head_grad).  A ``LossHead`` holds the workspace and the
outputs for up to ``tokens`` tokens.  The loss keeps no logits; the gradients keep
those of one piece of the vocabulary at a time, in 16 bits and at most 1 GiB up to
131072 tokens.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import abi
from .tensors import on_device, stream_of

DTYPES = {torch.float16: abi.ZERO_F16, torch.bfloat16: abi.ZERO_BF16}


class HeadLoss(NamedTuple):
    """The results of one call.  They are the head's own buffers, written when the stream has
    passed the call; the next call on the same head writes them again."""
    loss: torch.Tensor        # 0-dim float32: mean (or sum) over the valid tokens, unscaled
    loss_sum: torch.Tensor    # 0-dim float64
    token_loss: torch.Tensor  # [T] float32, 0 for ignored tokens
    lse: torch.Tensor         # [T] float32, 0 for ignored tokens
    valid: torch.Tensor       # 0-dim int64: tokens with a label
    bad: torch.Tensor         # 0-dim int64: labels >= vocab (loss and gradients are then NaN)
    dx: Optional[torch.Tensor] = None  # [T, H], type of x: gradient times loss_scale
    dw: Optional[torch.Tensor] = None  # [V, H]


class LossHead:
    """Softmax cross entropy of x @ w.T against labels, for up to ``tokens`` tokens.

    dtype: torch.float16 or torch.bfloat16, the type of x [T, hidden] and w [vocab, hidden];
    rows may be strided (up to 2^20 elements apart), elements of a row must be adjacent.
    labels: int64 [T]; a negative label ignores its token.  grad=False keeps the smaller
    workspace of the loss alone.  Calls run on the given stream (default: the current stream of
    the device), which has to wait for the stream that the head was made on, as for any tensor,
    and must not overlap on one head.  The head has to outlive the work of its calls, and the
    graphs that hold them.
    """

    def __init__(self, tokens: int, hidden: int, vocab: int, dtype: torch.dtype, device="cuda:0",
                 grad: bool = True):
        if dtype not in DTYPES:
            raise TypeError(f"dtype {dtype}: float16 and bfloat16 are supported")
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError(f"device {self.device} is not a GPU")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.tokens, self.hidden, self.vocab, self.dtype = tokens, hidden, vocab, dtype
        self.has_grad = grad
        head = abi.zero_head_t(tokens, hidden, vocab, 0, hidden, 0, hidden, 0, DTYPES[dtype], 1,
                               1.0)
        need = abi.zero_head_workspace_bytes(head, grad)
        if need == 0:
            raise ValueError(f"sizes out of range: tokens {tokens}, hidden {hidden}, "
                             f"vocab {vocab}")
        dev = self.device
        self.ws = torch.empty(need, dtype=torch.uint8, device=dev)
        self.res = torch.zeros(abi.LOSS_RESULT_BYTES, dtype=torch.uint8, device=dev)
        self._token_loss = torch.empty(tokens, dtype=torch.float32, device=dev)
        self._lse = torch.empty(tokens, dtype=torch.float32, device=dev)
        self._dx = torch.empty(tokens, hidden, dtype=dtype, device=dev) if grad else None
        self._dw = None  # made by the first loss_grad that is not given one
        d, f, q = (self.res.view(t) for t in (torch.float64, torch.float32, torch.int64))
        self._loss_sum, self._loss, self._valid, self._bad = d[0], f[2], q[2], q[3]

    def _matrix(self, t, rows, what):
        if not isinstance(t, torch.Tensor) or t.dim() != 2 or tuple(t.shape) != (rows, self.hidden):
            raise ValueError(f"{what} must be a [{rows}, {self.hidden}] tensor")
        if t.device != self.device:
            raise ValueError(f"{what} is on {t.device}, the head on {self.device}")
        if self.hidden > 1 and t.stride(1) != 1:
            raise ValueError(f"the elements of a row of {what} must be adjacent")
        ld = t.stride(0) if rows > 1 else self.hidden  # one row has no next
        if ld < self.hidden:
            raise ValueError(f"the rows of {what} overlap")
        return ld

    def _head(self, x, w, labels, mean, loss_scale):
        if not isinstance(labels, torch.Tensor) or labels.dtype != torch.int64 \
                or labels.dim() != 1 or not labels.is_contiguous():
            raise ValueError("labels must be a contiguous int64 vector")
        if labels.device != self.device:
            raise ValueError(f"labels are on {labels.device}, the head on {self.device}")
        t = labels.numel()
        if t > self.tokens:
            raise ValueError(f"{t} tokens on a head for {self.tokens}")
        ldx, ldw = self._matrix(x, t, "x"), self._matrix(w, self.vocab, "w")
        if x.dtype != self.dtype or w.dtype != self.dtype:
            raise TypeError(f"x is {x.dtype}, w is {w.dtype}, the head {self.dtype}")
        return abi.zero_head_t(t, self.hidden, self.vocab, x.data_ptr(), ldx, w.data_ptr(), ldw,
                               labels.data_ptr(), DTYPES[self.dtype], 1 if mean else 0,
                               loss_scale)

    def _workspace(self, head, grad, stream):
        # rows of w that do not start on 16-byte boundaries may take a copy in the workspace
        if (head.w | head.ldw * 2 | self.hidden * 2) % 16 \
                and abi.zero_head_workspace_bytes(head, grad) > self.ws.numel():
            # grown once, for every later call; a graph captured before holds the old one's
            # address, so that stays too
            full = abi.zero_head_t.from_buffer_copy(head)
            full.tokens = self.tokens
            self._first_ws = self.ws
            with torch.cuda.stream(stream):  # the memory is the call's stream's from the start
                self.ws = torch.empty(abi.zero_head_workspace_bytes(full, self.has_grad),
                                      dtype=torch.uint8, device=self.device)
        return self.ws

    def _result(self, t, **kw):
        return HeadLoss(self._loss, self._loss_sum, self._token_loss[:t], self._lse[:t],
                        self._valid, self._bad, **kw)

    def loss(self, x, w, labels, mean: bool = True, stream=None) -> HeadLoss:
        """The loss alone."""
        head = self._head(x, w, labels, mean, 1.0)
        handle = stream_of(self.device, stream)
        with on_device(self.device):
            ws = self._workspace(head, False, stream)
            abi.zero_head_loss(head, self._token_loss, self._lse, ws, ws.numel(), self.res,
                               handle)
        return self._result(head.tokens)

    def _grads(self, t, dx, dw, accumulate, stream):
        if not self.has_grad:
            raise ValueError("the head was made with grad=False")
        if dx is None:
            dx = self._dx[:t]
        if dw is None:
            if accumulate:
                raise ValueError("accumulate needs a dw to add to")
            if self._dw is None:
                with torch.cuda.stream(stream):  # as a grown workspace
                    self._dw = torch.empty(self.vocab, self.hidden, dtype=self.dtype,
                                           device=self.device)
            dw = self._dw
        lddx, lddw = self._matrix(dx, t, "dx"), self._matrix(dw, self.vocab, "dw")
        if dx.dtype != self.dtype or dw.dtype not in (self.dtype, torch.float32):
            raise TypeError(f"dx is {dx.dtype}, dw is {dw.dtype}, the head {self.dtype}")
        wt = abi.ZERO_F32 if dw.dtype == torch.float32 else DTYPES[self.dtype]
        return dx, dw, abi.zero_head_grads_t(dx.data_ptr(), lddx, dw.data_ptr(), lddw, wt,
                                             1 if accumulate else 0)

    def loss_grad(self, x, w, labels, mean: bool = True, loss_scale: float = 1.0, dx=None,
                  dw=None, accumulate: bool = False, stream=None) -> HeadLoss:
        """The loss, and its gradients times loss_scale.  dx [T, H] and dw [V, H] may be given
        (dw in the head's type or float32, e.g. the weight's part of a flat contribution row);
        accumulate adds to dw."""
        head = self._head(x, w, labels, mean, loss_scale)
        handle = stream_of(self.device, stream)
        dx, dw, grads = self._grads(head.tokens, dx, dw, accumulate, stream)
        with on_device(self.device):
            ws = self._workspace(head, True, stream)
            abi.zero_head_loss_grad(head, self._token_loss, self._lse, grads, ws, ws.numel(),
                                    self.res, handle)
        return self._result(head.tokens, dx=dx, dw=dw)

    def grad(self, x, w, labels, lse, mean: bool = True, loss_scale: float = 1.0, dx=None,
             dw=None, accumulate: bool = False, stream=None):
        """The gradients alone, (dx, dw), from the lse that ``loss`` returned for the same
        inputs."""
        head = self._head(x, w, labels, mean, loss_scale)
        if not isinstance(lse, torch.Tensor) or lse.dtype != torch.float32 \
                or lse.device != self.device or not lse.is_contiguous() \
                or lse.numel() != head.tokens:
            raise ValueError(f"lse must be a contiguous float32 vector of {head.tokens}")
        handle = stream_of(self.device, stream)
        dx, dw, grads = self._grads(head.tokens, dx, dw, accumulate, stream)
        with on_device(self.device):
            ws = self._workspace(head, True, stream)
            abi.zero_head_grad(head, lse, grads, ws, ws.numel(), handle)
        return dx, dw
