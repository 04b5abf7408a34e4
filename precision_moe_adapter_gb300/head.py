"""The vocabulary head of a training step, driven through the C ABI.

Holds the head's weights (BF16 [V, d]), the workspaces and the sizes, and
runs the two losses on hidden states X (BF16 [T, d]):

    logprob / logprob_backward   token log-probabilities
    distill / distill_backward   distance to a teacher's top K logits

Every computation happens in libpmoe's kernels; this module allocates,
checks shapes, types and layout (the C ABI sees bare pointers) and passes
pointers.  BF16 tensors may be torch.bfloat16 or int16 bits.
"""
from __future__ import annotations

import torch

from . import pmoe
from .layer import check_current
from .layer import check_tensor as _check

_BF16 = (torch.bfloat16, torch.int16)


class DeviceHead:
    """A head W (BF16 [V, d]) for calls of exactly T tokens.

    ``K`` is the number of teacher entries per token (distillation), ``scale``
    the factor of every logit (1 / temperature).  ``backward=False`` leaves
    out the backward's workspace.  Calls on one head share its workspaces and
    must be ordered (one stream, or events); they are made on torch's current
    device, which must be W's."""

    def __init__(self, W: torch.Tensor, T: int, K: int = 0, scale: float = 1.0,
                 backward: bool = True):
        if W.dim() != 2:
            raise ValueError(f"W: shape {tuple(W.shape)}, expected [V, d]")
        _check("W", W, _BF16, W.shape, W.device)
        check_current(W.device)
        self.W, self.scale, self.device = W, float(scale), W.device
        V, d = W.shape
        self.dims = pmoe.head_dims(T, d, V, K)
        self._ws = {}
        for op in (pmoe.HEAD_FORWARD, pmoe.HEAD_BACKWARD) if backward else (pmoe.HEAD_FORWARD,):
            n = pmoe.head_workspace_bytes(self.dims, op)
            if n == 0:
                raise ValueError(f"unsupported head: T={T}, d={d}, V={V}, K={K}")
            self._ws[op] = torch.empty(n, dtype=torch.uint8, device=self.device)
            pmoe.moe_clear_status(self._ws[op])

    def _in(self, X, **f32):
        h = self.dims
        check_current(self.device)
        _check("X", X, _BF16, (h.T, h.d), self.device)
        for name, t in f32.items():
            _check(name, t, (torch.float32,), (h.T,), self.device)

    def _targets(self, target):
        _check("target", target, (torch.int32,), (self.dims.T,), self.device)

    def _teacher(self, t_idx, t_logits):
        shape = (self.dims.T, self.dims.K)
        _check("t_idx", t_idx, (torch.int32,), shape, self.device)
        _check("t_logits", t_logits, (torch.float32,), shape, self.device)

    def _grads(self, dX, dW):
        h = self.dims
        if dX is not None:
            _check("dX", dX, _BF16, (h.T, h.d), self.device)
        if dW is not None:
            _check("dW", dW, _BF16, (h.V, h.d), self.device)
        if pmoe.HEAD_BACKWARD not in self._ws:
            raise RuntimeError("the head was made with backward=False")
        return self._ws[pmoe.HEAD_BACKWARD]

    def logprob(self, X, target, logp, lse):
        """logp, lse (f32 [T]) of the targets (int32 [T], negative: ignored)."""
        self._in(X, logp=logp, lse=lse)
        self._targets(target)
        pmoe.head_logprob_forward(self.dims, X, self.W, self.scale, target, logp, lse,
                                  self._ws[pmoe.HEAD_FORWARD])

    def logprob_backward(self, X, target, lse, g, dX, dW=None):
        """dX (and dW unless None: a frozen head) for g = dL/dlogp."""
        self._in(X, lse=lse, g=g)
        self._targets(target)
        ws = self._grads(dX, dW)
        pmoe.head_logprob_backward(self.dims, X, self.W, self.scale, target, lse, g, dX, dW, ws)

    def distill(self, X, t_idx, t_logits, loss, lse):
        """loss, lse (f32 [T]) against the teacher's entries ([T, K])."""
        self._in(X, loss=loss, lse=lse)
        self._teacher(t_idx, t_logits)
        pmoe.head_distill_forward(self.dims, X, self.W, self.scale, t_idx, t_logits, loss, lse,
                                  self._ws[pmoe.HEAD_FORWARD])

    def distill_backward(self, X, t_idx, t_logits, lse, g, dX, dW=None):
        """dX (and dW unless None: a frozen head) for g = dL/dloss."""
        self._in(X, lse=lse, g=g)
        self._teacher(t_idx, t_logits)
        ws = self._grads(dX, dW)
        pmoe.head_distill_backward(self.dims, X, self.W, self.scale, t_idx, t_logits, lse, g, dX,
                                   dW, ws)

    def status(self) -> int:
        """First device error recorded by the calls so far (synchronizes)."""
        check_current(self.device)
        s = pmoe.PMOE_OK
        for ws in self._ws.values():
            s = s or pmoe.moe_query_status(ws)
        return s
