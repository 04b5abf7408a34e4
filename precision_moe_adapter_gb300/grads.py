"""A list of gradients with their global norm and clipping, driven through the C
ABI.

The list (pointers and sizes) lies on the device, made once for buffers that
stay: the adapter gradients of every layer, a head's dW.  Every computation
happens in libpmoe's kernels; this module allocates, checks and passes
pointers.
"""
from __future__ import annotations

import torch

from . import pmoe
from .layer import check_cuda, check_current, check_tensor

_DTYPES = {torch.float32: pmoe.GRAD_F32, torch.bfloat16: pmoe.GRAD_BF16}


class GradList:
    """Gradients (f32 or bf16, any shapes, dense, 16-byte aligned) on one device.

    ``out`` holds the tensors that ``clip`` writes, shaped and typed like the
    gradients; None clips in place.  Calls on one list share its workspace and
    must be ordered (one stream, or events); they are made on torch's current
    device, which must be the list's.  The tensors are kept alive."""

    def __init__(self, grads, out=None, device=None):
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        if len(self.out) != len(self.grads):
            raise ValueError(f"out: {len(self.out)} tensors for {len(self.grads)} gradients")
        if device is None:
            device = self.grads[0].device if self.grads else torch.device("cuda", torch.cuda.current_device())
        self.device = torch.device(device)
        for i, (g, o) in enumerate(zip(self.grads, self.out)):
            check_tensor(f"gradient {i}", g, tuple(_DTYPES), g.shape, self.device)
            check_tensor(f"out {i}", o, (g.dtype,), g.shape, self.device)
        check_current(self.device)
        self._list, table = pmoe.grad_list_fill(
            [(g.data_ptr(), o.data_ptr(), g.numel(), _DTYPES[g.dtype])
             for g, o in zip(self.grads, self.out)])
        self._table = torch.frombuffer(bytearray(table), dtype=torch.uint8).to(self.device)
        self._list.table = self._table.data_ptr()
        self._ws = torch.zeros(pmoe.grad_ws_bytes(), dtype=torch.uint8, device=self.device)

    def _norm_ok(self, norm):
        check_current(self.device)
        check_tensor("norm", norm, (torch.float32,), (1,), self.device)
        check_cuda(self.device)

    def norm(self, norm):
        """norm (f32 [1]): the root of the sum of all squares."""
        self._norm_ok(norm)
        pmoe.grad_norm(self._list, norm, self._ws)

    def clip(self, max_norm: float, norm):
        """The norm, and every gradient times min(1, max_norm / (norm + 1e-6))."""
        self._norm_ok(norm)
        pmoe.grad_clip(self._list, float(max_norm), norm, self._ws)
