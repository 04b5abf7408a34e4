"""A frozen FP8 projection with 8-bit activations, driven through the C ABI.

Holds the weight (E4M3 [N, K], FP32 scales per [128, 128]), its transpose for
the gradient, the orthogonal adapter on its input and the workspace:

    forward    Y = bf16(Q(x~) W^T),  x~ = bf16(X blockdiag(R))
    backward   dX and, with an adapter, dR of an upstream dY

Every computation happens in libpmoe's kernels; this module allocates, checks
shapes, types and layout (the C ABI sees bare pointers) and passes pointers.
BF16 tensors may be torch.bfloat16 or int16 bits, E4M3 ones torch.float8_e4m3fn
or uint8 codes.
"""
from __future__ import annotations

import torch

from . import pmoe
from .layer import check_cuda, check_current, check_tensor

_BF16 = (torch.bfloat16, torch.int16)
_E4M3 = (torch.float8_e4m3fn, torch.uint8)


class DeviceLinearW8A8:
    """A weight q (E4M3 [N, K]), s (f32 [ceil(N/128), ceil(K/128)]) for calls of up
    to ``rows`` rows.

    ``R`` (BF16 [K/b, b, b]) is the adapter, or None; ``pow2`` makes the
    activations' scales powers of two; ``backward=False`` leaves out the transposed
    weight.  A row's results may differ in their last bit with the number of rows in
    the call; ``one_order=True`` makes them the same in any call, which takes longer
    for few rows.  Calls on one layer share its workspace and must be ordered (one
    stream, or events); they are made on torch's current device, which must be
    the weight's."""

    def __init__(self, q: torch.Tensor, s: torch.Tensor, rows: int, R: torch.Tensor | None = None,
                 pow2: bool = False, backward: bool = True, one_order: bool = False):
        if q.dim() != 2:
            raise ValueError(f"q: shape {tuple(q.shape)}, expected [N, K]")
        N, K = q.shape
        NB, KB = -(-N // 128), -(-K // 128)
        check_tensor("q", q, _E4M3, q.shape, q.device)
        check_tensor("s", s, (torch.float32,), (NB, KB), q.device)
        self.block = 0
        if R is not None:
            if R.dim() != 3 or R.shape[1] != R.shape[2]:
                raise ValueError(f"R: shape {tuple(R.shape)}, expected [K/b, b, b]")
            self.block = R.shape[1]
            check_tensor("R", R, _BF16, (K // max(self.block, 1), self.block, self.block), q.device)
        check_current(q.device)
        self.q, self.s, self.R, self.N, self.K = q, s, R, N, K
        self.rows, self.pow2, self.device = int(rows), bool(pow2), q.device
        self.one_order = bool(one_order)
        n = pmoe.dense_w8a8_ws_bytes(self.rows, N, K, R is not None)
        if n == 0:
            raise ValueError(f"unsupported layer: rows={rows}, N={N}, K={K}")
        self._ws = torch.empty(n, dtype=torch.uint8, device=self.device)
        pmoe.moe_clear_status(self._ws)
        self.qt = self.st = None
        if backward:
            self.qt = torch.empty((K, N), dtype=q.dtype, device=self.device)
            self.st = torch.empty((KB, NB), dtype=torch.float32, device=self.device)
            pmoe.fp8_transpose(N, K, q, s, self.qt, self.st)

    def _rows(self, name, x, cols):
        check_current(self.device)
        if x.dim() != 2 or x.shape[0] > self.rows:
            raise ValueError(f"{name}: shape {tuple(x.shape)}, expected at most {self.rows} rows of {cols}")
        check_tensor(name, x, _BF16, (x.shape[0], cols), self.device)
        return x.shape[0]

    def forward(self, X, Y):
        """Y (BF16 [rows, N]) of X (BF16 [rows, K])."""
        n = self._rows("X", X, self.K)
        check_tensor("Y", Y, _BF16, (n, self.N), self.device)
        check_cuda(self.device)
        pmoe.dense_w8a8_forward(self.q, self.s, self.N, self.K, self.block, self.R, n, X, Y, self._ws,
                                self.pow2, one_order=self.one_order)

    def backward(self, X, dY, dX, dR=None):
        """dX (BF16 [rows, K]) and, with an adapter, dR (f32, shaped like R, over-
        written) of dY (BF16 [rows, N]); X is only looked at with an adapter."""
        if self.qt is None:
            raise RuntimeError("the layer was made with backward=False")
        n = self._rows("dY", dY, self.N)
        check_tensor("dX", dX, _BF16, (n, self.K), self.device)
        if self.R is not None:
            check_tensor("X", X, _BF16, (n, self.K), self.device)
            if dR is None:
                raise ValueError("dR is missing: the layer has an adapter")
            check_tensor("dR", dR, (torch.float32,), tuple(self.R.shape), self.device)
        elif dR is not None:
            raise ValueError("dR: the layer has no adapter")
        check_cuda(self.device)
        pmoe.dense_w8a8_backward(self.qt, self.st, self.N, self.K, self.block, self.R, n, X, dY, dX, dR,
                                 self._ws, self.pow2, one_order=self.one_order)

    def status(self) -> int:
        """First device error recorded by the calls so far (synchronizes)."""
        check_current(self.device)
        return pmoe.moe_query_status(self._ws)
