"""A device-resident MoE layer driven through the C ABI.

Holds the frozen quantized experts, the router and the adapter as torch
device tensors (torch is only the allocator here), the routing buffers and
the workspaces, and runs one step of the layer:

    moe_route -> moe_permute -> moe_chunked_forward -> moe_backward_data

and the router's training side: moe_balance_forward, moe_route_backward.

Every computation happens in libpmoe's kernels; this module only allocates
and passes pointers.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch

from . import pmoe
from .inputs import LayerConfig


def check_tensor(name, t, dtypes, shape, device):
    """Raises unless t is a dense tensor of one of the dtypes, of the shape, on
    the device (the C ABI sees bare pointers)."""
    if t.dtype in dtypes and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    raise ValueError(f"{name}: must be contiguous")


def check_current(device):
    """Raises unless the CUDA device is torch's current one, on which (and on
    whose stream) the library launches."""
    index = device.index   # (None on the CPU)
    if index is not None and torch.cuda.current_device() != index:
        raise RuntimeError(f"the current device is cuda:{torch.cuda.current_device()}, the tensors are "
                           f"on {device}: call under torch.cuda.device({index})")


def _dev(a, device) -> torch.Tensor:
    if isinstance(a, torch.Tensor):   # already a tensor (e.g. drawn on the device)
        return a.to(device)
    t = torch.from_numpy(np.ascontiguousarray(a))
    if t.dtype == torch.uint16:
        t = t.view(torch.int16)
    return t.to(device)


@dataclass
class Routing:
    idx: torch.Tensor
    w: torch.Tensor
    counts: torch.Tensor
    offsets: torch.Tensor
    perm: torch.Tensor
    inv_perm: torch.Tensor
    active: torch.Tensor
    num_active: torch.Tensor

    def c(self) -> pmoe.Routing:
        return pmoe.routing(self.idx, self.w, self.counts, self.offsets, self.perm, self.inv_perm,
                            self.active, self.num_active)


@dataclass
class Balance:
    """The balance loss of each packed sequence and what its gradient needs."""
    counts: torch.Tensor      # int32 [nseq, E]
    ntok: torch.Tensor        # int32 [nseq]
    pmean: torch.Tensor       # f32 [nseq, E]
    loss: torch.Tensor        # f32 [nseq]


class DeviceLayer:
    """Frozen experts + router + adapter of one layer on a CUDA device.

    ``S_up`` / ``S_down`` (f32 [n_sets, dim/b, b, b], n_sets = E or 1) are
    the adapter's skew parameters; the rotations R = Cayley(S) are computed
    on the device by ``adapter_cayley``.  ``R_up`` / ``R_down`` (BF16 bits)
    may be given instead.  Passing neither disables the adapter."""

    def __init__(self, cfg: LayerConfig, w13, s13, w2, s2, Wr=None, bias=None, S_up=None,
                 S_down=None, R_up=None, R_down=None, device="cuda"):
        self.cfg = cfg
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.dims = pmoe.dims(cfg.T, cfg.d, cfg.E, cfg.k, cfg.I, cfg.b)
        self.w13, self.s13 = _dev(w13, self.device), _dev(s13, self.device)
        self.w2, self.s2 = _dev(w2, self.device), _dev(s2, self.device)
        self.wts = pmoe.weights(cfg.fmt, self.w13, self.s13, self.w2, self.s2)
        self.Wr = None if Wr is None else _dev(Wr, self.device)
        self.bias = None if bias is None else _dev(bias, self.device)
        self.R_up = self.R_down = None
        self.S_up = self.S_down = None
        self.Rf_up = self.Rf_down = None
        if S_up is not None:
            self.S_up = _dev(S_up, self.device)
            self.R_up, self.Rf_up = self._cayley(self.S_up)
        elif R_up is not None:
            self.R_up = _dev(R_up, self.device)
        if S_down is not None:
            self.S_down = _dev(S_down, self.device)
            self.R_down, self.Rf_down = self._cayley(self.S_down)
        elif R_down is not None:
            self.R_down = _dev(R_down, self.device)
        self.adp = None
        if self.R_up is not None:
            su = 0 if self.R_up.shape[0] == 1 else cfg.d * cfg.b
            sd = 0 if (self.R_down is None or self.R_down.shape[0] == 1) else cfg.I * cfg.b
            self.adp = pmoe.adapter(self.R_up, self.R_down, su, sd)
        self._ws = {}

    def _cayley(self, S):
        b = self.cfg.b
        nblk = S.numel() // (b * b)
        Rb = torch.empty(S.shape, dtype=torch.int16, device=self.device)
        Rf = torch.empty(S.shape, dtype=torch.float32, device=self.device)
        pmoe.adapter_cayley(nblk, b, S, Rb, Rf)
        return Rb, Rf

    def workspace(self, op, C=1, mode=pmoe.MODE_FUSED) -> torch.Tensor:
        key = (op, C, mode)
        if key not in self._ws:
            n = pmoe.moe_workspace_bytes(self.dims, op, C, mode)
            self._ws[key] = torch.zeros(max(n, 256), dtype=torch.uint8, device=self.device)
        return self._ws[key]

    def new_routing(self) -> Routing:
        cfg, dev = self.cfg, self.device
        i32 = dict(dtype=torch.int32, device=dev)
        return Routing(idx=torch.zeros((cfg.T, cfg.k), **i32),
                       w=torch.zeros((cfg.T, cfg.k), dtype=torch.float32, device=dev),
                       counts=torch.zeros(cfg.E, **i32), offsets=torch.zeros(cfg.E + 1, **i32),
                       perm=torch.zeros(cfg.P, **i32), inv_perm=torch.zeros(cfg.P, **i32),
                       active=torch.zeros(cfg.E, **i32), num_active=torch.zeros(1, **i32))

    # -------------------------------------------------------------- steps
    def route(self, X: torch.Tensor, rt: Routing, logits: torch.Tensor | None = None,
              mode: int = pmoe.ROUTE_FAST):
        ws = self.workspace(pmoe.OP_PERMUTE)
        pmoe.moe_route(self.dims, X, self.Wr, self.bias, logits, rt.idx, rt.w, ws, mode=mode)

    def permute(self, rt: Routing):
        pmoe.moe_permute(self.dims, rt.idx, rt.c(), self.workspace(pmoe.OP_PERMUTE))

    def new_ctx(self) -> torch.Tensor:
        """The forward's saved context for the backward (moe_ctx_bytes)."""
        return torch.empty(max(pmoe.moe_ctx_bytes(self.dims), 16), dtype=torch.uint8,
                           device=self.device)

    def forward(self, X, rt: Routing, Y, C=None, mode=pmoe.MODE_FUSED, ctx=None):
        C = C or self.cfg.C
        ws = self.workspace(pmoe.OP_FORWARD, C, mode)
        pmoe.moe_chunked_forward(self.dims, self.wts, self.adp, rt.c(), X, C, mode, Y, ctx, ws)

    def backward(self, X, dY, ctx, rt: Routing, dX, d_topk_w=None, dR_up=None, dR_down=None,
                 C=None):
        C = C or self.cfg.C
        ws = self.workspace(pmoe.OP_BACKWARD, C)
        pmoe.moe_backward_data(self.dims, self.wts, self.adp, rt.c(), X, dY, ctx, C, dX,
                               d_topk_w, dR_up, dR_down, ws)

    def new_balance(self, nseq: int = 1) -> Balance:
        E, dev = self.cfg.E, self.device
        return Balance(counts=torch.zeros((nseq, E), dtype=torch.int32, device=dev),
                       ntok=torch.zeros(nseq, dtype=torch.int32, device=dev),
                       pmean=torch.zeros((nseq, E), dtype=torch.float32, device=dev),
                       loss=torch.zeros(nseq, dtype=torch.float32, device=dev))

    def _balance_ws(self, nseq: int) -> torch.Tensor:
        key = ("balance", nseq)
        if key not in self._ws:
            n = pmoe.moe_balance_ws_bytes(self.dims, nseq)
            if n == 0:
                raise ValueError(f"unsupported number of sequences: {nseq}")
            self._ws[key] = torch.zeros(n, dtype=torch.uint8, device=self.device)
        return self._ws[key]

    def _balance_args(self, logits, valid, seq, nseq):
        cfg, dev = self.cfg, self.device
        check_current(dev)
        check_tensor("logits", logits, (torch.float32,), (cfg.T, cfg.E), dev)
        if valid is not None:
            check_tensor("valid", valid, (torch.uint8,), (cfg.T,), dev)
        if seq is not None:
            check_tensor("seq", seq, (torch.int32,), (nseq + 1,), dev)

    def balance(self, logits, rt: Routing, bal: Balance, valid=None, seq=None):
        """Counts, mean probabilities and balance loss of the routing ``rt`` of
        ``logits`` (f32 [T, E], as ``route`` writes them); ``valid`` uint8 [T]
        or None, ``seq`` int32 [nseq + 1] bounds or None (one sequence)."""
        nseq = bal.loss.shape[0]
        self._balance_args(logits, valid, seq, nseq)
        pmoe.moe_balance_forward(self.dims, logits, rt.idx, valid, seq, nseq, bal.counts, bal.ntok,
                                 bal.pmean, bal.loss, self._balance_ws(nseq))

    def route_backward(self, logits, rt: Routing, dlogits, d_topk_w=None, bal: Balance | None = None,
                       g_loss=None, valid=None, seq=None):
        """dlogits (f32 [T, E]) from the routing weights' gradient (``d_topk_w``
        of ``backward``) and from the balance losses (upstream ``g_loss``
        f32 [nseq], ``bal`` from ``balance``); either may be left out."""
        cfg, dev = self.cfg, self.device
        nseq = 1 if bal is None else bal.loss.shape[0]
        if (g_loss is None) != (bal is None):
            raise ValueError("bal and g_loss go together")
        self._balance_args(logits, valid, seq, nseq)
        check_tensor("dlogits", dlogits, (torch.float32,), (cfg.T, cfg.E), dev)
        if d_topk_w is not None:
            check_tensor("d_topk_w", d_topk_w, (torch.float32,), (cfg.T, cfg.k), dev)
        if g_loss is not None:
            check_tensor("g_loss", g_loss, (torch.float32,), (nseq,), dev)
        pmoe.moe_route_backward(self.dims, logits, rt.idx, rt.w, d_topk_w, valid, seq, nseq,
                                bal.counts if bal else None, bal.ntok if bal else None, g_loss,
                                dlogits, self._balance_ws(nseq))

    def grads(self):
        """Fresh (dR_up, dR_down) buffers shaped like the rotations."""
        dru = None if self.R_up is None else torch.zeros(self.R_up.shape, dtype=torch.float32,
                                                         device=self.device)
        drd = None if self.R_down is None else torch.zeros(self.R_down.shape,
                                                           dtype=torch.float32, device=self.device)
        return dru, drd

    def status(self) -> int:
        """OR of the device error words of every workspace used so far."""
        s = 0
        for ws in self._ws.values():
            s = s or pmoe.moe_query_status(ws)
        return s
