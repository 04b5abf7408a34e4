"""A block on an FP8 base, every operator of its training step in turn: router
logits -> scored gate -> experts -> an 8-bit projection with its adapter, and
back: projection -> experts -> gate and balance loss -> Cayley gradients -> clip.

Each stage is compared with FP64 on the device's own inputs of that stage
(tolerances: those stages' own), the whole step is repeated, and captured."""
import math

import numpy as np
import pytest
import torch

from helpers import assert_close
from precision_moe_adapter_gb300 import build, pmoe
from precision_moe_adapter_gb300 import inputs as gi
from precision_moe_adapter_gb300.grads import GradList
from precision_moe_adapter_gb300.layer import DeviceLayer
from precision_moe_adapter_gb300.linear import DeviceLinearW8A8

from test_gpu_gate import reference as gate_reference
from test_gpu_w8a8 import near, product, quantised

pytestmark = pytest.mark.gpu
BF16, D = torch.bfloat16, torch.float64


class Block:
    def __init__(self, seed=0):
        import dataclasses
        cfg = dataclasses.replace(gi.CONFIGS["tiny"], fmt=gi.FP8)
        self.cfg = cfg
        T, d, E, b, N = cfg.T, cfg.d, cfg.E, cfg.b, 272
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        randn = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.layer = DeviceLayer(cfg, *gi.gen_weights(cfg), Wr=gi.gen_router(cfg)[0],
                                 **dict(zip(("S_up", "S_down"), gi.gen_adapter_params(cfg))))
        self.bias = 0.05 * randn(E)
        self.gate = pmoe.gate(T, E, cfg.k, groups=4, topk_groups=2, factor=2.5)
        q, s = randn(N, d).to(torch.float8_e4m3fn), 0.005 + 0.015 * torch.rand((3, 2), generator=g, device="cuda")
        S = 0.02 * randn(d // b, b, b)
        self.S = S - S.transpose(1, 2)
        self.R, self.Rf = torch.empty((d // b, b, b), dtype=BF16, device="cuda"), torch.empty_like(self.S)
        pmoe.adapter_cayley(d // b, b, self.S, self.R, self.Rf)
        self.lin = DeviceLinearW8A8(q, s, T, R=self.R)
        self.X = randn(T, d).to(BF16)
        self.dO = (0.1 * randn(T, N)).to(BF16)
        f32 = dict(dtype=torch.float32, device="cuda")
        self.rt, self.ctx, self.bal = self.layer.new_routing(), self.layer.new_ctx(), self.layer.new_balance()
        self.logits, self.dlogits = torch.empty((T, E), **f32), torch.empty((T, E), **f32)
        self.Y, self.dY, self.dX = (torch.empty_like(self.X) for _ in range(3))
        self.O = torch.empty((T, N), dtype=BF16, device="cuda")
        self.dtw, self.g_bal = torch.empty((T, cfg.k), **f32), torch.full((1,), 0.05, **f32)
        self.dR = torch.empty_like(self.S)
        self.dRu, self.dRd = self.layer.grads()
        params = [self.S, self.layer.S_up, self.layer.S_down]
        self.dS = [torch.empty_like(p) for p in params] + [self.dlogits]
        self.clipped = [torch.empty_like(p) for p in self.dS]
        self.list, self.norm = GradList(self.dS, out=self.clipped), torch.empty(1, **f32)

    def step(self):
        L, b = self.layer, self.cfg.b
        L.router_logits(self.X, self.logits)
        L.gate(self.gate, self.logits, self.rt, bias=self.bias)
        L.permute(self.rt)
        L.forward(self.X, self.rt, self.Y, ctx=self.ctx)
        L.balance(self.logits, self.rt, self.bal)
        self.lin.forward(self.Y, self.O)
        self.lin.backward(self.Y, self.dO, self.dY, self.dR)
        L.backward(self.X, self.dY, self.ctx, self.rt, self.dX, self.dtw, self.dRu, self.dRd)
        L.route_backward(self.logits, self.rt, self.dlogits, None, self.bal, self.g_bal)
        L.gate_backward(self.gate, self.logits, self.rt, self.dtw, self.dlogits, accumulate=True)
        for S, Rf, dR, dS in ((self.S, self.Rf, self.dR, self.dS[0]), (L.S_up, L.Rf_up, self.dRu, self.dS[1]),
                              (L.S_down, L.Rf_down, self.dRd, self.dS[2])):
            pmoe.adapter_cayley_grad(S.numel() // (b * b), b, S, Rf, dR, dS)
        self.list.clip(0.5, self.norm)

    def outputs(self):
        return [t.clone() for t in (self.rt.idx, self.rt.w, self.Y, self.O, self.dX, self.dlogits, self.norm, *self.clipped)]


@pytest.fixture(scope="module")
def block():
    build.build()
    pmoe.lib()
    b = Block()
    b.step()
    torch.cuda.synchronize()
    assert b.layer.status() == pmoe.PMOE_OK and b.lin.status() == pmoe.PMOE_OK
    return b


def test_router_logits_are_those_of_route(block):
    logits, rt = torch.empty_like(block.logits), block.layer.new_routing()
    for mode in (pmoe.ROUTE_FAST, pmoe.ROUTE_EXACT):
        block.layer.route(block.X, rt, logits, mode=mode)
        alone = torch.empty_like(logits)
        block.layer.router_logits(block.X, alone, mode=mode)
        assert torch.equal(alone, logits)


def test_each_stage(block):
    B, cfg = block, block.cfg
    idx, w, dl, mag = gate_reference(B.logits, B.bias, cfg.k, "sigmoid", 4, 2, 2, True, 2.5, B.dtw)
    assert torch.equal(B.rt.idx.long(), idx)
    assert torch.all((B.rt.w.to(D) - w).abs() <= 2.0 ** -16 * w)
    # the layer with this routing: the same experts and weights by its own path, in any chunking
    Y2 = torch.empty_like(B.Y)
    B.layer.forward(B.X, B.rt, Y2, C=1)
    assert torch.equal(Y2, B.Y)
    Yr = torch.empty_like(B.Y)
    pmoe.adapter_apply(cfg.T, cfg.d, cfg.b, B.Y, B.R, Yr)
    near(B.O, *product(*quantised(Yr), B.lin.q, B.lin.s))
    # the gate's part beside the balance loss's
    bal = torch.empty_like(B.dlogits)
    B.layer.route_backward(B.logits, B.rt, bal, None, B.bal, B.g_bal)
    tol = 2.0 ** -15 * mag + 2.0 ** -23 * (bal.abs() + dl.abs())
    assert torch.all((B.dlogits.to(D) - bal.to(D) - dl).abs() <= tol)
    norm = math.sqrt(sum(float((t.to(D) ** 2).sum()) for t in B.dS))
    assert abs(float(B.norm) - norm) <= 2.0 ** -21 * norm and norm > 0.5
    for t, c in zip(B.dS, B.clipped):
        want = t.to(D) * (0.5 / (norm + 1e-6))
        assert torch.all((c.to(D) - want).abs() <= 2.0 ** -21 * want.abs() + 2.0 ** -149)


def test_the_projections_gradients(block):
    B, cfg = block, block.cfg
    dyt, _ = product(*quantised(B.dO), B.lin.q.T, B.lin.s.T.contiguous())
    t = dyt.view(cfg.T, cfg.d // cfg.b, cfg.b)
    f = lambda x: x.to(D).cpu().numpy()
    want = torch.einsum("rjk,jik->rji", t, B.R.to(D)).reshape(cfg.T, cfg.d)
    scale = float(want.abs().mean())
    assert_close(f(B.dY) / scale, f(want) / scale, "dY")
    want = torch.einsum("rji,rjk->jik", B.Y.to(D).view(cfg.T, cfg.d // cfg.b, cfg.b), t)
    scale = float(want.abs().mean())
    assert_close(f(B.dR) / scale, f(want) / scale, "dR")
    assert np.isfinite(f(B.dX)).all() and float(B.dX.abs().max()) > 0


def test_steps_repeat_and_replay(block):
    ref = block.outputs()
    block.step()
    assert all(torch.equal(a, b) for a, b in zip(ref, block.outputs()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        block.step()
    for _ in range(2):
        for t in (block.O, block.dX, block.dlogits, block.norm, *block.clipped):
            t.zero_()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(ref, block.outputs()))


def test_two_blocks_at_once():
    """Two blocks with workspaces of their own, on two streams at the same time."""
    blocks = [Block(seed=s) for s in (1, 2)]
    refs = []
    for b in blocks:
        b.step()
        torch.cuda.synchronize()
        refs.append(b.outputs())
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(5):
        for b, st in zip(blocks, streams):
            with torch.cuda.stream(st):
                b.step()
    torch.cuda.synchronize()
    for b, ref in zip(blocks, refs):
        assert all(torch.equal(x, y) for x, y in zip(ref, b.outputs()))
        assert b.layer.status() == pmoe.PMOE_OK and b.lin.status() == pmoe.PMOE_OK


@pytest.mark.parametrize("rows", [[1, 700], [64, 64], [3000, 17]])
def test_two_projections_at_once(rows):
    """Shared tiles in clusters beside pairs and single CTAs, on two streams."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    lins, Xs, Ys = [], [], []
    for n in rows:
        q = torch.randn((4096, 2048), generator=g, device="cuda").to(torch.float8_e4m3fn)
        lins.append(DeviceLinearW8A8(q, torch.full((32, 16), 0.01, device="cuda"), n))
        Xs.append(torch.randn((n, 2048), generator=g, device="cuda").to(BF16))
        Ys.append(torch.empty((n, 4096), dtype=BF16, device="cuda"))
    refs = []
    for lin, X, Y in zip(lins, Xs, Ys):
        lin.forward(X, Y)
        torch.cuda.synchronize()
        refs.append(Y.clone())
        Y.zero_()
    streams = [torch.cuda.Stream() for _ in rows]
    torch.cuda.synchronize()
    for _ in range(20):
        for lin, X, Y, st in zip(lins, Xs, Ys, streams):
            with torch.cuda.stream(st):
                lin.forward(X, Y)
    torch.cuda.synchronize()
    assert all(torch.equal(y, r) for y, r in zip(Ys, refs))
    assert all(lin.status() == pmoe.PMOE_OK for lin in lins)
