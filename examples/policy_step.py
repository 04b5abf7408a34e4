"""One block's training steps, every part of the library at once.

A MoE layer on a frozen INT4 base with an orthogonal adapter, a frozen
vocabulary head, and the three losses of adapter-first RL:

    route -> permute -> forward -> H = X + Y
      policy     -A_t log p(y_t)             head.logprob
      reference  KL to the base's top logits head.distill (teacher: no adapter)
      balance    the router's load           layer.balance
    head backward -> layer backward -> route_backward -> Cayley gradient

The adapter's skew parameters and the router are trained by plain gradient
descent; the objective must fall.  Run: python examples/policy_step.py [steps]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from precision_moe_adapter_gb300 import inputs as gi  # noqa: E402
from precision_moe_adapter_gb300 import pmoe  # noqa: E402
from precision_moe_adapter_gb300.head import DeviceHead  # noqa: E402
from precision_moe_adapter_gb300.layer import DeviceLayer  # noqa: E402


def run(steps=10, V=1000, K=16, lr_adapter=0.1, lr_router=0.01, c_ref=0.1, c_bal=0.05, seed=0):
    """The objective of each step (a list of floats)."""
    cfg = gi.CONFIGS["tiny"]
    T, d, E, b = cfg.T, cfg.d, cfg.E, cfg.b
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w13, s13, w2, s2 = gi.gen_weights(cfg)
    Wr, _ = gi.gen_router(cfg)
    Su, Sd = gi.gen_adapter_params(cfg)
    layer = DeviceLayer(cfg, w13, s13, w2, s2, Wr=Wr, S_up=Su, S_down=Sd)
    base = DeviceLayer(cfg, w13, s13, w2, s2, Wr=Wr)          # the reference policy: no adapter
    X = torch.from_numpy(gi.gen_x(cfg)).view(torch.bfloat16).cuda()
    W = (0.05 * torch.randn((V, d), generator=g, device="cuda")).to(torch.bfloat16)
    y = torch.randint(0, V, (T,), generator=g, device="cuda").to(torch.int32)
    y[: T // 8] = -1                                           # prompt tokens
    adv = torch.rand(T, generator=g, device="cuda") + 0.5
    head = DeviceHead(W, T, K=K)

    f32 = dict(dtype=torch.float32, device="cuda")
    rt, bal, ctx = layer.new_routing(), layer.new_balance(), layer.new_ctx()
    logits, dlogits = torch.empty((T, E), **f32), torch.empty((T, E), **f32)
    Y, dH1, dH2, dX = (torch.empty_like(X) for _ in range(4))
    logp, kl, lse = (torch.empty(T, **f32) for _ in range(3))
    dtw = torch.empty((T, cfg.k), **f32)
    ntrain = int((y >= 0).sum())
    g_logp, g_kl = -adv / ntrain, torch.full((T,), c_ref / T, **f32)
    g_bal = torch.full((1,), c_bal, **f32)

    # the teacher: the base's own top K logits of each token
    base.route(X, rt)
    base.permute(rt)
    base.forward(X, rt, Y)
    z0 = (X + Y).float() @ W.float().T
    t_logits, t_idx = z0.topk(K, dim=1)
    t_logits, t_idx = t_logits.contiguous(), t_idx.to(torch.int32).contiguous()

    history = []
    for _ in range(steps):
        layer.route(X, rt, logits)
        layer.permute(rt)
        layer.forward(X, rt, Y, ctx=ctx)
        H = X + Y
        head.logprob(H, y, logp, lse)
        head.logprob_backward(H, y, lse, g_logp, dH1)          # frozen head: no dW
        head.distill(H, t_idx, t_logits, kl, lse)
        head.distill_backward(H, t_idx, t_logits, lse, g_kl, dH2)
        layer.balance(logits, rt, bal)
        history.append(float((g_logp * logp).sum() + (g_kl * kl).sum() + c_bal * bal.loss[0]))

        dRu, dRd = layer.grads()
        layer.backward(X, dH1 + dH2, ctx, rt, dX, dtw, dRu, dRd)
        layer.route_backward(logits, rt, dlogits, dtw, bal, g_bal)
        layer.Wr -= lr_router * (X.float().T @ dlogits)
        for S, R, Rf, dR in ((layer.S_up, layer.R_up, layer.Rf_up, dRu),
                             (layer.S_down, layer.R_down, layer.Rf_down, dRd)):
            n, dS = S.numel() // (b * b), torch.empty_like(S)
            pmoe.adapter_cayley_grad(n, b, S, Rf, dR, dS)
            S -= lr_adapter * dS
            pmoe.adapter_cayley(n, b, S, R, Rf)
    status = layer.status() or base.status() or head.status()
    if status != pmoe.PMOE_OK:
        raise pmoe.PmoeError(status, "policy_step")
    return history


if __name__ == "__main__":
    for i, v in enumerate(run(int(sys.argv[1]) if len(sys.argv) > 1 else 10)):
        print(f"step {i:3d}  objective {v:.5f}")
