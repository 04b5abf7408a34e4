"""The example that runs the layer, the head's losses and the router's training
side together: its objective falls, by what the gradient promises, and two
runs are identical."""
import os
import sys

import pytest

from precision_moe_adapter_gb300 import build, pmoe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def step():
    build.build()
    pmoe.lib()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import policy_step
    return policy_step


def test_objective_falls_and_repeats(step):
    a = step.run(8)
    assert all(y < x for x, y in zip(a, a[1:]))
    assert a == step.run(8)


def test_first_step_is_first_order(step):
    """With the router fixed the objective is smooth in the adapter: the drop
    of one step is proportional to the step (10% for the second order)."""
    drop = [(lambda h: h[0] - h[1])(step.run(2, lr_adapter=lr, lr_router=0.0)) for lr in (0.05, 0.1)]
    assert drop[0] > 0 and 1.8 < drop[1] / drop[0] < 2.2


def test_layer_checks_its_tensors(step):
    import torch

    from precision_moe_adapter_gb300 import inputs as gi
    from precision_moe_adapter_gb300.layer import DeviceLayer
    cfg = gi.CONFIGS["tiny"]
    layer = DeviceLayer(cfg, *gi.gen_weights(cfg), Wr=gi.gen_router(cfg)[0])
    rt, bal = layer.new_routing(), layer.new_balance(2)
    logits = torch.zeros((cfg.T, cfg.E), device="cuda")
    seq = torch.tensor([0, 3, cfg.T], dtype=torch.int32, device="cuda")
    layer.balance(logits, rt, bal, seq=seq)
    with pytest.raises(ValueError):
        layer.balance(logits.T, rt, bal, seq=seq)
    with pytest.raises(TypeError):
        layer.balance(logits.half(), rt, bal, seq=seq)
    with pytest.raises(ValueError):
        layer.balance(logits, rt, bal, seq=seq[:2])
    with pytest.raises(ValueError):
        layer.route_backward(logits, rt, torch.zeros_like(logits), bal=bal)      # no g_loss
    with pytest.raises(pmoe.PmoeError):
        layer.balance(logits, rt, bal)                                           # two sequences, no bounds
