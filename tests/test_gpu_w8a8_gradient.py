"""The 8-bit layer's gradient against differences of the layer itself, without a tolerance.

Everything is a small whole number: activations and upstream gradients of at most 3 but for
14 in the first column of each block of 128, so that the block's scale is 14 / 448 = 2^-5
and the codes hold the numbers exactly (E4M3 holds whole numbers up to 16).  The weight is the
sum of four signed permutations times scales of 1 or 2, so that no result exceeds 4 * 14 * 2 =
112, which BF16 holds exactly (whole numbers up to 256).
"""
import pytest
import torch

from precision_moe_adapter_gb300 import build, pmoe
from precision_moe_adapter_gb300.linear import DeviceLinearW8A8
from test_gpu_w8a8 import BF16, D, E4M3, blocks, gen

pytestmark = pytest.mark.gpu
B = 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    pmoe.lib()


def whole(g, low, *shape):
    return torch.randint(low, -low + 1, shape, generator=g, device="cuda").float()


def permutation(g, n):
    """A signed permutation, [n, n]."""
    sign = 1.0 - 2.0 * torch.randint(0, 2, (n, 1), generator=g, device="cuda")
    return torch.eye(n, device="cuda")[torch.randperm(n, generator=g, device="cuda")] * sign


@pytest.mark.parametrize("one_order", [False, True])
@pytest.mark.parametrize("adapter", [False, True])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("rows,N", [(5, 384), (64, 384), (300, 1024)])
def test_gradient_by_differences(rows, N, pow2, adapter, one_order):
    g = gen(rows + N)
    K = N
    X, V, dY = whole(g, -3, rows, K), whole(g, -1, rows, K), whole(g, -3, rows, N)
    X[:, ::128] = dY[:, ::128] = 14.0
    V[:, ::128] = 0.0
    Wq = sum(permutation(g, N) for _ in range(4)).to(E4M3)
    Ws = torch.randint(1, 3, (N // 128, K // 128), generator=g, device="cuda").float()
    R = dR = None
    if adapter:                                # permutations within a block of 64: every rotated row is exact too
        R = torch.stack([permutation(g, B) for _ in range(K // B)]).to(BF16)
        dR = torch.empty((K // B, B, B), device="cuda")
    lin = DeviceLinearW8A8(Wq, Ws, rows, R=R, pow2=pow2, one_order=one_order)
    Y = []
    for sign in (1, -1, 0):
        Y.append(torch.empty((rows, N), dtype=BF16, device="cuda"))
        lin.forward((X + sign * V).to(BF16), Y[-1])
    dX = torch.empty((rows, K), dtype=BF16, device="cuda")
    lin.backward(X.to(BF16), dY.to(BF16), dX, dR)
    assert lin.status() == pmoe.PMOE_OK
    # <dY, Y> of each row along V
    num = ((Y[0].to(D) - Y[1].to(D)) / 2 * dY.to(D)).sum(1)
    want = (dX.to(D) * V.to(D)).sum(1)
    assert torch.equal(num, want)
    assert (want != 0).float().mean() > 0.8
    W = Wq.to(D) * blocks(Ws, N, K)
    xt, dxt = X.to(D), dY.to(D) @ W
    if adapter:
        r = R.to(D)
        x = xt.view(rows, -1, B)
        assert torch.equal(dR.to(D), torch.einsum("rji,rjk->jik", x, dxt.view(rows, -1, B)))
        xt = torch.einsum("rji,jik->rjk", x, r).reshape(rows, K)
        dxt = torch.einsum("rjk,jik->rji", dxt.view(rows, -1, B), r).reshape(rows, K)
    assert torch.equal(Y[2].to(D), xt @ W.T) and torch.equal(dX.to(D), dxt)
