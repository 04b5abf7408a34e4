"""The 8-bit linear layer in one order: a row's results are the same bits whatever the
number of rows in the call, as those of the layer's other products are.
"""
import pytest
import torch

from precision_moe_adapter_gb300 import build, pmoe
from precision_moe_adapter_gb300.linear import DeviceLinearW8A8
from test_gpu_w8a8 import BF16, activations, gen, near, product, quantised, weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    pmoe.lib()


@pytest.mark.parametrize("adapter", [False, True])
@pytest.mark.parametrize("N,K", [(4096, 7168), (7168, 2048), (1040, 2112), (128, 18432), (256, 576)])
def test_a_row_does_not_depend_on_the_batch(N, K, adapter):
    """Batches of one row up to some thousands: shared and not, single CTAs and pairs."""
    rows = 2500
    X, dY = activations(rows, K, seed=1, spread=0.3), activations(rows, N, seed=2, spread=0.3)
    Wq, Ws = weight(N, K)
    R = dR = None
    if adapter:
        S = 0.05 * torch.randn((K // 64, 64, 64), generator=gen(4), device="cuda")
        R, dR = torch.empty((K // 64, 64, 64), dtype=BF16, device="cuda"), torch.empty_like(S)
        pmoe.adapter_cayley(K // 64, 64, S - S.transpose(1, 2), R, None)
    lin = DeviceLinearW8A8(Wq, Ws, rows, R=R, one_order=True)

    def both(r):
        x, dy = X[r].contiguous(), dY[r].contiguous()
        y, dx = torch.empty_like(dy), torch.empty_like(x)
        lin.forward(x, y)
        lin.backward(x, dy, dx, dR)
        return y, dx

    Y, dX = both(slice(0, rows))
    for r in (slice(0, 1), slice(7, 9), slice(40, 57), slice(100, 164), slice(3, 130), slice(0, 128), slice(200, 457),
              slice(5, 700), slice(1, 1999)):
        y, dx = both(r)
        assert torch.equal(y, Y[r]) and torch.equal(dx, dX[r]), r
    assert lin.status() == pmoe.PMOE_OK
    if not adapter:
        r = slice(100, 164)
        near(Y[r], *product(*quantised(X[r]), Wq, Ws))
        near(dX[r], *product(*quantised(dY[r]), Wq.T, Ws.T.contiguous()))


@pytest.mark.parametrize("rows,N,K", [(1, 4096, 7168), (64, 7168, 7168), (333, 1104, 2064), (2500, 4096, 528)])
def test_one_order_is_the_products(rows, N, K):
    """The layer's product and fp8_gemm are the same; with rows enough the two orders are."""
    X = activations(rows, K, seed=rows)
    Wq, Ws = weight(N, K)
    q, s = torch.empty((rows, K), dtype=torch.uint8, device="cuda"), torch.empty((-(-K // 128), rows), device="cuda")
    ws = torch.zeros(pmoe.fp8_gemm_ws_bytes(rows, N, K), dtype=torch.uint8, device="cuda")
    Y, Z, V = (torch.empty((rows, N), dtype=BF16, device="cuda") for _ in range(3))
    DeviceLinearW8A8(Wq, Ws, rows, backward=False, one_order=True).forward(X, Y)
    pmoe.fp8_quantize(rows, K, X, q, s)
    pmoe.fp8_gemm(rows, N, K, q, s, Wq, Ws, Z, ws, one_order=True)
    assert torch.equal(Y, Z)
    pmoe.fp8_gemm(rows, N, K, q, s, Wq, Ws, V, ws)
    want, M = product(q.view(torch.float8_e4m3fn), s, Wq, Ws)
    near(Z, want, M)
    near(V, want, M)
    if rows > 2000:
        assert torch.equal(V, Z)
