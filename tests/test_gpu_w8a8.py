"""The 8-bit linear layer on the GPU: the quantisation bit for bit against its
definition in FP64, the product within the error of its sums.

Tolerance of the product.  A block's 128 products of E4M3 numbers are exact; the
tensor cores add them to FP32 with truncation, each addition losing at most 2^-23 of
the largest partial sum: under 128 * 2^-23 = 2^-16 of the sum of magnitudes.  The
scales' product and the sum over blocks (at most 144 here, one FP32 rounding each)
add less than 2^-16 again: 2^-15 of M = sum_b As Ws sum_k |A W|, and half a step of
BF16 (2^-8) of the result.
"""
import math

import pytest
import torch

from helpers import assert_close
from precision_moe_adapter_gb300 import build, pmoe
from precision_moe_adapter_gb300.linear import DeviceLinearW8A8

pytestmark = pytest.mark.gpu
BF16, F32, D, E4M3 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn
EPS, ACC = 2.0 ** -8, 2.0 ** -15


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    pmoe.lib()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def activations(rows, K, seed=0, spread=1.0):
    g = gen(seed)
    x = torch.randn((rows, K), generator=g, device="cuda")
    x *= torch.exp(spread * torch.randn(K, generator=g, device="cuda"))
    return (x * torch.exp(spread * torch.randn((rows, 1), generator=g, device="cuda"))).to(BF16)


def weight(N, K, seed=0):
    g = gen(seed + 1000)
    q = torch.randn((N, K), generator=g, device="cuda").to(E4M3)
    s = 0.005 + 0.015 * torch.rand((-(-N // 128), -(-K // 128)), generator=g, device="cuda")
    return q, s


def e4m3(v):
    """Doubles to the nearest E4M3 value, ties to even."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def quantised(X, pow2=False):
    """q (as doubles) and s [blocks, rows] of the definition."""
    rows, K = X.shape
    KB = -(-K // 128)
    P = torch.zeros((rows, KB * 128), dtype=D, device="cuda")
    P[:, :K] = X.to(D)
    P = P.view(rows, KB, 128)
    a = P.abs().amax(2, keepdim=True).clamp(min=2.0 ** -100)
    if pow2:
        s = torch.exp2(torch.ceil(torch.log2(a / 448)))
        s = torch.where(s / 2 * 448 >= a, s / 2, s)           # (log2 of an exact power may be a unit off)
        s = torch.where(s * 448 < a, s * 2, s)
        q = e4m3(P / s)
    else:
        s = (a / 448).float().to(D)
        q = e4m3(P * 448 / a)
    return q.view(rows, KB * 128)[:, :K], s[:, :, 0].T.contiguous()


def blocks(s, n, k):
    return s.to(D).repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]


def product(q, s, Wq, Ws):
    """(Y, M) in FP64 of E4M3 values q with scales s [blocks, rows]."""
    N, K = Wq.shape
    A = q.to(D) * s.to(D).T.repeat_interleave(128, 1)[:, :K]
    W = Wq.to(D) * blocks(Ws, N, K)
    return A @ W.T, A.abs() @ W.abs().T


def near(got, want, M):
    bad = (got.to(D) - want).abs() > EPS * want.abs() + ACC * M
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(),
                           float(((got.to(D) - want).abs() / (EPS * want.abs() + ACC * M)).max()))


# ---------------------------------------------------------------- quantisation

@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("rows,K", [(1, 16), (1, 128), (3, 144), (7, 112), (33, 1040), (130, 2064), (5, 7168), (1000, 256)])
def test_quantize(rows, K, pow2):
    X = activations(rows, K, seed=rows + K, spread=2.0)
    X[0, :8] = torch.tensor([0, 1, -1, 448, -0.0, 1e-30, 3e38, 1.75], dtype=BF16)
    X[-1, -16:] = 0
    KB = -(-K // 128)
    q = torch.full((rows + 2, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((KB * rows + 8,), math.nan, device="cuda")
    pmoe.fp8_quantize(rows, K, X, q, s, pow2)
    rq, rs = quantised(X, pow2)
    assert torch.equal(s[:KB * rows].view(KB, rows).to(D), rs) and s[KB * rows:].isnan().all()
    assert torch.equal(q[:rows].view(E4M3).to(D), rq) and (q[rows:] == 0x55).all()


def test_quantize_every_quotient():
    """Every BF16 significand over every largest one, at 40 distances: each midpoint
    of E4M3 that a quotient can meet is met."""
    a = (1 + torch.arange(128, device="cuda") / 128).to(D)
    for sh in range(0, 40):
        X = (a[None, :] * 2.0 ** -sh).repeat(128, 1)                     # row i: significands under a_i * 2
        X[:, 0] = 2 * a
        X = torch.cat([X, -X * 0.5], 1).to(BF16)
        q = torch.empty((128, 256), dtype=torch.uint8, device="cuda")
        s = torch.empty((2, 128), device="cuda")
        for pow2 in (False, True):
            pmoe.fp8_quantize(128, 256, X, q, s, pow2)
            rq, rs = quantised(X, pow2)
            assert torch.equal(s.to(D), rs) and torch.equal(q.view(E4M3).to(D), rq), sh


@pytest.mark.parametrize("pow2", [False, True])
def test_quantize_extremes(pow2):
    """Blocks of zeros, of BF16's least and largest numbers, and of NaN or infinity."""
    X = torch.zeros((8, 256), dtype=BF16, device="cuda")
    X[1] = 2.0 ** -133
    X[2] = 2.0 ** -100
    X[3, :128] = torch.finfo(BF16).max
    X[4, 5] = math.nan
    X[5, 200] = math.inf
    X[6, 0] = -math.inf
    X[7] = 1.0
    q = torch.empty((8, 256), dtype=torch.uint8, device="cuda")
    s = torch.empty((2, 8), device="cuda")
    pmoe.fp8_quantize(8, 256, X, q, s, pow2)
    rows = [0, 1, 2, 3, 7]
    rq, rs = quantised(X[rows], pow2)
    assert torch.equal(q[rows].view(E4M3).to(D), rq) and torch.equal(s[:, rows].to(D), rs)
    v = q.view(E4M3).to(F32).view(8, 2, 128) * s.T[:, :, None]
    bad = torch.zeros((8, 2), dtype=torch.bool, device="cuda")
    bad[4, 0] = bad[5, 1] = bad[6, 0] = True
    assert v[bad].isnan().all() and not v[~bad].isnan().any()


@pytest.mark.parametrize("N,K", [(16, 16), (64, 64), (128, 256), (1104, 2064), (272, 48), (112, 1040)])
def test_transpose(N, K):
    q = torch.randint(0, 256, (N, K), generator=gen(N), device="cuda").to(torch.uint8)
    s = torch.rand((-(-N // 128), -(-K // 128)), device="cuda")
    qt, st = torch.zeros((K + 1, N), dtype=torch.uint8, device="cuda"), torch.zeros((s.numel() + 1,), device="cuda")
    pmoe.fp8_transpose(N, K, q, s, qt, st)
    assert torch.equal(qt[:K], q.T) and (qt[K] == 0).all()
    assert torch.equal(st[:-1].view(s.shape[1], s.shape[0]), s.T) and st[-1] == 0


# ---------------------------------------------------------------- product

SHAPES = [(1, 16, 16), (1, 128, 128), (2, 144, 272), (7, 4096, 1024), (8, 112, 7168), (9, 256, 128 * 5 + 16),
          (33, 1040, 2064), (64, 7168, 2048), (127, 128, 640), (128, 256, 512), (129, 384, 640), (200, 16, 4096),
          (255, 512, 1536), (256, 128, 18432), (257, 1104, 2064), (333, 2048, 768), (1000, 5008, 1040),
          (2050, 2560, 528), (2305, 4112, 272)]


@pytest.mark.parametrize("rows,N,K", SHAPES)
def test_gemm(rows, N, K):
    X = activations(rows, K, seed=rows)
    Wq, Ws = weight(N, K, seed=N)
    KB = -(-K // 128)
    q, s = torch.empty((rows, K), dtype=torch.uint8, device="cuda"), torch.empty((KB, rows), device="cuda")
    pmoe.fp8_quantize(rows, K, X, q, s)
    ws = torch.full((pmoe.fp8_gemm_ws_bytes(rows, N, K),), 0xFF, dtype=torch.uint8, device="cuda")
    pmoe.moe_clear_status(ws)
    Y = torch.full((rows + 3, N), math.nan, dtype=BF16, device="cuda")
    pmoe.fp8_gemm(rows, N, K, q, s, Wq, Ws, Y, ws)
    assert pmoe.moe_query_status(ws) == pmoe.PMOE_OK
    near(Y[:rows], *product(q.view(E4M3), s, Wq, Ws))
    assert Y[rows:].isnan().all()
    Y2 = torch.empty_like(Y[:rows])
    pmoe.fp8_gemm(rows, N, K, q, s, Wq, Ws, Y2, ws)
    assert torch.equal(Y2, Y[:rows])


def test_gemm_scales_are_taken_where_they_belong():
    """One block at a time: small whole numbers, so that every result is exact."""
    rows, N, K = 300, 400, 1040
    g = gen(5)
    q = torch.randint(-3, 4, (rows, K), generator=g, device="cuda").float().to(E4M3)
    Wq = torch.randint(-3, 4, (N, K), generator=g, device="cuda").float().to(E4M3)
    KB, NB = 9, 4
    ws = torch.zeros(pmoe.fp8_gemm_ws_bytes(rows, N, K), dtype=torch.uint8, device="cuda")
    Y = torch.empty((rows, N), dtype=BF16, device="cuda")
    for b in range(KB):
        s = torch.zeros((KB, rows), device="cuda")
        s[b] = torch.exp2(torch.randint(-4, 5, (rows,), generator=g, device="cuda").float())
        Ws = torch.exp2(torch.randint(-4, 5, (NB, KB), generator=g, device="cuda").float())
        pmoe.fp8_gemm(rows, N, K, q, s, Wq, Ws, Y, ws)
        want, _ = product(q, s, Wq, Ws)
        assert torch.equal(Y, want.to(BF16))


def test_gemm_nan_stays_in_its_row_or_column():
    rows, N, K = 140, 272, 400
    X = activations(rows, K)
    X[77, 130] = math.nan
    Wq, Ws = weight(N, K)
    lin = DeviceLinearW8A8(Wq, Ws, rows)
    Y = torch.empty((rows, N), dtype=BF16, device="cuda")
    lin.forward(X, Y)
    bad = Y.isnan()
    assert bad[77].all() and bad.sum() == N


# ---------------------------------------------------------------- the layer

@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("rows,N,K", [(1, 256, 384), (1, 16, 16), (2, 24576, 144), (3, 4096, 7168), (9, 1104, 2064),
                                      (15, 25600, 640), (16, 7168, 4112), (17, 7168, 4112), (33, 1040, 2064),
                                      (333, 1104, 2064), (1500, 4096, 512)])
def test_layer(rows, N, K, pow2):
    X, dY = activations(rows, K, seed=1), activations(rows, N, seed=2)
    Wq, Ws = weight(N, K)
    lin = DeviceLinearW8A8(Wq, Ws, rows + 5, pow2=pow2)
    Y, dX = torch.empty((rows, N), dtype=BF16, device="cuda"), torch.empty((rows, K), dtype=BF16, device="cuda")
    lin.forward(X, Y)
    lin.backward(X, dY, dX)
    assert lin.status() == pmoe.PMOE_OK
    near(Y, *product(*quantised(X, pow2), Wq, Ws))
    near(dX, *product(*quantised(dY, pow2), Wq.T, Ws.T.contiguous()))


@pytest.mark.parametrize("rows,N,K,b", [(200, 272, 384, 64), (1, 128, 256, 16), (77, 1040, 512, 128), (129, 256, 192, 32)])
def test_layer_with_an_adapter(rows, N, K, b):
    """x~ through the library's rotation, then Q; the gradient's dx~ into dR and, rotated
    back, dX."""
    X, dY = activations(rows, K, seed=1, spread=0.5), activations(rows, N, seed=2, spread=0.2)
    Wq, Ws = weight(N, K)
    S = 0.05 * torch.randn((K // b, b, b), generator=gen(4), device="cuda")
    S = S - S.transpose(1, 2)
    R = torch.empty((K // b, b, b), dtype=BF16, device="cuda")
    pmoe.adapter_cayley(K // b, b, S, R, None)
    lin = DeviceLinearW8A8(Wq, Ws, rows, R=R)
    Y, dX = torch.empty((rows, N), dtype=BF16, device="cuda"), torch.empty((rows, K), dtype=BF16, device="cuda")
    dR = torch.full((K // b, b, b), math.nan, device="cuda")
    lin.forward(X, Y)
    lin.backward(X, dY, dX, dR)
    assert lin.status() == pmoe.PMOE_OK
    Xr = torch.empty_like(X)
    pmoe.adapter_apply(rows, K, b, X, R, Xr)
    near(Y, *product(*quantised(Xr), Wq, Ws))
    dxt, _ = product(*quantised(dY), Wq.T, Ws.T.contiguous())
    t = dxt.view(rows, K // b, b)
    want_dR = torch.einsum("rji,rjk->jik", X.to(D).view(rows, K // b, b), t)
    want_dX = torch.einsum("rjk,jik->rji", t, R.to(D)).reshape(rows, K)
    f = lambda x: x.to(D).cpu().numpy()
    scale = float(want_dX.abs().mean())
    assert_close(f(dX) / scale, f(want_dX) / scale, "dX")
    scale = float(want_dR.abs().mean())
    assert_close(f(dR) / scale, f(want_dR) / scale, "dR")
    lin.backward(X[:0], dY[:0], dX[:0], dR)
    assert (dR == 0).all()


def test_gradient_is_that_of_the_layer_without_rounding():
    """Differences of <dY, Y> along a direction: activations and upstream gradients that
    Q represents exactly, steps too, so that Q's rounding is no part of it."""
    rows, N, K = 64, 256, 384
    g = gen(9)
    small = lambda *s: torch.randint(-8, 9, s, generator=g, device="cuda").float()
    X, V, dY = small(rows, K), small(rows, K), small(rows, N)
    for t in (X, V, dY):
        t[:, ::128] = 14.0                    # 14 = 448 / 32: the scale is a power of two, whole numbers are exact
    V[:, ::128] = 0.0
    Wq, Ws = weight(N, K)
    lin = DeviceLinearW8A8(Wq, Ws, rows)
    Y = [torch.empty((rows, N), dtype=BF16, device="cuda") for _ in range(2)]
    for sign, y in zip((1, -1), Y):
        lin.forward((X + sign * (V > 0)).to(BF16), y)
    dX = torch.empty((rows, K), dtype=BF16, device="cuda")
    lin.backward(X.to(BF16), dY.to(BF16), dX)
    num = ((Y[0].to(D) - Y[1].to(D)) / 2 * dY.to(D)).sum()
    want = (dX.to(D) * (V > 0)).sum()
    slack = (EPS * (Y[0].to(D).abs() + Y[1].to(D).abs()) / 2 * dY.to(D).abs()).sum() + (EPS * dX.to(D).abs()).sum()
    assert abs(num - want) <= slack           # (each BF16 rounding by half a step)


@pytest.mark.parametrize("rows,N,K", [(1, 4096, 7168), (5, 24576, 272), (16, 1040, 2064), (700, 4096, 384)])
def test_layer_is_its_two_calls(rows, N, K):
    """The layer gives the same result bit for bit as fp8_quantize and fp8_gemm, NaN and
    infinity among the rows too."""
    X = activations(rows, K, seed=rows)
    if rows > 1:
        X[1, 5], X[rows - 1, K - 1] = math.nan, math.inf
    Wq, Ws = weight(N, K)
    KB = -(-K // 128)
    q, s = torch.empty((rows, K), dtype=torch.uint8, device="cuda"), torch.empty((KB, rows), device="cuda")
    ws = torch.zeros(pmoe.fp8_gemm_ws_bytes(rows, N, K), dtype=torch.uint8, device="cuda")
    Y, Z = (torch.empty((rows, N), dtype=BF16, device="cuda") for _ in range(2))
    lin = DeviceLinearW8A8(Wq, Ws, rows)
    lin.forward(X, Y)
    pmoe.fp8_quantize(rows, K, X, q, s)
    pmoe.fp8_gemm(rows, N, K, q, s, Wq, Ws, Z, ws)
    assert lin.status() == pmoe.PMOE_OK
    assert torch.equal(Y.isnan(), Z.isnan()) and torch.equal(Y.nan_to_num(), Z.nan_to_num())
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    if rows > 1:
        bad[1] = bad[rows - 1] = True
    assert torch.equal(Y.isnan().all(1), bad) and torch.equal(Y.isnan().any(1), bad)


def test_rows_do_not_depend_on_the_others():
    """Batches whose blocks are not shared out give the same rows bit for bit."""
    N, K = 4096, 1040
    X = activations(2000, K)
    lin = DeviceLinearW8A8(*weight(N, K), 2000)
    Y = torch.empty((2000, N), dtype=BF16, device="cuda")
    lin.forward(X, Y)
    for r in (slice(0, 700), slice(3, 1999)):
        Z = torch.empty((r.stop - r.start, N), dtype=BF16, device="cuda")
        lin.forward(X[r].contiguous(), Z)
        assert torch.equal(Z, Y[r])


def test_more_than_2_to_the_31_elements():
    rows, N, K = 300_011, 128, 7168
    X = torch.empty((rows, K), dtype=BF16, device="cuda").normal_()
    Wq, Ws = weight(N, K)
    lin = DeviceLinearW8A8(Wq, Ws, rows)
    Y, dX = torch.empty((rows, N), dtype=BF16, device="cuda"), torch.empty((rows, K), dtype=BF16, device="cuda")
    lin.forward(X, Y)
    lin.backward(X, Y, dX)
    assert lin.status() == pmoe.PMOE_OK
    for r in (slice(0, 50), slice(rows - 50, rows)):
        near(Y[r], *product(*quantised(X[r]), Wq, Ws))
        near(dX[r], *product(*quantised(Y[r]), Wq.T, Ws.T.contiguous()))


def test_streams_and_graphs():
    rows, N, K = 40, 1024, 2048               # (shared blocks: the workspace holds sums)
    X, dY = activations(rows, K, seed=1), activations(rows, N, seed=2)
    lin = DeviceLinearW8A8(*weight(N, K), rows)
    Y, dX = torch.empty((rows, N), dtype=BF16, device="cuda"), torch.empty((rows, K), dtype=BF16, device="cuda")

    def step():
        lin.forward(X, Y)
        lin.backward(X, dY, dX)

    step()
    ref = Y.clone(), dX.clone()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    st = torch.cuda.Stream()
    for run in (step, graphs[0].replay, graphs[1].replay, graphs[0].replay):
        Y.zero_(), dX.zero_()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            run()
        torch.cuda.current_stream().wait_stream(st)
        assert torch.equal(Y, ref[0]) and torch.equal(dX, ref[1])
    X.mul_(2)                                 # (a power of two: the same codes, doubled scales)
    graphs[1].replay()
    assert torch.equal(Y, ref[0] * 2) and torch.equal(dX, ref[1])


@pytest.mark.parametrize("rows", [9, 40, 5000])
def test_a_wait_that_runs_out_is_reported(rows):
    """Few rows, single CTAs and pairs: the first item's signal is withheld for 2 ms."""
    N, K = 2048, 1024
    X = activations(rows, K)
    lin = DeviceLinearW8A8(*weight(N, K), rows)
    Y, Z = (torch.empty((rows, N), dtype=BF16, device="cuda") for _ in range(2))
    lin.forward(X, Y)
    assert lin.status() == pmoe.PMOE_OK
    pmoe.pmoe_debug_expire_gemm_wait(2_000_000)
    lin.forward(X, Z)
    assert lin.status() == pmoe.PMOE_ERR_TIMEOUT
    lin.forward(X, Z)
    assert lin.status() == pmoe.PMOE_OK and torch.equal(Y, Z)
