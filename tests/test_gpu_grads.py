"""The global gradient norm and clipping on the GPU against FP64.

Tolerances.  Squares are summed in FP64, those of 8 vectors of a thread in FP32 before
(at most 8 + 3 roundings of 2^-24 of the sum in a row): the norm is off by at most 5.5 of
these, and by its own rounding: under 2^-21.  coef takes the norm's error and one rounding, the product
one more: 2^-21 for f32, half a step of BF16 (2^-8) beside it for bf16.
"""
import math

import pytest
import torch

from precision_moe_adapter_gb300 import build, pmoe
from precision_moe_adapter_gb300.grads import GradList

pytestmark = pytest.mark.gpu
F32, BF16, D = torch.float32, torch.bfloat16, torch.float64
TOL = {F32: 2.0 ** -21, BF16: 2.0 ** -8 + 2.0 ** -21}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    pmoe.lib()


def padded(n, dtype, seed=0, scale=1.0, fill=-7.0):
    """(a buffer, a view of its first n elements): what lies behind stays as it is."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    buf = torch.full((n + 64,), fill, dtype=dtype, device="cuda")
    buf[:n] = (torch.randn(n, generator=g, device="cuda") * scale).to(dtype)
    return buf, buf[:n]


def reference(gs, max_norm):
    norm = math.sqrt(sum(float((g.to(D) ** 2).sum()) for g in gs))
    return norm, min(1.0, max_norm / (norm + 1e-6))


def check(bufs, gs, outs, norm, want_norm, coef):
    assert abs(norm - want_norm) <= 2.0 ** -21 * want_norm
    for g, o in zip(gs, outs):
        want = g.to(D) * coef
        assert torch.all((o.to(D) - want).abs() <= TOL[g.dtype] * want.abs())
    for b, o in zip(bufs, outs):
        assert torch.all(b[o.numel():] == -7.0)


SIZES = [0, 1, 2, 3, 4, 5, 7, 8, 9, 31, 1023, 8191, 8192, 8193, 16383, 16384, 16385, 100003]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", SIZES)
def test_one_tensor(n, dtype):
    gb, g = padded(n, dtype, seed=n)
    ob, o = padded(n, dtype, fill=-7.0, scale=0.0)
    norm = torch.empty(1, device="cuda")
    want, coef = reference([g], 0.25 * math.sqrt(n + 1))
    GradList([g], out=[o]).clip(0.25 * math.sqrt(n + 1), norm)
    check([gb, ob], [g], [o], float(norm), want, coef)
    norm2 = torch.empty(1, device="cuda")
    GradList([g]).norm(norm2)
    assert torch.equal(norm, norm2)


@pytest.mark.parametrize("order", [0, 1, 2])
def test_many_tensors_in_place(order):
    """Every size beside every other one, empty ones at both ends and in runs."""
    ns = {0: [0, 0] + SIZES + [0, 0, 0, 5, 0], 1: SIZES[::-1], 2: [3] * 700 + [0] * 50 + [9000] * 40}[order]
    both = [padded(n, F32 if (i + order) % 3 else BF16, seed=i) for i, n in enumerate(ns)]
    bufs, gs = [b for b, _ in both], [g for _, g in both]
    before = [g.clone() for g in gs]
    norm = torch.empty(1, device="cuda")
    lst = GradList(gs)
    want, coef = reference(before, 1.0)
    lst.clip(1.0, norm)
    check(bufs, before, gs, float(norm), want, coef)
    # the norm is now the limit's (each rounding moves it by at most that of its type)
    lst.norm(norm)
    assert abs(float(norm) - 1.0) <= 2.0 ** -8


def test_a_norm_below_the_limit_changes_nothing():
    gs = [padded(n, t, seed=n)[1] for n in (5, 8193, 40000) for t in (F32, BF16)]
    outs = [torch.zeros_like(g) for g in gs]
    before = [g.clone() for g in gs]
    norm = torch.empty(1, device="cuda")
    want, _ = reference(gs, 1.0)
    GradList(gs).clip(2 * want, norm)
    GradList(gs, out=outs).clip(2 * want, norm)
    assert all(torch.equal(a, b) and torch.equal(a, o) for a, b, o in zip(gs, before, outs))
    GradList(gs).clip(want * (1 - 2.0 ** -18), norm)
    assert any(not torch.equal(a, b) for a, b in zip(gs, before))


def test_no_gradients():
    norm = torch.full((1,), 5.0, device="cuda")
    GradList([]).clip(1.0, norm)
    assert float(norm) == 0.0
    GradList([torch.empty(0, device="cuda")]).norm(norm)
    assert float(norm) == 0.0


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-22, 1e-15, 1e15, 1e19, 1e25, 1e37])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_squares_outside_the_range_of_fp32(scale, dtype):
    gs = [padded(n, dtype, seed=n, scale=scale)[1] for n in (3, 20000)]
    gs.append(torch.zeros(9000, dtype=dtype, device="cuda"))
    norm = torch.empty(1, device="cuda")
    want, _ = reference(gs, 1.0)
    GradList(gs).norm(norm)
    if want < 3e38:
        assert abs(float(norm) - want) <= 2.0 ** -21 * want + 2.0 ** -149
    else:
        assert float(norm) == math.inf
    before = [g.clone() for g in gs]
    m = want / 2 if want / 2 > 1e-30 and want < 1e38 else 1.0
    want, coef = reference(gs, m)
    GradList(gs).clip(m, norm)
    for a, b in zip(gs, before):
        w = b.to(D) * coef                      # (2^-134: half a step of BF16's least numbers)
        assert torch.all((a.to(D) - w).abs() <= TOL[dtype] * w.abs() + (2.0 ** -134 if dtype == BF16 else 2.0 ** -149))


def test_large_and_small_side_by_side():
    """A vector with one large element among tiny ones, and vectors of each kind."""
    g = torch.full((100000,), 1e-25, device="cuda")
    g[::7] = 1e-3
    g[50001] = 1e20
    norm = torch.empty(1, device="cuda")
    GradList([g]).norm(norm)
    want, _ = reference([g], 1.0)
    assert abs(float(norm) - want) <= 2.0 ** -21 * want


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_nan_or_an_infinity(bad):
    a, b = padded(20000, F32, seed=1)[1], padded(77, BF16, seed=2)[1]
    a[12345] = bad
    x, y = a.clone(), b.clone()
    norm = torch.empty(1, device="cuda")
    GradList([a, b]).clip(1.0, norm)
    if math.isnan(bad):
        assert math.isnan(float(norm)) and a.isnan().all() and b.isnan().all()
    else:
        assert float(norm) == math.inf
        assert a[12345].isnan() and torch.all(b == 0) and torch.all(a[:12345] == 0)
    # nothing is kept: the next call is clean
    a.copy_(x), b.copy_(y)
    a[12345] = 0.5
    want, _ = reference([a, b], 1.0)
    GradList([a, b]).norm(norm)
    assert abs(float(norm) - want) <= 2.0 ** -21 * want


def test_more_than_2_to_the_31_elements():
    n = 2 ** 31 + 12345
    big = torch.zeros(n, dtype=BF16, device="cuda")
    big[-3:] = 3.0
    big[2 ** 31 + 5] = 4.0
    small = torch.ones(5, device="cuda")
    norm = torch.empty(1, device="cuda")
    GradList([big, small]).clip(1.0, norm)
    want = math.sqrt(3 * 9 + 16 + 5)
    assert abs(float(norm) - want) <= 2.0 ** -21 * want
    c = 1 / (want + 1e-6)
    assert abs(float(big[-1]) - 3 * c) <= 2.0 ** -8 * 3 * c and abs(float(big[2 ** 31 + 5]) - 4 * c) <= 2.0 ** -8 * 4 * c
    assert abs(float(small[4]) - c) <= 2.0 ** -21 * c


def test_runs_are_identical_on_any_stream_and_in_graphs():
    gs = [padded(n, t, seed=n)[1] for n in (70001, 5, 300007) for t in (F32, BF16)]
    outs = [torch.empty_like(g) for g in gs]
    lst, norm = GradList(gs, out=outs), torch.empty(1, device="cuda")
    lst.clip(1.0, norm)
    ref, rn = [o.clone() for o in outs], norm.clone()

    def same():
        ok = torch.equal(norm, rn) and all(torch.equal(a, b) for a, b in zip(outs, ref))
        for o in outs:
            o.zero_()
        norm.zero_()
        return ok

    assert same()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        lst.clip(1.0, norm)
    torch.cuda.current_stream().wait_stream(st)
    assert same()
    graphs = []
    for _ in range(2):                       # two graphs share the list's workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lst.clip(1.0, norm)
        graphs.append(g)
    for i in (0, 1, 1, 0):
        graphs[i].replay()
        assert same()
    # the values at replay count, not those at capture
    gs[0].mul_(3)
    want, _ = reference(gs, 1.0)
    graphs[1].replay()
    assert abs(float(norm) - want) <= 2.0 ** -21 * want
