"""The scored gate on the GPU against FP64: the choice bit for bit, weights and
gradients within FP32's error.

Tolerances.  A score is an exponential (2 units of 2^-23), for softmax a sum of at
most 4096 positive terms (133 roundings in a row), a sum or a division more: under
2^-16 of itself; so are the weights, quotients of such sums.  The gradient's
terms take four products and quotients more: 2^-15 of their magnitudes.
"""
import math

import pytest
import torch

from precision_moe_adapter_gb300 import build, pmoe

pytestmark = pytest.mark.gpu
D = torch.float64
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    pmoe.lib()


def scores(l, kind):
    if kind == "sigmoid":
        return torch.sigmoid(l)
    m = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(m == -INF, torch.zeros_like(m), m))
    z = e.sum(1, keepdim=True)
    return torch.where(z > 0, e / z, torch.zeros_like(e))


def reference(logits, bias, k, kind, groups, top, gsum, renorm, factor, dw=None):
    """idx, w and (with dw) the gradient and its terms' magnitude, in FP64."""
    l = logits.to(D)
    T, E = l.shape
    s = scores(l, kind)
    c = s + bias.to(D) if bias is not None else l.clone()      # without a bias: the order of the logits
    c = torch.where(l == -INF, torch.full_like(c, -INF), c)
    if top < groups:
        v = torch.where(l == -INF, torch.zeros_like(c), c if bias is not None else s)
        cg = c.view(T, groups, -1)
        o = torch.sort(cg, dim=2, descending=True, stable=True).indices[:, :, :gsum]
        gs = cg.max(2).values if gsum == 1 else v.view(T, groups, -1).gather(2, o).sum(2)
        gs = torch.where(cg.max(2).values == -INF, torch.full_like(gs, -INF), gs)
        best = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :top]
        keep = torch.zeros((T, groups), dtype=torch.bool, device=l.device).scatter_(1, best, True)
        keep = keep.repeat_interleave(E // groups, 1)
    else:
        keep = torch.ones((T, E), dtype=torch.bool, device=l.device)
    # (an expert of a dropped group stands behind those at -inf of a kept one)
    first = torch.sort(c, dim=1, descending=True, stable=True).indices
    kept = keep.gather(1, first)
    idx = first.gather(1, torch.sort(kept.to(torch.int8), dim=1, descending=True, stable=True).indices)[:, :k]
    sel = s.gather(1, idx)
    den = sel.sum(1, keepdim=True) + 1e-20 if renorm else torch.ones((T, 1), dtype=D, device=l.device)
    w = factor * sel / den
    if dw is None:
        return idx, w
    dw = dw.to(D)
    u = factor * dw / den
    au = u.abs()
    if renorm:
        u = u - (u * sel).sum(1, keepdim=True) / den
        au = au + (au * sel).sum(1, keepdim=True) / den
    dl, mag = torch.zeros_like(l), torch.zeros_like(l)
    if kind == "sigmoid":
        j = sel * torch.sigmoid(-l.gather(1, idx))
        dl.scatter_(1, idx, u * j), mag.scatter_(1, idx, au * j)
    else:
        dl.scatter_(1, idx, u * sel), mag.scatter_(1, idx, au * sel)
        dl -= s * (u * sel).sum(1, keepdim=True)
        mag += s * (au * sel).sum(1, keepdim=True)
    return idx, w, dl, mag


def inputs(T, E, seed=0, scale=1.5, bias=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    l = scale * torch.randn((T, E), generator=g, device="cuda")
    b = 0.1 * torch.randn(E, generator=g, device="cuda") if bias else None
    return l, b, g


def call(l, b, k, kind="sigmoid", groups=1, top=1, gsum=2, renorm=True, factor=1.0, dw=None, accumulate=None):
    T, E = l.shape
    g = pmoe.gate(T, E, k, kind, groups, top, gsum, renorm, factor)
    idx = torch.full((T + 2, k), -9, dtype=torch.int32, device="cuda")
    w = torch.full((T + 2, k), math.nan, device="cuda")
    pmoe.moe_gate_forward(g, l, b, idx, w)
    assert (idx[T:] == -9).all() and w[T:].isnan().all()        # rows behind the last token
    if dw is None:
        return idx[:T], w[:T]
    dl = torch.full((T + 1, E), math.nan, device="cuda")
    if accumulate is not None:
        dl[:T] = accumulate
    pmoe.moe_gate_backward(g, l, idx, dw, dl, accumulate is not None)
    assert dl[T:].isnan().all()
    return idx[:T], w[:T], dl[:T]


def compare(l, b, k, seed=0, **kw):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 77)
    dw = torch.randn((l.shape[0], k), generator=g, device="cuda")
    args = dict(kind="sigmoid", groups=1, top=1, gsum=2, renorm=True, factor=1.0)
    args.update(kw)
    idx, w, dl = call(l, b, k, dw=dw, **args)
    ridx, rw, rdl, mag = reference(l, b, k, args["kind"], args["groups"], args["top"], args["gsum"],
                                   args["renorm"], args["factor"], dw)
    assert torch.equal(idx.long(), ridx), (idx.long() != ridx).nonzero()[:5]
    # (1e-37: scores below FP32's normal range)
    assert torch.all((w.to(D) - rw).abs() <= 2.0 ** -16 * rw.abs() + 1e-37)
    assert torch.all((dl.to(D) - rdl).abs() <= 2.0 ** -15 * mag + 1e-37)
    base = torch.randn(l.shape, generator=g, device="cuda")
    acc = call(l, b, k, dw=dw, accumulate=base, **args)[2]
    assert torch.all((acc.to(D) - base.to(D) - rdl).abs() <= 2.0 ** -15 * mag + 2.0 ** -23 * (base.abs() + rdl.abs()) + 1e-37)
    return idx, w, dl


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 1), (5, 2, 2), (64, 8, 2), (33, 31, 7), (9, 32, 32), (130, 33, 8),
                                   (200, 60, 6), (77, 127, 9), (500, 128, 8), (65, 255, 4), (1000, 256, 8),
                                   (300, 384, 8), (400, 256, 24), (300, 384, 31), (100, 511, 16), (50, 1000, 8), (20, 1024, 32), (10, 1025, 8),
                                   (7, 4096, 32), (3, 4095, 5)])
def test_sizes(T, E, k, bias, kind):
    l, b, _ = inputs(T, E, seed=T + E, bias=bias)
    compare(l, b, k, kind=kind, renorm=E % 2 == 0, factor=2.5)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E,groups,top,gsum,k", [
    (16, 16, 5, 2, 5), (16, 16, 16, 1, 4), (16, 8, 1, 1, 2), (60, 6, 3, 1, 6), (60, 3, 1, 2, 8), (96, 32, 20, 2, 32),
    (256, 8, 4, 2, 8), (256, 8, 3, 1, 8), (384, 4, 2, 2, 8), (1000, 5, 2, 2, 9), (99, 9, 4, 2, 11), (33, 33 // 3, 7, 2, 3),
    (1024, 31 + 1, 9, 2, 8), (4096, 16, 4, 2, 8), (210, 30, 7, 2, 4), (2, 2, 1, 2, 1)])
def test_groups(E, groups, top, gsum, k, bias, kind):
    l, b, _ = inputs(301, E, seed=E + groups, bias=bias)
    compare(l, b, k, kind=kind, groups=groups, top=top, gsum=gsum, renorm=groups % 2 == 0, factor=1.5)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups", [1, 4])
def test_many_tokens_and_equal_logits(kind, groups):
    """Logits of few values: ties everywhere, between experts and between groups."""
    l, b, _ = inputs(4000, 64, seed=5)
    l = (l * 2).round() / 2
    compare(l, None, 6, kind=kind, groups=groups, top=max(1, groups // 2))
    compare(l, torch.zeros_like(b), 6, kind=kind, groups=groups, top=max(1, groups // 2))
    compare(l, (b * 8).round() / 8, 6, kind=kind, groups=groups, top=max(1, groups // 2))
    compare(torch.zeros_like(l), None, 6, kind=kind, groups=groups, top=max(1, groups // 2))
    idx, _, _ = compare(torch.zeros_like(l), torch.zeros_like(b), 6, kind=kind, groups=groups, top=max(1, groups // 2))
    assert torch.equal(idx, torch.arange(6, dtype=torch.int32, device="cuda").expand_as(idx))


@pytest.mark.parametrize("k", [1, 8, 20, 31, 32])
def test_close_calls_between_experts(k):
    """Pairs of experts whose score + bias is the same to a few units of FP32 or
    less, at every place of the order."""
    T, E = 2000, 128
    l, b, g = inputs(T, E, seed=k, scale=1.0)
    c = torch.sigmoid(l.to(D)) + b.to(D)
    perm = torch.argsort(c, dim=1, descending=True)
    for a in range(0, 40, 2):                  # the second of each pair of neighbours is moved beside the first
        i, j = perm[:, a:a + 1], perm[:, a + 1:a + 2]
        s = c.gather(1, i) - b.to(D)[j[:, 0]][:, None]
        ok = (s > 0.01) & (s < 0.99)
        lj = torch.log(s / (1 - s)).float()
        l.scatter_(1, j, torch.where(ok, lj, l.gather(1, j)))
    idx, _, _ = compare(l, b, k, seed=k)
    c2 = torch.sort(torch.sigmoid(l.to(D)) + b.to(D), dim=1, descending=True).values
    assert ((c2[:, :k] - c2[:, 1:k + 1]) < 2.0 ** -22).float().mean() > 0.2


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("gsum", [1, 2])
def test_close_calls_between_groups(bias, gsum):
    T, E, G = 2000, 64, 4
    l, b, g = inputs(T, E, seed=3, scale=1.0, bias=bias)
    bb = b.to(D) if bias else torch.zeros(E, dtype=D, device="cuda")
    c = torch.sigmoid(l.to(D)) + bb
    v, o = torch.sort(c.view(T, G, -1), dim=2, descending=True)
    gs = v[:, :, :gsum].sum(2)
    order = torch.argsort(gs, dim=1, descending=True)
    g1, g2 = order[:, 1:2], order[:, 2:3]       # the last one in and the first one out, of two
    best = o[:, :, 0].gather(1, g2) + g2 * (E // G)
    want = gs.gather(1, g1) - (v[:, :, 1].gather(1, g2) if gsum == 2 else 0)
    s = want - bb[best[:, 0]][:, None]
    ok = (s > 0.01) & (s < 0.99)
    l.scatter_(1, best, torch.where(ok, torch.log(s / (1 - s)).float(), l.gather(1, best)))
    compare(l, b, 8, groups=G, top=2, gsum=gsum)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2)])
def test_experts_that_cannot_be_chosen(groups, top, bias, kind):
    l, b, g = inputs(400, 48, seed=9, bias=bias)
    l[torch.rand(l.shape, generator=g, device="cuda") < 0.6] = -INF
    l[:20] = -INF                              # nothing is left
    l[20:40, 3:] = -INF                        # fewer than k are left
    l[40:60, :47] = -INF
    l[60:80, 12:] = -INF                       # one group
    for renorm in (True, False):
        idx, w, dl = compare(l, b, 6, kind=kind, groups=groups, top=top, renorm=renorm)
        assert not w.isnan().any() and not dl.isnan().any()
        assert (w[:20] == 0).all()
        assert (torch.sort(idx, 1).values.diff(dim=1) > 0).all()       # k different experts all the same


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_large_logits(kind):
    """Scores that are 1 or 0 to FP32, and far apart."""
    l, b, _ = inputs(300, 64, seed=4, scale=30.0)
    l = l.clamp(-80, 34)
    compare(l, b, 8, kind=kind, factor=2.5)
    compare(l, None, 8, kind=kind, renorm=False)
    compare(l - 60, b, 8, kind=kind)


def test_finite_differences():
    for kind in ("sigmoid", "softmax"):
        for renorm in (True, False):
            l, b, g = inputs(6, 12, seed=8)
            dw = torch.randn((6, 3), generator=g, device="cuda")
            idx, _, dl = call(l, b, 3, kind=kind, renorm=renorm, factor=1.7, dw=dw)
            mag = reference(l, b, 3, kind, 1, 1, 2, renorm, 1.7, dw)[3]

            def value(x):
                s = scores(x, kind).gather(1, idx.long())
                return (1.7 * s / (s.sum(1, keepdim=True) + 1e-20 if renorm else 1.0) * dw.to(D)).sum(1)

            for e in range(12):
                h = torch.zeros((6, 12), dtype=D, device="cuda")
                h[:, e] = 1e-5
                num = (value(l.to(D) + h) - value(l.to(D) - h)) / 2e-5
                # the difference's error: h^2 times a third derivative of at most about 10
                assert torch.all((num - dl[:, e].to(D)).abs() <= 1e-8 + 2.0 ** -15 * mag[:, e])


def test_gradient_takes_any_ids():
    """The same expert twice adds up; an id that is none takes no part."""
    T, E, k = 40, 20, 4
    l, _, g = inputs(T, E, seed=11)
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda").to(torch.int32)
    idx[:, 1] = idx[:, 0]
    idx[::3, 2] = -1
    idx[1::3, 3] = E
    dw = torch.randn((T, k), generator=g, device="cuda")
    for kind in ("sigmoid", "softmax"):
        dl = torch.full((T, E), math.nan, device="cuda")
        pmoe.moe_gate_backward(pmoe.gate(T, E, k, kind), l, idx, dw, dl)
        x = l.to(D).requires_grad_()
        s = scores(x, kind)
        ok = (idx >= 0) & (idx < E)
        sel = torch.where(ok, s.gather(1, idx.long().clamp(0, E - 1)), torch.zeros((), dtype=D, device="cuda"))
        want = torch.autograd.grad((sel / (sel.sum(1, keepdim=True) + 1e-20) * dw.to(D)).sum(), x)[0]
        assert torch.all((dl.to(D) - want).abs() <= 2.0 ** -15 * (4 * dw.abs().amax(1, keepdim=True)))


def test_a_token_does_not_depend_on_the_batch():
    l, b, _ = inputs(777, 256, seed=2)
    kw = dict(groups=8, top=4, factor=2.5)
    idx, w = call(l, b, 8, **kw)
    for r in (slice(0, 1), slice(5, 38), slice(700, 777)):
        i2, w2 = call(l[r].contiguous(), b, 8, **kw)
        assert torch.equal(i2, idx[r]) and torch.equal(w2, w[r])


def test_more_than_2_to_the_31_logits():
    T, E, k = (1 << 21) + 5, 1024, 2
    l = torch.empty((T, E), device="cuda").normal_()
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), device="cuda")
    g = pmoe.gate(T, E, k)
    pmoe.moe_gate_forward(g, l, None, idx, w)
    r = slice(T - 100, T)
    ridx, rw = reference(l[r], None, k, "sigmoid", 1, 1, 2, True, 1.0)
    assert torch.equal(idx[r].long(), ridx)
    assert torch.all((w[r].to(D) - rw).abs() <= 2.0 ** -16 * rw)
    dw = torch.ones((T, k), device="cuda")
    dw[:, 0] = 0
    dl = torch.empty((T, E), device="cuda")
    pmoe.moe_gate_backward(g, l, idx, dw, dl)
    _, _, want, mag = reference(l[r], None, k, "sigmoid", 1, 1, 2, True, 1.0, dw[r])
    assert torch.all((dl[r].to(D) - want).abs() <= 2.0 ** -15 * mag)


def test_streams_and_graphs():
    l, b, g = inputs(500, 384, seed=1)
    dw = torch.randn((500, 8), generator=g, device="cuda")
    gate = pmoe.gate(500, 384, 8, factor=2.5)
    idx, w = torch.empty((500, 8), dtype=torch.int32, device="cuda"), torch.empty((500, 8), device="cuda")
    dl = torch.empty((500, 384), device="cuda")

    def step():
        pmoe.moe_gate_forward(gate, l, b, idx, w)
        pmoe.moe_gate_backward(gate, l, idx, dw, dl)

    step()
    ref = [idx.clone(), w.clone(), dl.clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    st = torch.cuda.Stream()
    for run in (step, graph.replay):
        for t in (idx, w, dl):
            t.zero_()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            run()
        torch.cuda.current_stream().wait_stream(st)
        assert torch.equal(idx, ref[0]) and torch.equal(w, ref[1]) and torch.equal(dl, ref[2])
    l.copy_(l.flip(0))
    graph.replay()
    ridx, rw = reference(l, b, 8, "sigmoid", 1, 1, 2, True, 2.5)
    assert torch.equal(idx.long(), ridx)
