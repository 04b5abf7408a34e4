"""The router's balance loss, per-expert counts and logit gradient on the GPU
against FP64.

Tolerances.  p = softmax in FP32: the argument's rounding (|l - max| <= 40
here, so 20 units in 2^24 of p), expf and the row's sum leave under 64 units
in 2^24; the means add up to about 200 positive terms in a row on top of
that: relative 2^-16.  The loss is a sum of positive products of two of
these: 2^-15.  A logit gradient's error is bounded by the same fractions of
its terms' magnitudes.  Counts are exact.
"""
import ctypes

import pytest
import torch

from precision_moe_adapter_gb300 import build, pmoe

D = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    pmoe.lib()


def make(T, E, k, seed=0, dup=False):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    logits = 2 * torch.randn((T, E), generator=g, device="cuda")
    idx = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32)
    if dup and k > 1:
        idx[:, 1] = idx[:, 0]
    w = torch.softmax(logits.gather(1, idx.long()), dim=1)
    dw = torch.randn((T, k), generator=g, device="cuda")
    return logits, idx.contiguous(), w.contiguous(), dw, g


def call(logits, idx, w, dw, valid=None, seq=None, S=1, gl=None, forward=True):
    T, E = logits.shape
    k = idx.shape[1]
    dm = pmoe.dims(T, 64, E, k, 64, 16)
    nan = float("nan")
    ws = torch.zeros(pmoe.moe_balance_ws_bytes(dm, S), dtype=torch.uint8, device="cuda")
    ws[256:] = 0xFF
    counts = torch.full((S, E), -7, dtype=torch.int32, device="cuda")
    ntok = torch.full((S,), -7, dtype=torch.int32, device="cuda")
    pmean, loss = torch.full((S, E), nan, device="cuda"), torch.full((S,), nan, device="cuda")
    dl = torch.full((T, E), nan, device="cuda")
    pmoe.moe_balance_forward(dm, logits, idx, valid, seq, S, counts, ntok, pmean, loss, ws)
    pmoe.moe_route_backward(dm, logits, idx, w, dw, valid, seq, S, counts, ntok, gl, dl, ws)
    return counts, ntok, pmean, loss, dl, pmoe.moe_query_status(ws)


def reference(logits, idx, w, dw, valid, bounds, gl):
    T, E = logits.shape
    k, S = idx.shape[1], len(bounds) - 1
    p = torch.softmax(logits.to(D), 1)
    counts = torch.zeros((S, E), dtype=torch.int64, device="cuda")
    ntok = torch.zeros(S, dtype=torch.int64, device="cuda")
    pmean = torch.zeros((S, E), dtype=D, device="cuda")
    dl, mag = torch.zeros((T, E), dtype=D, device="cuda"), torch.zeros((T, E), dtype=D, device="cuda")
    for s in range(S):
        r = torch.arange(bounds[s], bounds[s + 1], device="cuda")
        if valid is not None:
            r = r[valid[r] != 0]
        n = len(r)
        ntok[s] = n
        if n == 0:
            continue
        counts[s] = torch.bincount(idx[r].reshape(-1).long(), minlength=E)
        pmean[s] = p[r].mean(0)
        if gl is not None:
            a = gl[s].to(D) * E * counts[s].to(D) / (k * n * n)
            pa = (p[r] * a).sum(1, keepdim=True)
            dl[r] += p[r] * (a - pa)
            mag[r] += p[r] * (a.abs() + pa.abs())
    loss = E * (counts.to(D) / (k * ntok.clamp(min=1)[:, None]) * pmean).sum(1)
    if dw is not None:
        wd, dd = w.to(D), dw.to(D)
        dl.scatter_add_(1, idx.long(), wd * (dd - (wd * dd).sum(1, keepdim=True)))
        mag.scatter_add_(1, idx.long(), wd * (dd.abs() + (wd * dd).abs().sum(1, keepdim=True)))
    return counts, ntok, pmean, loss, dl, mag


def check(got, ref):
    assert torch.equal(got[0].long(), ref[0]) and torch.equal(got[1].long(), ref[1])
    assert torch.all((got[2].to(D) - ref[2]).abs() <= 2.0 ** -16 * ref[2])
    assert torch.all((got[3].to(D) - ref[3]).abs() <= 2.0 ** -15 * ref[3])
    assert torch.all((got[4].to(D) - ref[4]).abs() <= 2.0 ** -15 * ref[5])


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [
    (1, 1, 1), (1, 8, 2), (3, 2, 1), (64, 8, 2), (65, 33, 32), (700, 127, 4), (701, 128, 8), (33, 250, 3),
    (5000, 256, 8), (8192, 384, 8), (77, 500, 6), (300, 512, 8), (90, 1000, 5), (55, 1025, 32), (130, 4096, 8)])
def test_one_batch(T, E, k):
    logits, idx, w, dw, g = make(T, E, k, seed=T + E, dup=T % 2 == 1)
    gl = torch.tensor([0.3], device="cuda")
    got = call(logits, idx, w, dw, gl=gl)
    assert got[5] == pmoe.PMOE_OK
    check(got, reference(logits, idx, w, dw, None, [0, T], gl))
    # each term alone
    only = call(logits, idx, w, None, gl=gl)
    check(only, reference(logits, idx, w, None, None, [0, T], gl))
    only = call(logits, idx, w, dw, gl=None)
    check(only, reference(logits, idx, w, dw, None, [0, T], None))


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,bounds", [
    (50, 16, 2, [0, 0, 1, 1, 30, 50]), (2000, 64, 4, [0, 7, 8, 1000, 1001, 1999, 2000, 2000]),
    (9000, 130, 8, list(range(0, 9000, 300)) + [9000]), (64, 1500, 2, [0, 9, 40, 64]), (40, 32, 2, [3, 17, 30])])
def test_packed_sequences_with_padding(T, E, k, bounds):
    logits, idx, w, dw, g = make(T, E, k, seed=T)
    S = len(bounds) - 1
    valid = (torch.rand(T, generator=g, device="cuda") < 0.7).to(torch.uint8)
    valid[bounds[-2]:] = 0                                # a sequence of padding only
    seq = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    gl = torch.rand(S, generator=g, device="cuda") + 0.1
    got = call(logits, idx, w, dw, valid, seq, S, gl)
    assert got[5] == pmoe.PMOE_OK
    ref = reference(logits, idx, w, dw, valid, bounds, gl)
    check(got, ref)
    assert got[3][-1] == 0 and torch.all(got[2][-1] == 0)
    for a, b in zip(got[:5], call(logits, idx, w, dw, valid, seq, S, gl)[:5]):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,S", [(60, 33, 2000), (60, 250, 1500), (200, 4096, 300)])
def test_clusters_of_mostly_empty_sequences(T, E, S):
    """A CTA of an empty sequence has its share of the loss almost at once and
    hands it to the first CTA of its cluster, which must have started: many
    such clusters, the few tokens spread among them."""
    logits, idx, w, dw, g = make(T, E, 4, seed=S)
    cuts = torch.sort(torch.randint(0, T + 1, (9,), generator=g, device="cuda")).values.tolist()
    bounds = [0] * (S // 2) + [cuts[i * 9 // (S - S // 2)] for i in range(S - S // 2)] + [T]
    seq = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    gl = torch.rand(S, generator=g, device="cuda") + 0.1
    got = call(logits, idx, w, dw, None, seq, S, gl)
    assert got[5] == pmoe.PMOE_OK
    check(got, reference(logits, idx, w, dw, None, bounds, gl))
    for _ in range(5):
        for a, b in zip(got[:5], call(logits, idx, w, dw, None, seq, S, gl)[:5]):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_disabled_experts_and_bad_ids():
    logits, idx, w, dw, g = make(40, 24, 2)
    logits[:, 5] = -float("inf")
    logits[7] = -float("inf")                             # a token with no expert at all: p = 0
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[7] = False
    gl = torch.tensor([1.0], device="cuda")
    counts, ntok, pmean, loss, dl, st = call(logits, idx, w, None, gl=gl)
    assert st == pmoe.PMOE_OK and int(ntok[0]) == 40
    p = torch.softmax(logits[keep].to(D), 1).sum(0) / 40
    assert torch.all((pmean[0].to(D) - p).abs() <= 2.0 ** -16 * p) and pmean[0, 5] == 0
    assert torch.all(dl[7] == 0) and torch.all(dl[:, 5] == 0) and torch.isfinite(dl).all()
    # ids outside [0, E): left out of the counts and the gradient, reported
    logits, idx, w, dw, g = make(40, 24, 2)
    bad = idx.clone()
    bad[3, 0], bad[9, 1] = 24, -1
    counts, ntok, pmean, loss, dl, st = call(logits, bad, w, dw, gl=gl)
    assert st == pmoe.PMOE_ERR_BAD_INDEX
    assert int(counts.sum()) == 78 and torch.isfinite(dl).all()


@pytest.mark.gpu
def test_sequence_bounds_out_of_order_are_reported():
    logits, idx, w, dw, g = make(100, 16, 2)
    for b in ([0, 60, 40, 100], [0, 50, 101, 101], [-1, 50, 60, 100]):
        seq = torch.tensor(b, dtype=torch.int32, device="cuda")
        assert call(logits, idx, w, dw, None, seq, 3, torch.ones(3, device="cuda"))[5] == pmoe.PMOE_ERR_BAD_INDEX


@pytest.mark.gpu
def test_gradient_against_differences():
    """Both terms against central differences: the balance loss of the forward
    (the counts depend on idx alone), and sum w dw with w the softmax over the
    selected logits.  Step 1/64: the third-order term leaves under 1e-3, the
    FP32 loss (2^-22 of about 1, over a step of 1/32) about 1e-5."""
    T, E, k = 60, 24, 3
    logits, idx, w, dw, g = make(T, E, k)
    gl = torch.tensor([1.0], device="cuda")
    for use_gl, use_dw in ((gl, None), (None, dw)):
        dl = call(logits, idx, w, use_dw, gl=use_gl)[4].to(D)
        for _ in range(3):
            U = torch.randn((T, E), generator=g, device="cuda")
            if use_gl is not None:
                f = lambda l: call(l, idx, w, None, gl=gl)[3].to(D).sum()
            else:
                f = lambda l: (torch.softmax(l.to(D).gather(1, idx.long()), 1) * dw.to(D)).sum()
            num = (f(logits + U / 64) - f(logits - U / 64)) * 32
            ana = (dl * U.to(D)).sum()
            assert abs(num - ana) <= 2e-3 * dl.norm() * 5 + 5e-5


@pytest.mark.gpu
def test_routed_by_the_library():
    """moe_route's own logits, selection and weights go in as they are."""
    T, d, E, k = 200, 256, 48, 4
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    X = torch.randn((T, d), generator=g, device="cuda").to(torch.bfloat16)
    Wr, bias = 0.05 * torch.randn((d, E), generator=g, device="cuda"), torch.randn(E, generator=g, device="cuda")
    dm = pmoe.dims(T, d, E, k, 64, 16)
    ws = torch.zeros(pmoe.moe_workspace_bytes(dm, pmoe.OP_PERMUTE), dtype=torch.uint8, device="cuda")
    logits = torch.empty((T, E), device="cuda")
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), device="cuda")
    pmoe.moe_route(dm, X, Wr, bias, logits, idx, w, ws)
    dw = torch.randn((T, k), generator=g, device="cuda")
    gl = torch.tensor([0.01], device="cuda")
    got = call(logits, idx, w, dw, gl=gl)
    assert got[5] == pmoe.PMOE_OK
    check(got, reference(logits, idx, w, dw, None, [0, T], gl))


@pytest.mark.gpu
def test_no_tokens():
    e = torch.empty((0, 8), device="cuda")
    i, f = torch.empty((0, 2), dtype=torch.int32, device="cuda"), torch.empty((0, 2), device="cuda")
    counts, ntok, pmean, loss, dl, st = call(e, i, f, f, gl=torch.ones(1, device="cuda"))
    assert st == pmoe.PMOE_OK and int(counts.sum()) == 0 and int(ntok[0]) == 0 and float(loss[0]) == 0


def test_refusals():
    L = pmoe.lib()
    buf = ctypes.create_string_buffer(64)
    p = ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 16
    big, INV, WS = 1 << 40, pmoe.PMOE_ERR_INVALID_ARG, pmoe.PMOE_ERR_WORKSPACE
    dm = pmoe.dims(64, 64, 8, 2, 64, 16)
    assert pmoe.moe_balance_ws_bytes(dm, 1) > 256
    assert pmoe.moe_balance_ws_bytes(dm, 0) == 0
    assert pmoe.moe_balance_ws_bytes(pmoe.dims(64, 64, 8, 9, 64, 16), 1) == 0
    fwd, bwd = L.moe_balance_forward, L.moe_route_backward
    good = [dm, p, p, None, None, 1, p, p, p, p, p, big, None]
    for i, v in ((0, pmoe.dims(64, 64, 8, 9, 64, 16)), (1, None), (2, None), (5, 0), (5, 2), (6, None), (7, None),
                 (8, None), (9, None), (1, p + 4), (2, p + 4), (3, p + 1), (9, p + 4)):
        assert fwd(*(good[:i] + [v] + good[i + 1:])) == INV, (i, v)
    assert fwd(*(good[:10] + [None] + good[11:])) == WS
    assert fwd(*(good[:11] + [256] + good[12:])) == WS
    good = [dm, p, p, p, p, None, None, 1, p, p, p, p, p, big, None]
    for i, v in ((1, None), (2, None), (3, None), (7, 0), (7, 2), (8, None), (9, None), (11, None), (11, p + 4)):
        assert bwd(*(good[:i] + [v] + good[i + 1:])) == INV, (i, v)
    assert bwd(*(good[:4] + [None] + good[5:10] + [None] + good[11:])) == INV     # neither term
    assert bwd(*(good[:12] + [None] + good[13:])) == WS


def test_a_router_without_a_layer():
    """The sizes that the operators do not use are not looked at; those that
    they use are."""
    bare, full = pmoe.dims(64, 0, 8, 2, 0, 0), pmoe.dims(64, 64, 8, 2, 64, 16)
    assert pmoe.moe_balance_ws_bytes(bare, 3) == pmoe.moe_balance_ws_bytes(full, 3) > 256
    assert pmoe.moe_balance_ws_bytes(pmoe.dims(64, 100, 8, 2, 100, 7), 1) > 256
    for bad in ((-1, 8, 2), (64, 0, 2), (64, 4097, 2), (64, 8, 0), (64, 40, 33), (64, 8, 9), (1 << 28, 8, 5)):
        assert pmoe.moe_balance_ws_bytes(pmoe.dims(bad[0], 0, bad[1], bad[2], 0, 0), 1) == 0, bad
    L, buf = pmoe.lib(), ctypes.create_string_buffer(64)
    p = ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 16
    WS = pmoe.PMOE_ERR_WORKSPACE                          # (past the checks of the sizes)
    assert L.moe_balance_forward(bare, p, p, None, None, 1, p, p, p, p, p, 256, None) == WS
    assert L.moe_route_backward(bare, p, p, p, p, None, None, 1, p, p, p, p, p, 256, None) == WS
