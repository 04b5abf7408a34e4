"""The vocabulary head's losses on the GPU against FP64: token
log-probabilities and distillation from a teacher's top logits, forward and
backward.

Tolerances.  lse and the values come from FP32 sums of exact BF16 products.
A sum of d products in chunks of 512 columns: the tensor cores lose at most
about one unit in 2^24 of the running sum per 16 columns, 32 times a chunk,
and the FP32 additions of the chunks less than that again, so a logit is
within 2^-24 (32 + d / 512) sum |x w| <= 48 * 2^-24 sum |x w| of the exact
one; exp2, the sums of the softmax and the logarithm add a few units in 2^24
of |lse| and of 1.  Gradients are BF16 results of BF16 G: the layer's own
tolerance for BF16 outputs (tests/helpers.py).
"""
import math

import numpy as np
import pytest
import torch

from helpers import assert_close
from precision_moe_adapter_gb300 import build, pmoe
from precision_moe_adapter_gb300.head import DeviceHead

pytestmark = pytest.mark.gpu
D = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    pmoe.lib()


def make(T, d, V, seed=0, lean=8.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    W = (torch.randn((V, d), generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    X = torch.randn((T, d), generator=g, device="cuda")
    X += lean * torch.rand((T, 1), generator=g, device="cuda") * W[y].float() / (4e-4 * d)
    up = torch.randn(T, generator=g, device="cuda")
    return X.to(torch.bfloat16), W, y.to(torch.int32), up, g


def reference(X, W, scale, Q, Qx, g, sign):
    """FP64: lse, the value sum_v Q (logQ - logp) or logp, dX, dW for the
    target distribution Q [T, V] (rows may be empty)."""
    z = scale * (X.to(D) @ W.to(D).T)
    lse = torch.logsumexp(z, 1)
    logp = z - lse[:, None]
    G = (logp.exp() * Q.sum(1, keepdim=True) - Q) * (sign * scale * g.to(D))[:, None]
    value = Qx - sign * (Q * logp).sum(1)
    return lse, value, G @ W.to(D), G.T @ X.to(D)


def logit_bound(X, W, scale):
    return scale * 48 * 2.0 ** -24 * (X.to(D).abs() @ W.to(D).abs().T).amax(1)


def run_logprob(X, W, y, up, scale, dW=True):
    T = X.shape[0]
    h = DeviceHead(W, T, scale=scale)
    logp, lse = (torch.full((T,), float("nan"), device="cuda") for _ in range(2))
    dX = torch.full_like(X, float("nan"))
    dWt = torch.full_like(W, float("nan")) if dW else None
    h.logprob(X, y, logp, lse)
    h.logprob_backward(X, y, lse, up, dX, dWt)
    torch.cuda.synchronize()
    return h, logp, lse, dX, dWt


def check_values(X, W, scale, lse, value, rlse, rvalue):
    b = logit_bound(X, W, scale) + 2.0 ** -20 * (1 + rlse.abs())
    assert torch.all((lse.to(D) - rlse).abs() <= b), ((lse.to(D) - rlse).abs() / b).max()
    b = 2 * b + 2.0 ** -20 * (1 + rvalue.abs())
    assert torch.all((value.to(D) - rvalue).abs() <= b), ((value.to(D) - rvalue).abs() / b).max()


def check_grad(got, ref, what):
    assert_close(got.float().cpu().numpy(), ref.cpu().numpy(), what)


@pytest.mark.parametrize("T,d,V,scale", [
    (1, 64, 1, 1.0), (1, 64, 2, 1.0), (1, 2048, 4099, 1.0), (2, 128, 127, 0.5), (7, 576, 129, 2.0),
    (127, 256, 128, 1.0), (128, 512, 1000, 1.0), (129, 1088, 257, 1 / 0.7), (300, 256, 5003, 1.0),
    (513, 192, 3001, 1.0), (64, 8192, 600, 1.0), (2100, 64, 640, 1.0), (260, 2048, 20011, 1.0)])
def test_logprob(T, d, V, scale):
    X, W, y, up, g = make(T, d, V, seed=T + d + V)
    y = torch.where(torch.rand(T, generator=g, device="cuda") < 0.2, torch.full_like(y, -1), y)
    h, logp, lse, dX, dW = run_logprob(X, W, y, up, scale)
    assert h.status() == pmoe.PMOE_OK
    Q = torch.zeros((T, V), dtype=D, device="cuda")
    r = torch.nonzero(y >= 0)[:, 0]
    Q[r, y[r].long()] = 1
    rlse, rv, rdX, rdW = reference(X, W, scale, Q, 0.0, up, -1.0)
    check_values(X, W, scale, lse, logp, rlse, rv)
    assert torch.all(logp[y < 0] == 0) and torch.all(dX[y < 0] == 0)
    check_grad(dX, rdX, "dX")
    check_grad(dW, rdW, "dW")


@pytest.mark.parametrize("T,d,V,K,scale", [
    (1, 64, 3, 1, 1.0), (5, 64, 100, 7, 0.5), (130, 256, 1003, 64, 0.5), (33, 128, 256, 256, 1.0),
    (300, 320, 5003, 33, 2.0), (16, 2048, 300, 129, 1.0)])
def test_distill(T, d, V, K, scale):
    X, W, y, up, g = make(T, d, V, seed=T + K)
    perm = torch.rand((T, V), generator=g, device="cuda").argsort(1)[:, :K].to(torch.int32)
    ids = perm.contiguous()
    t = 2 * torch.randn((T, K), generator=g, device="cuda")
    gone = torch.rand((T, K), generator=g, device="cuda") < 0.2
    ids[gone] = -1
    if T > 2:
        ids[1] = -1                                   # a row without entries
        t[2, K // 2] = -math.inf                      # an entry of probability zero
    if T > 4 and K > 3:
        ids[3] = ids[3, 0].clamp(min=0)               # one id many times
        ids[4] = V - 1 - torch.arange(K, device="cuda", dtype=torch.int32).clamp(max=V - 1)
    h = DeviceHead(W, T, K=K, scale=scale)
    loss, lse = (torch.full((T,), float("nan"), device="cuda") for _ in range(2))
    dX, dW = torch.full_like(X, float("nan")), torch.full_like(W, float("nan"))
    h.distill(X, ids, t, loss, lse)
    h.distill_backward(X, ids, t, lse, up, dX, dW)
    assert h.status() == pmoe.PMOE_OK
    td = (scale * t.to(D)).masked_fill(ids < 0, -math.inf)
    q = torch.nan_to_num(torch.softmax(td, 1))
    Q = torch.zeros((T, V), dtype=D, device="cuda").scatter_add_(1, ids.clamp(min=0).long(), q)
    rlse, rv, rdX, rdW = reference(X, W, scale, Q, torch.xlogy(q, q).sum(1), up, 1.0)
    check_values(X, W, scale, lse, loss, rlse, rv)
    if T > 2:
        assert loss[1] == 0 and torch.all(dX[1] == 0)
    check_grad(dX, rdX, "dX")
    check_grad(dW, rdW, "dW")


@pytest.mark.parametrize("T,d,V", [(8192, 64, 70001), (4100, 1216, 66001)])
def test_vocabulary_in_several_pieces(T, d, V):
    """T = 8192 tokens bound a piece to 32768 entries: three pieces, the last
    one ragged; at T = 4100 two pieces, with dX's tiles cut among the SMs."""
    X, W, y, up, _ = make(T, d, V)
    h, logp, lse, dX, dW = run_logprob(X, W, y, up, 1.0)
    assert h.status() == pmoe.PMOE_OK
    rdW = torch.zeros((V, d), dtype=D, device="cuda")
    for a in range(0, T, 1024):
        r = slice(a, min(a + 1024, T))
        n = r.stop - a
        Q = torch.zeros((n, V), dtype=D, device="cuda")
        Q[torch.arange(n, device="cuda"), y[r].long()] = 1
        rlse, rv, rdX, dw = reference(X[r], W, 1.0, Q, 0.0, up[r], -1.0)
        rdW += dw
        check_values(X[r], W, 1.0, lse[r], logp[r], rlse, rv)
        check_grad(dX[r], rdX, "dX")
    check_grad(dW, rdW, "dW")


def test_gradient_against_differences():
    """dL/dX along random sign directions against central differences of the
    forward.  X lies on a grid of 1/64 below 2, so X +- 1/64 is exact in
    BF16; the step's third-order term and the FP32 forward leave under 1%."""
    T, d, V = 37, 128, 1003
    X, W, y, up, g = make(T, d, V)
    W = (W.float() * 8).to(torch.bfloat16)
    X = ((X.float().clamp(-1.9, 1.9) * 64).round() / 64).to(torch.bfloat16)
    h, _, _, dX, dW = run_logprob(X, W, y, up, 1.0)
    logp, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")

    def L(x):
        h.logprob(x, y, logp, lse)
        return logp.to(D) * up.to(D)

    for _ in range(3):
        U = torch.randint(0, 2, (T, d), generator=g, device="cuda").float() * 2 - 1
        num = (L((X.float() + U / 64).to(torch.bfloat16)) - L((X.float() - U / 64).to(torch.bfloat16))) * 32
        ana = (dX.to(D) * U.to(D)).sum(1)
        assert (num - ana).norm() <= 1e-2 * ana.norm()


def test_a_token_does_not_depend_on_the_batch():
    T, d, V = 700, 2048, 20011
    X, W, y, up, _ = make(T, d, V)
    full = run_logprob(X, W, y, up, 1.0, dW=False)
    for n in (1, 7, 128, 129, 300):
        part = run_logprob(X[:n].clone(), W, y[:n].clone(), up[:n].clone(), 1.0, dW=False)
        assert torch.equal(part[1], full[1][:n]) and torch.equal(part[2], full[2][:n]), n


def test_runs_are_identical_and_use_the_given_stream():
    T, d, V = 333, 256, 9001
    X, W, y, up, _ = make(T, d, V)
    ref = run_logprob(X, W, y, up, 1.0)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        again = run_logprob(X, W, y, up, 1.0)
    for a, b in zip(ref[1:], again[1:]):
        assert torch.equal(a, b)


def test_no_tokens_and_ids_out_of_range():
    W = torch.ones((50, 64), dtype=torch.bfloat16, device="cuda")
    e = torch.empty(0, device="cuda")
    h = DeviceHead(W, 0)
    dW = torch.full_like(W, 3.0)
    X = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    h.logprob(X, e.to(torch.int32), e, e)
    h.logprob_backward(X, e.to(torch.int32), e, e, X, dW)
    assert torch.all(dW == 0) and h.status() == pmoe.PMOE_OK
    # a target past the vocabulary is ignored and reported
    X, W, y, up, _ = make(4, 64, 50)
    y[2] = 50
    h, logp, lse, dX, _ = run_logprob(X, W, y, up, 1.0)
    assert h.status() == pmoe.PMOE_ERR_BAD_INDEX
    assert logp[2] == 0 and torch.all(dX[2] == 0) and torch.all(torch.isfinite(lse))
    h = DeviceHead(W, 4, K=2)
    ids = torch.tensor([[0, 1], [50, 3], [2, -1], [2 ** 31 - 1, 60]], dtype=torch.int32, device="cuda")
    t = torch.zeros((4, 2), device="cuda")
    loss, lse = torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    h.distill(X, ids, t, loss, lse)
    assert h.status() == pmoe.PMOE_ERR_BAD_INDEX
    assert loss[3] == 0 and np.isfinite(loss.cpu().numpy()).all()


@pytest.mark.parametrize("T,d,V", [(64, 64, 40), (300, 256, 5003), (2570, 2048, 2700), (2001, 192, 263),
                                   (4100, 1024, 600)])
def test_large_entries_of_the_gradient_keep_16_bits(T, d, V):
    """Confident tokens whose target is another one: G is about +g at one
    entry and -g at the target, next to nothing elsewhere (1 - p <= 2%).
    Kept to 16 bits, its rounding is 2^-8 of the outputs' own BF16 rounding,
    so the gradients are as close to the exact ones as those rounded to BF16
    (5% allowed); with 8 bits the error would be about 1.4 times that."""
    X, W, y, up, g = make(T, d, V, lean=0.0)
    y = torch.arange(T, device="cuda") * 7 % V
    at = (y + 1 + torch.randint(0, V - 1, (T,), generator=g, device="cuda")) % V
    X = (0.05 * X.float() + 14 * W[at].float() / (4e-4 * d)).to(torch.bfloat16)
    y = y.to(torch.int32)
    h, logp, lse, dX, dW = run_logprob(X, W, y, up, 1.0)
    Q = torch.zeros((T, V), dtype=D, device="cuda")
    Q[torch.arange(T, device="cuda"), y.long()] = 1
    rlse, rv, rdX, rdW = reference(X, W, 1.0, Q, 0.0, up, -1.0)
    for got, ref in ((dX, rdX), (dW, rdW)):
        best = (ref.to(torch.bfloat16).to(D) - ref).norm()
        assert (got.to(D) - ref).norm() <= 1.05 * best


def test_ignored_tokens_may_hold_anything():
    """NaN and infinities in the hidden states of ignored tokens reach neither
    the other tokens nor their own rows of dX."""
    T, d, V, K = 300, 128, 1003, 4
    X, W, y, up, g = make(T, d, V)
    off = torch.rand(T, generator=g, device="cuda") < 0.3
    y = torch.where(off, torch.full_like(y, -1), y)
    Xn = X.clone()
    Xn[off] = float("nan")
    Xn[off.nonzero()[0, 0], ::2] = float("inf")
    upn = torch.where(off, torch.full_like(up, float("nan")), up)
    ref = run_logprob(X, W, y, up, 1.0, dW=False)
    got = run_logprob(Xn, W, y, upn, 1.0, dW=False)
    assert torch.equal(got[1], ref[1]) and torch.equal(got[2][~off], ref[2][~off])
    assert torch.equal(got[3], ref[3]) and torch.all(got[3][off] == 0)
    ids = torch.randint(0, V, (T, K), generator=g, device="cuda").to(torch.int32)
    ids[off] = -1
    t = torch.randn((T, K), generator=g, device="cuda")
    out = []
    for x, u in ((X, up), (Xn, upn)):
        h = DeviceHead(W, T, K=K)
        loss, lse, dX = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(X)
        h.distill(x, ids, t, loss, lse)
        h.distill_backward(x, ids, t, lse, u, dX)
        out.append((loss, dX))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    assert torch.all(out[1][0][off] == 0) and torch.all(out[1][1][off] == 0)


@pytest.mark.parametrize("T,d,V,K", [(1, 2048, 4000, 0), (40, 7168, 300, 0), (300, 512, 5003, 0), (33, 2048, 1003, 5)])
def test_confident_tokens_keep_fp32_accuracy(T, d, V, K):
    """Where the target holds most of the probability its logit is 10 to 20,
    and the tensor cores' biased sums would be off by 1e-5 of it.  The value
    is the difference of two FP32 numbers of that size (half a unit each, and
    the FP32 dot product's few units): within 2^-21 (1 + |lse|).  p - 1 has
    the same absolute error, so a token's row of dX is within 2^-21 (1 + |lse|)
    of |g s| times the rows of W that carry it, besides the BF16 rounding."""
    X, W, y, up, g = make(T, d, V, seed=5, lean=0.0)
    X = (0.05 * X.float() + (10 + 10 * torch.rand((T, 1), generator=g, device="cuda")) * W[y.long()].float()
         / W[y.long()].float().square().sum(1, keepdim=True)).to(torch.bfloat16)
    Q = torch.zeros((T, V), dtype=D, device="cuda")
    if K:
        ids = torch.cat([y[:, None], torch.randint(0, V, (T, K - 1), generator=g, device="cuda")], 1).to(torch.int32).contiguous()
        t = torch.randn((T, K), generator=g, device="cuda")
        t[:, 0] += 9
        q = torch.softmax(t.to(D), 1)
        Q.scatter_add_(1, ids.long(), q)
        h = DeviceHead(W, T, K=K)
        val, lse, dX = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(X)
        h.distill(X, ids, t, val, lse)
        h.distill_backward(X, ids, t, lse, up, dX)
        rlse, rv, rdX, _ = reference(X, W, 1.0, Q, torch.xlogy(q, q).sum(1), up, 1.0)
    else:
        _, val, lse, dX, _ = run_logprob(X, W, y, up, 1.0, dW=False)
        Q[torch.arange(T, device="cuda"), y.long()] = 1
        rlse, rv, rdX, _ = reference(X, W, 1.0, Q, 0.0, up, -1.0)
    tol = 2.0 ** -21 * (1 + rlse.abs())
    assert torch.all((lse.to(D) - rlse).abs() <= tol), ((lse.to(D) - rlse).abs() / tol).max()
    assert torch.all((val.to(D) - rv).abs() <= tol), ((val.to(D) - rv).abs() / tol).max()
    err = (dX.to(D) - rdX).norm(dim=1)
    row = up.to(D).abs() * W.to(D).norm(dim=1).max()
    assert torch.all(err <= 2.0 ** -8 * rdX.norm(dim=1) + 2 * tol * row), (err / row).max()


@pytest.mark.parametrize("K", [0, 3])
def test_upstream_coefficients_that_underflow(K):
    """Tokens whose factor is so small that a share of it is no FP32 number
    have no large entries; the other tokens' gradients are what they are with
    a zero there, and runs are identical."""
    T, d, V = 300, 512, 5003
    X, W, y, up, g = make(T, d, V)
    tiny = torch.rand(T, generator=g, device="cuda") < 0.3
    up = torch.where(tiny, torch.full_like(up, 1.4e-45), up)
    up[tiny.nonzero()[::2, 0]] *= -3
    zero = torch.where(tiny, torch.zeros_like(up), up)
    ids = torch.randint(0, V, (T, max(K, 1)), generator=g, device="cuda").to(torch.int32)
    t = torch.randn((T, max(K, 1)), generator=g, device="cuda")
    h = DeviceHead(W, T, K=K)
    val, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    out = []
    for u in (up, zero, up):
        dX, dW = torch.full_like(X, float("nan")), torch.full_like(W, float("nan"))
        if K:
            h.distill(X, ids, t, val, lse)
            h.distill_backward(X, ids, t, lse, u, dX, dW)
        else:
            h.logprob(X, y, val, lse)
            h.logprob_backward(X, y, lse, u, dX, dW)
        out.append((dX, dW))
    assert h.status() == pmoe.PMOE_OK
    assert torch.equal(out[0][0], out[2][0]) and torch.equal(out[0][1], out[2][1])
    assert torch.equal(out[0][0][~tiny], out[1][0][~tiny])
    assert torch.all(out[0][0][tiny].float().abs() < 1e-38)
    assert torch.equal(out[0][1].float(), out[1][1].float())


@pytest.mark.parametrize("V,bad", [(1003, 500), (1025, 1024), (5003, 0)])
@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_a_vocabulary_row_that_is_not_a_number_shows(V, bad, what):
    """A NaN (or infinite) row of the head makes every token's sum NaN (or
    infinite): no token's value or lse may look like a number then, its own
    target's logit being finite, whether or not the row shares its unit of
    128 with others."""
    T, d = 70, 128
    X, W, y, up, g = make(T, d, V)
    y = torch.where(y == bad, (y + 7) % V, y)
    W[bad] = what
    logp, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    h = DeviceHead(W, T, K=2)
    h.logprob(X, y, logp, lse)
    assert not torch.isfinite(logp).any() and not torch.isfinite(lse).any()
    ids = torch.stack([y, (y + 1 + (y + 1 == bad)) % V], 1).to(torch.int32).contiguous()
    h.distill(X, ids, torch.tensor([[3.0, 0.0]], device="cuda").repeat(T, 1), logp, lse)
    assert not torch.isfinite(logp).any() and not torch.isfinite(lse).any()


@pytest.mark.parametrize("T,d,V,K,scale", [(40, 2048, 4000, 0, 1.0), (33, 512, 1003, 0, 1 / 0.7), (300, 7168, 640, 0, 1.0),
                                           (64, 256, 129, 0, 2.0), (50, 2048, 1003, 1, 1.0)])
def test_confident_values_are_accurate_relative_to_themselves(T, d, V, K, scale):
    """-log p = log1p(sum over the others of exp(s (z_v - z_y))).  Each
    exponent is off by at most the errors of its two logits and a unit in 2^24
    of its size (here under 40); exp2, the sums and log1p add some units in
    2^24.  All are relative errors of the sum, so of the value however small
    it is: from about e^-2 down to e^-30."""
    X, W, y, up, g = make(T, d, V, seed=11, lean=0.0)
    Wy = W[y.long()].float()
    X = (0.05 * X.float() + (6 + 26 * torch.rand((T, 1), generator=g, device="cuda")) / scale * Wy
         / Wy.square().sum(1, keepdim=True)).to(torch.bfloat16)
    h = DeviceHead(W, T, K=K, scale=scale, backward=False)
    val, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    if K:
        h.distill(X, y[:, None].contiguous(), torch.zeros((T, 1), device="cuda"), val, lse)
    else:
        h.logprob(X, y, val, lse)
        val = -val
    z = scale * (X.to(D) @ W.to(D).T)
    rest = z.scatter(1, y[:, None].long(), -math.inf) - z.gather(1, y[:, None].long())
    ref = torch.log1p(rest.exp().sum(1))
    tol = 2 * logit_bound(X, W, scale) + 64 * 2.0 ** -24
    err = (val.to(D) - ref).abs() / ref
    assert torch.all(err <= tol), (err / tol).max()


@pytest.mark.parametrize("T,d,V,K", [(300, 128, 1003, 0), (700, 192, 9001, 0), (300, 256, 5003, 4), (40, 64, 300, 4)])
def test_ignored_tokens_do_not_reach_the_heads_gradient(T, d, V, K):
    """NaN and infinities in the hidden states of ignored tokens, the first one
    among them, leave dW what it is with zeros there."""
    X, W, y, up, g = make(T, d, V)
    off = torch.rand(T, generator=g, device="cuda") < 0.3
    off[0] = True
    y = torch.where(off, torch.full_like(y, -1), y)
    ids = torch.randint(0, V, (T, max(K, 1)), generator=g, device="cuda").to(torch.int32)
    ids[off] = -1
    t = torch.randn((T, max(K, 1)), generator=g, device="cuda")
    h = DeviceHead(W, T, K=K)
    val, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    out = []
    for fill in (0.0, math.nan, math.inf):
        Xf = X.clone()
        Xf[off] = fill
        dX, dW = torch.full_like(X, float("nan")), torch.full_like(W, float("nan"))
        if K:
            h.distill(Xf, ids, t, val, lse)
            h.distill_backward(Xf, ids, t, lse, up, dX, dW)
        else:
            h.logprob(Xf, y, val, lse)
            h.logprob_backward(Xf, y, lse, up, dX, dW)
        out.append((dX, dW))
    assert torch.isfinite(out[0][1].float()).all()
    for dX, dW in out[1:]:
        assert torch.equal(dX, out[0][0]) and torch.equal(dW, out[0][1])


@pytest.mark.parametrize("T,d,V,K", [(300, 256, 5003, 0), (1100, 512, 9001, 0), (64, 64, 40, 0), (600, 256, 9001, 6)])
def test_gradient_of_the_head_alone(T, d, V, K):
    """dW without dX (hidden states that take no gradient) is the dW of both."""
    X, W, y, up, g = make(T, d, V)
    y = torch.where(torch.rand(T, generator=g, device="cuda") < 0.2, torch.full_like(y, -1), y)
    ids = torch.randint(0, V, (T, max(K, 1)), generator=g, device="cuda").to(torch.int32)
    t = 3 * torch.randn((T, max(K, 1)), generator=g, device="cuda")
    h = DeviceHead(W, T, K=K)
    val, lse, dX = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(X)
    both, alone = torch.full_like(W, float("nan")), torch.full_like(W, float("nan"))
    if K:
        h.distill(X, ids, t, val, lse)
        h.distill_backward(X, ids, t, lse, up, dX, both)
        h.distill_backward(X, ids, t, lse, up, None, alone)
    else:
        h.logprob(X, y, val, lse)
        h.logprob_backward(X, y, lse, up, dX, both)
        h.logprob_backward(X, y, lse, up, None, alone)
    assert h.status() == pmoe.PMOE_OK
    assert torch.isfinite(alone.float()).all() and torch.equal(both, alone)


def test_targets_in_one_block_of_the_vocabulary():
    """Every token has the same target, so that one row of dW takes a remainder
    from each of them: 1024 extra K steps, from a list that does not fit its
    builder's shared memory.  The sums are of one sign, so what the tensor cores
    truncate would add up: at most 128 MMAs a run lose 2^-24 of it each, and the
    4096 of the extra steps the same of the last of 32 runs, which is 2^-17 of
    the whole each.  The mean over d elements of their BF16 rounding (at most 2^-9
    each; the columns' factors of 1 to 2 spread the sums over many BF16 steps)
    has a standard deviation of 2^-9 / sqrt(3 d), of which 5 are allowed."""
    T, d, V = 65536, 8192, 4096
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    X = torch.randn((T, d), generator=g, device="cuda", dtype=torch.bfloat16).abs_() + 0.5
    X *= torch.exp2(torch.arange(d, device="cuda") / d).to(torch.bfloat16)
    W = torch.randn((V, d), generator=g, device="cuda", dtype=torch.bfloat16).mul_(0.002)
    y = torch.full((T,), 300, dtype=torch.int32, device="cuda")
    up = 0.5 + torch.rand(T, generator=g, device="cuda")
    h, logp, lse, _, dW = run_logprob(X, W, y, up, 1.0)
    assert h.status() == pmoe.PMOE_OK
    ref = torch.zeros(d, dtype=D, device="cuda")
    for a in range(0, T, 4096):
        r = slice(a, a + 4096)
        ref += (up[r].to(D) * (1 - logp[r].to(D).exp())) @ X[r].to(D)
    bias = ((dW[300].to(D) - ref) / ref).mean().abs()
    assert bias <= 2 * 2.0 ** -17 + 5 * 2.0 ** -9 / math.sqrt(3 * d), bias


def _distill_in_parts(X, W, ids, t, up, scale, dW):
    T, V = X.shape[0], W.shape[0]
    h = DeviceHead(W, T, K=ids.shape[1], scale=scale)
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dX = torch.full_like(X, float("nan"))
    dWt = torch.full_like(W, float("nan")) if dW else None
    h.distill(X, ids, t, loss, lse)
    h.distill_backward(X, ids, t, lse, up, dX, dWt)
    assert h.status() == pmoe.PMOE_OK
    rdW = torch.zeros((V, W.shape[1]), dtype=D, device="cuda")
    for a in range(0, T, 512):
        r = slice(a, min(a + 512, T))
        q = torch.nan_to_num(torch.softmax((scale * t[r].to(D)).masked_fill(ids[r] < 0, -math.inf), 1))
        Q = torch.zeros((r.stop - a, V), dtype=D, device="cuda").scatter_add_(1, ids[r].clamp(min=0).long(), q)
        rlse, rv, rdX, w = reference(X[r], W, scale, Q, torch.xlogy(q, q).sum(1), up[r], 1.0)
        rdW += w
        check_values(X[r], W, scale, lse[r], loss[r], rlse, rv)
        check_grad(dX[r], rdX, "dX")
    if dW:
        check_grad(dWt, rdW, "dW")


@pytest.mark.parametrize("T,d,V,K,top,dW", [
    (700, 256, 8009, 16, 0.0, True), (1030, 128, 10007, 40, 6.0, True),          # pairs of CTAs, lists
    (8192, 64, 70001, 9, 4.0, True), (4100, 320, 66001, 64, 3.0, False)])        # several pieces
def test_distill_as_training_runs_it(T, d, V, K, top, dW):
    """Entries and anchors anywhere in the vocabulary, so in every piece and in
    both halves of a pair's tile; some tokens have one confident entry, some
    none, some repeat an id."""
    X, W, y, up, g = make(T, d, V, seed=K)
    ids = torch.randint(0, V, (T, K), generator=g, device="cuda").to(torch.int32)
    ids[:, 0] = y
    ids[::7, 1] = ids[::7, 2]
    ids[::11, K // 2:] = -1
    ids[5::50] = -1
    t = torch.randn((T, K), generator=g, device="cuda")
    t[:, 0] += top
    _distill_in_parts(X, W, ids.contiguous(), t, up, 0.7, dW)


def test_distill_of_a_token_does_not_depend_on_the_batch():
    T, d, V, K = 700, 512, 20011, 12
    X, W, y, up, g = make(T, d, V)
    ids = torch.randint(0, V, (T, K), generator=g, device="cuda").to(torch.int32)
    ids[:, 0] = y
    t = 2 * torch.randn((T, K), generator=g, device="cuda")
    t[::2, 0] += 6
    out = []
    for n in (T, 1, 7, 128, 129, 300):
        h = DeviceHead(W, n, K=K, backward=False)
        loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        h.distill(X[:n].clone(), ids[:n].clone(), t[:n].clone(), loss, lse)
        assert torch.equal(loss, (out or [loss])[0][:n]) and torch.equal(lse, (out or [0, lse])[1][:n]), n
        out = out or [loss, lse]


@pytest.mark.parametrize("T,d,V", [(40, 256, 300), (300, 512, 5003), (700, 256, 8009)])
def test_a_wait_that_runs_out_is_reported(T, d, V):
    """One accumulator-full signal of every product is withheld and waits end
    after 2 ms: the call ends, reports PMOE_ERR_TIMEOUT, and the next one is
    what it was.  Single CTAs with whole remainders, with lists, and pairs."""
    X, W, y, up, g = make(T, d, V)
    ref = run_logprob(X, W, y, up, 1.0)
    h, (logp, lse, dX, dW) = ref[0], [torch.empty_like(t) for t in ref[1:]]
    assert h.status() == pmoe.PMOE_OK
    pmoe.pmoe_debug_expire_gemm_wait(2_000_000)
    h.logprob(X, y, logp, lse)
    assert h.status() == pmoe.PMOE_ERR_TIMEOUT
    h.logprob(X, y, logp, lse)
    assert h.status() == pmoe.PMOE_OK
    assert torch.equal(logp, ref[1]) and torch.equal(lse, ref[2])
    for x, w in ((dX, dW), (dX, None), (None, dW)):
        pmoe.pmoe_debug_expire_gemm_wait(2_000_000)
        h.logprob_backward(X, y, lse, up, x, w)
        assert h.status() == pmoe.PMOE_ERR_TIMEOUT
        h.logprob_backward(X, y, lse, up, x, w)
        assert h.status() == pmoe.PMOE_OK
        assert x is None or torch.equal(x, ref[3])
        assert w is None or torch.equal(w, ref[4])


def test_inputs_rewritten_between_calls():
    """Calls behind one another on a stream, each behind kernels that have just
    rewritten the hidden states, the targets and the head in place: every call
    sees its own."""
    T, d, V = 130, 256, 1003
    sets = [make(T, d, V, seed=i)[:4] for i in range(4)]
    want = [run_logprob(*s, 1.0)[1:] for s in sets]
    X, W, y, up = (t.clone() for t in sets[0])
    h = DeviceHead(W, T)
    got = []
    for i in range(24):
        for t, new in zip((X, W, y, up), sets[i % 4]):
            t.copy_(new)
        logp, lse, dX, dW = (torch.empty_like(t) for t in want[0])
        h.logprob(X, y, logp, lse)
        h.logprob_backward(X, y, lse, up, dX, dW)
        got.append((logp, lse, dX, dW))
    for i, g in enumerate(got):
        for a, b in zip(g, want[i % 4]):
            assert torch.equal(a, b), i


def test_absent_teacher_entries_may_hold_anything():
    """The logits of absent entries are not looked at, whatever they hold."""
    T, d, V, K = 70, 128, 1003, 9
    X, W, y, up, g = make(T, d, V)
    ids = torch.randint(0, V, (T, K), generator=g, device="cuda").to(torch.int32)
    gone = torch.rand((T, K), generator=g, device="cuda") < 0.4
    gone[3] = True
    ids[gone] = -1
    t = 2 * torch.randn((T, K), generator=g, device="cuda")
    out = []
    for fill in (0.0, math.nan, math.inf, -math.inf, 3e38):
        tf = torch.where(gone, torch.full_like(t, fill), t)
        h = DeviceHead(W, T, K=K, scale=2.0)
        loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        dX, dW = torch.empty_like(X), torch.empty_like(W)
        h.distill(X, ids, tf, loss, lse)
        h.distill_backward(X, ids, tf, lse, up, dX, dW)
        out.append((loss, lse, dX, dW))
        assert h.status() == pmoe.PMOE_OK
    assert torch.isfinite(out[0][0]).all() and out[0][0][3] == 0
    for o in out[1:]:
        for a, b in zip(o, out[0]):
            assert torch.equal(a, b)
