"""The gate's choice where experts are alike or nearly so, bit for bit against the
order of the exact scores (the reference of test_gpu_gate, in FP64).
"""
import pytest
import torch

from precision_moe_adapter_gb300 import build, pmoe
from test_gpu_gate import D, call, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    pmoe.lib()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def check(l, b, k, kind="sigmoid", groups=1, top=1, gsum=2, rows=None):
    """The choice of the tokens in `rows` (None: all)."""
    idx, _ = call(l, b, k, kind=kind, groups=groups, top=top, gsum=gsum)
    # (+ 0: the reference's sorts see one zero)
    want, _ = reference(l + 0.0, b, k, kind, groups, top, gsum, True, 1.0)
    bad = (idx.long() != want).any(1)
    if rows is not None:
        bad &= rows
    assert not bad.any(), (int(bad.sum()), idx[bad][:2].tolist(), want[bad][:2].tolist())


# ---------------------------------------------------------------- zeros of both signs

def signs(shape, seed):
    """Zeros, half of them -0."""
    return torch.where(torch.rand(shape, generator=gen(seed), device="cuda") < 0.5, -0.0, 0.0)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E,k", [(2, 1), (20, 6), (64, 8), (384, 8), (384, 31), (384, 32), (1025, 8)])
def test_zeros_of_both_signs(E, k, bias, kind):
    """-0 and +0 are equal logits, whether they are all that there is or among others,
    few (ranked in one pass) or many (taken one at a time)."""
    T = 60
    l = signs((T, E), E + k)
    b = signs((E,), 5) if bias else None
    check(l, b, k, kind)
    g = gen(7)
    for share in (0.9, 0.3, 0.05):
        rest = torch.rand((T, E), generator=g, device="cuda") > share
        for sign in (-1.0, 1.0):
            check(torch.where(rest, sign * (0.5 + torch.rand((T, E), generator=g, device="cuda")), l), b, k, kind)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("gsum", [1, 2])
@pytest.mark.parametrize("E,groups,top,k", [(2, 2, 1, 1), (16, 8, 3, 2), (64, 8, 4, 8), (384, 4, 2, 8), (99, 9, 1, 3)])
def test_zeros_of_both_signs_in_groups(E, groups, top, k, gsum, bias, kind):
    T = 60
    l = signs((T, E), E + k)
    b = signs((E,), 5) if bias else None
    check(l, b, k, kind, groups, top, gsum)
    rest = torch.rand((T, E), generator=gen(7), device="cuda") < 0.6
    check(torch.where(rest, -1.0, l), b, k, kind, groups, top, gsum)
    if E == 2:
        l = torch.tensor([[-0.0, 0.0], [0.0, -0.0]], device="cuda")
        assert call(l, b, 1, kind=kind, groups=2, top=1, gsum=gsum)[0].tolist() == [[0], [0]]


# ---------------------------------------------------------------- equal experts beside close ones

def shuffled(l, seed):
    """Each row in an order of its own."""
    o = torch.rand(l.shape, generator=gen(seed), device="cuda").argsort(1)
    return l.gather(1, o)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("alike", [2, 3, 7, 40, 200])
@pytest.mark.parametrize("k", [1, 2, 8, 30, 31, 32])
def test_a_close_expert_behind_equal_ones(k, alike, kind):
    """The k-th place is taken among experts that are exactly alike and one whose score is
    1e-8 of itself above theirs: the same FP32 number, and behind them where its id is."""
    T, E = 300, 384
    row = torch.full((E,), -9.0)
    row[:k - 1] = torch.linspace(4.0, 1.0, k - 1)
    row[k - 1:k - 1 + alike] = 0.0
    row[k - 1 + alike] = 1e-8
    row = row.cuda()
    z = torch.zeros(E, device="cuda")
    check(shuffled(row.expand(T, E), k + alike), z, k, kind)
    row[k + alike] = -1e-8                     # and one below them
    check(shuffled(row.expand(T, E), k + alike + 1), z, k, kind)
    l = torch.full((1, E), -9.0, device="cuda")          # the least case, with its ids
    l[0, :alike] = 0.0
    l[0, E - 1] = 1e-8
    assert call(l, z, 1, kind=kind)[0].item() == E - 1


def nearly_alike(T, E, seed, share):
    """Logits that are 0 but for a share of values beside it (sums of two of them differ)."""
    g = gen(seed)
    near = torch.tensor([1e-8, -1.1e-8, 0.3e-8, 2.7e-8], device="cuda")
    l = near[torch.randint(0, 4, (T, E), generator=g, device="cuda")]
    return torch.where(torch.rand((T, E), generator=g, device="cuda") < share, l, 0.0)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E", [24, 128, 384, 1030])
@pytest.mark.parametrize("k", [1, 4, 8, 20, 24])
def test_experts_that_are_nearly_alike(k, E, kind):
    g = gen(E + k)
    steps = torch.randint(0, 3, (E,), generator=g, device="cuda") / 8.0
    for share in (0.005, 0.05, 0.5):
        l = nearly_alike(300, E, E + k, share)
        for b in (torch.zeros(E, device="cuda"), steps):
            check(l, b, k, kind)
        # few of them, the others far below
        check(torch.where(torch.rand(l.shape, generator=g, device="cuda") < 20 / E, l, -9.0), steps, k, kind)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("gsum", [1, 2])
@pytest.mark.parametrize("E,groups", [(64, 8), (64, 2), (384, 4), (96, 32)])
def test_groups_whose_experts_are_nearly_alike(E, groups, gsum, kind):
    """A group's best experts are alike to FP32, equal ones before one that is above them."""
    z = torch.zeros(E, device="cuda")
    for share in (0.02, 0.1, 0.5):
        for top in sorted({1, groups // 2}):
            check(nearly_alike(400, E, E + groups, share), z, 2, kind, groups, top, gsum)
    n = E // groups
    if n >= 8 and gsum == 1:                   # the least case: the best one behind two equal ones
        l = torch.full((1, E), -9.0, device="cuda")
        l[0, 0:2], l[0, 2], l[0, n] = 0.0, 1e-8, 0.5e-8
        assert call(l, z, 1, kind=kind, groups=groups, top=1, gsum=1)[0].item() == 2


# ---------------------------------------------------------------- groups of large biases

@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("spread", [0.0, 0.1])
@pytest.mark.parametrize("B", [4.0, 16.0, 1e3, 1e4])
def test_groups_of_biases_that_cancel(B, spread, kind):
    """Groups of two experts with biases of opposite sign: their sums are small beside what
    FP32 rounds away of each.  The first group out is moved beside the last one in."""
    T, G, top = 4000, 8, 4
    g = gen(int(B))
    l = torch.randn((T, 2 * G), generator=g, device="cuda")
    b = torch.tensor([B, -B], device="cuda").repeat(G) + spread * torch.randn(2 * G, generator=g, device="cuda")

    def sums(l):
        s = torch.sigmoid(l.to(D)) if kind == "sigmoid" else torch.softmax(l.to(D), 1)
        return (s + b.to(D)).view(T, G, 2).sum(2)

    gs = sums(l)
    order = torch.argsort(gs, dim=1, descending=True)
    a, o = order[:, top - 1:top], order[:, top:top + 1]
    delta = (2 * torch.rand((T, 1), generator=g, device="cuda", dtype=D) - 1) * B * 2.0 ** -23
    if kind == "sigmoid":
        want = gs.gather(1, a) + delta - (torch.sigmoid(l.to(D)) + b.to(D)).gather(1, 2 * o + 1) - b.to(D)[2 * o]
        l.scatter_(1, 2 * o, torch.log(want.clamp(0.001, 0.999) / (1 - want.clamp(0.001, 0.999))).float())
    else:                                      # (equal logits, but for a few units)
        l.scatter_(1, 2 * o, (l.gather(1, 2 * a) + delta).float())
        l.scatter_(1, 2 * o + 1, l.gather(1, 2 * a + 1))
    s = torch.sort(sums(l), dim=1, descending=True).values
    gap = (s[:, :-1] - s[:, 1:]).amin(1)
    # (a sum in FP64 is off by 2^-52 of B; tokens whose sums are within 100 times that are left out)
    clear = gap > 100 * 2.0 ** -52 * B
    assert clear.float().mean() > 0.9
    if kind == "sigmoid" and spread == 0:
        assert ((s[:, top - 1] - s[:, top]) < B * 2.0 ** -22).float().mean() > 0.3
    check(l, b, 4, kind, G, top, 2, rows=clear)
