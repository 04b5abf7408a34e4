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
