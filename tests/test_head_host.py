"""The head's entry points on the host: sizes and refusals, before any
device work."""
import ctypes

import pytest
import torch

from precision_moe_adapter_gb300 import build, head, pmoe

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def L():
    build.build()
    return pmoe.lib()


def test_workspace_bytes(L):
    f = lambda *a, op=pmoe.HEAD_FORWARD: pmoe.head_workspace_bytes(pmoe.head_dims(*a), op)
    assert f(1, 64, 1) > 256
    assert f(8, 2048, 131072) >= 256 + 8 * 1024 * 8      # one pair per token and 128 entries
    # the backward holds G of one piece of the vocabulary, never of all of it
    b = f(8192, 7168, 131072, op=pmoe.HEAD_BACKWARD)
    assert 512 << 20 <= b < (512 << 20) + 2 * 8192 * 7168 * 4
    for bad in ((1, 63, 10), (1, 0, 10), (1, 8256, 10), (-1, 64, 10), (1, 64, 0), (1, 64, 10, 257),
                (1, 64, 10, -1), (1, 64, (1 << 24) + 1)):
        assert f(*bad) == 0, bad
    assert pmoe.head_workspace_bytes(pmoe.head_dims(1, 64, 1), 2) == 0


def test_refusals(L):
    buf = ctypes.create_string_buffer(256)
    p = ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 16
    big = 1 << 40
    h = pmoe.head_dims(4, 64, 100, 2)
    INV, WS = pmoe.PMOE_ERR_INVALID_ARG, pmoe.PMOE_ERR_WORKSPACE
    lf, lb, df, db = (L.head_logprob_forward, L.head_logprob_backward, L.head_distill_forward,
                      L.head_distill_backward)
    assert lf(h, p, p, 1.0, p, p, p, None, 0, None) == WS
    assert lf(h, p, p, 1.0, p, p, p, p, 256, None) == WS
    assert lf(h, p, p, 1.0, p, p, p, p + 4, big, None) == WS
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert lf(h, p, p, scale, p, p, p, p, big, None) == INV
    assert lf(pmoe.head_dims(4, 100, 100), p, p, 1.0, p, p, p, p, big, None) == INV
    for i in (1, 2, 4, 5, 6):                            # a missing or misaligned pointer
        for bad in (None, p + 4):
            args = [h, p, p, 1.0, p, p, p, p, big, None]
            args[i] = bad
            assert lf(*args) == INV, (i, bad)
    assert lb(h, p, p, 1.0, p, p, p, None, None, p, big, None) == INV    # no gradient asked for
    assert lb(h, p, p, 1.0, p, p, p, p + 2, None, p, big, None) == INV
    assert lb(h, p, p, 1.0, p, p, p, p, p + 2, p, big, None) == INV
    assert lb(h, p, p, 1.0, p, None, p, p, None, p, big, None) == INV
    assert df(h, p, p, 1.0, p, None, p, p, p, big, None) == INV
    assert df(pmoe.head_dims(4, 64, 100, 0), p, p, 1.0, p, p, p, p, p, big, None) == INV
    assert db(h, p, p, 1.0, p, p, p, None, p, None, p, big, None) == INV
    # no tokens: nothing to do
    assert lf(pmoe.head_dims(0, 64, 100), None, None, 1.0, None, None, None, p, big, None) == pmoe.PMOE_OK


def test_device_head_checks(monkeypatch):
    monkeypatch.setattr(pmoe, "moe_clear_status", lambda ws, stream=None: None)
    W = torch.zeros((100, 64), dtype=BF16)
    with pytest.raises(ValueError):
        head.DeviceHead(W[:, ::2], 4)                    # not contiguous
    with pytest.raises(TypeError):
        head.DeviceHead(W.float(), 4)
    with pytest.raises(ValueError):
        head.DeviceHead(W[:, :32].contiguous(), 4)       # d % 64
    h = head.DeviceHead(W, 4, K=2, backward=False)
    X, f = torch.zeros((4, 64), dtype=BF16), torch.zeros(4)
    y = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError):
        h.logprob(X, y.long(), f, f)
    with pytest.raises(ValueError):
        h.logprob(X[:3], y, f, f)
    with pytest.raises(TypeError):
        h.logprob(X, y, f.double(), f)
    with pytest.raises(ValueError):
        h.distill(X, torch.zeros((4, 3), dtype=torch.int32), torch.zeros((4, 3)), f, f)
    with pytest.raises(RuntimeError):
        h.logprob_backward(X, y, f, f, X)


def test_calls_on_another_device_are_refused(monkeypatch):
    """The library launches on the current device: a head (or a layer's router)
    whose tensors are on another one says so before it looks at anything else."""
    from precision_moe_adapter_gb300 import layer
    monkeypatch.setattr(pmoe, "moe_clear_status", lambda ws, stream=None: None)
    h = head.DeviceHead(torch.zeros((100, 64), dtype=BF16), 4, K=2)
    h.device = torch.device("cuda", 1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for call in (lambda: h.logprob(None, None, None, None), lambda: h.distill(None, None, None, None, None),
                 lambda: h.logprob_backward(None, None, None, None, None),
                 lambda: h.distill_backward(None, None, None, None, None, None), h.status):
        with pytest.raises(RuntimeError, match="cuda:1"):
            call()
    with pytest.raises(RuntimeError, match="cuda:1"):
        layer.check_current(torch.device("cuda", 1))
    L = layer.DeviceLayer.__new__(layer.DeviceLayer)
    L.cfg, L.device = None, torch.device("cuda", 1)
    with pytest.raises(RuntimeError, match="cuda:1"):
        L._balance_args(None, None, None, 1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    layer.check_current(torch.device("cuda", 1))
    layer.check_current(torch.device("cpu"))


@pytest.mark.parametrize("T,d,V", [(32768, 7168, 163840), (20000, 7168, 131072), (8192, 7168, 163840), (4096, 2048, 131072),
                                   (1, 8192, 131072), (64, 2048, 32000), (100000, 512, 163840)])
def test_backward_workspace_is_what_the_header_says(L, T, d, V):
    """G of a piece, 6 bytes per hidden value, the parts of the cut tiles (fewer
    than 152 tiles of 64 KB, or 76 of 256 KB, times at most a few tens), about
    8 KB a token: not a whole FP32 dX for every part of a cut tile."""
    G = max(512 << 20, T * 512)
    n = pmoe.head_workspace_bytes(pmoe.head_dims(T, d, V), pmoe.HEAD_BACKWARD)
    assert n <= G + 6 * T * d + (192 << 20) + 8600 * T
