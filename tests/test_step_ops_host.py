"""The gate, the 8-bit linear layer and the gradient list on the host: sizes and
refusals, before any device work."""
import ctypes

import pytest
import torch

from precision_moe_adapter_gb300 import build, grads, linear, pmoe

BF16, F32 = torch.bfloat16, torch.float32
INV, WS, OK = pmoe.PMOE_ERR_INVALID_ARG, pmoe.PMOE_ERR_WORKSPACE, pmoe.PMOE_OK
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    build.build()
    return pmoe.lib()


@pytest.fixture(scope="module")
def p():
    buf = ctypes.create_string_buffer(256)
    p.keep = buf
    return ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 16


def each_pointer(f, args, where, status=INV):
    """A missing or misaligned pointer at any of the places is refused."""
    for i in where:
        for bad in (None, args[i] + 4):
            a = list(args)
            a[i] = bad
            assert f(*a) == status, (i, bad)


# ---------------------------------------------------------------- gate

def test_gate_refusals(L, p):
    f, b = L.moe_gate_forward, L.moe_gate_backward
    g = pmoe.gate(4, 16, 4)
    each_pointer(f, [g, p, p, p, p, None], (1, 3, 4))
    assert f(g, p, p + 4, p, p, None) == INV
    each_pointer(b, [g, p, p, p, 0, p, None], (1, 2, 3, 5))
    for bad in (dict(E=0), dict(E=4097), dict(k=0), dict(k=17), dict(k=33, E=64), dict(T=-1),
                dict(groups=0), dict(groups=3), dict(groups=33, E=66), dict(groups=4, topk_groups=5),
                dict(groups=4, topk_groups=0), dict(groups=8, topk_groups=1),     # 2 experts for k = 4
                dict(group_sum=0), dict(group_sum=3), dict(factor=float("nan")), dict(factor=float("inf"))):
        kw = dict(T=4, E=16, k=4)
        kw.update(bad)
        assert f(pmoe.gate(**kw), p, None, p, p, None) == INV, bad
        assert b(pmoe.gate(**kw), p, p, p, 0, p, None) == INV, bad
    g.score = 2
    assert f(g, p, None, p, p, None) == INV
    with pytest.raises(ValueError):
        pmoe.gate(4, 16, 4, score="tanh")
    assert f(pmoe.gate(0, 16, 4), None, None, None, None, None) == OK     # no tokens
    assert b(pmoe.gate(0, 16, 4), None, None, None, 0, None, None) == OK


def test_router_logits_refusals(L, p):
    d = pmoe.dims(4, 64, 8, 2, 64, 16)
    f = L.moe_router_logits
    each_pointer(f, [d, p, p, p, 0, p, BIG, None], (1, 2, 3))
    assert f(d, p, p, p, 2, p, BIG, None) == INV
    assert f(d, p, p, p, 0, p, 256, None) == WS
    assert f(d, p, p, p, 0, None, 0, None) == WS
    assert f(pmoe.dims(4, 60, 8, 2, 64, 16), p, p, p, 0, p, BIG, None) == INV


# ---------------------------------------------------------------- 8-bit linear

@pytest.mark.parametrize("rows,N,K", [(-1, 64, 64), (4, 0, 64), (4, 72, 64), (4, 64, 72), (4, 64, 1 << 21),
                                      ((1 << 24) + 1, 64, 64), (1 << 24, 64, 1 << 20)])
def test_linear_shapes_refused(L, p, rows, N, K):
    assert L.fp8_gemm(rows, N, K, p, p, p, p, p, p, BIG, None) == INV
    assert L.dense_w8a8_forward(p, p, N, K, 0, None, rows, p, 0, p, p, BIG, None) == INV
    assert L.dense_w8a8_backward(p, p, N, K, 0, None, rows, p, p, 0, p, None, p, BIG, None) == INV
    assert pmoe.fp8_gemm_ws_bytes(rows, N, K) == 0 and pmoe.dense_w8a8_ws_bytes(rows, N, K) == 0


def test_linear_refusals(L, p):
    each_pointer(L.fp8_quantize, [4, 64, p, 0, p, p, None], (2, 4, 5))
    assert L.fp8_quantize(4, 40, p, 0, p, p, None) == INV
    q = p + 16
    each_pointer(L.fp8_transpose, [64, 64, p, p, q, q, None], (2, 3, 4, 5))
    assert L.fp8_transpose(64, 64, p, p, p, q, None) == INV               # in place
    assert L.fp8_transpose(64, 24, p, p, q, q, None) == INV
    each_pointer(L.fp8_gemm, [4, 64, 64, p, p, p, p, p, p, BIG, None], (3, 4, 5, 6, 7))
    assert L.fp8_gemm(4, 64, 64, p, p, p, p, p, p, 255, None) == WS
    assert L.fp8_gemm(4, 64, 64, p, p, p, p, p, p + 8, BIG, None) == WS
    fwd = [p, p, 64, 64, 16, p, 4, p, 0, p, p, BIG, None]
    each_pointer(L.dense_w8a8_forward, fwd, (0, 1, 7, 9))
    bwd = [p, p, 64, 64, 16, p, 4, p, p, 0, p, p, p, BIG, None]
    each_pointer(L.dense_w8a8_backward, bwd, (0, 1, 7, 8, 10, 11))
    for block in (0, 24, 128):                                            # 64 % 128
        fwd[4] = bwd[4] = block
        assert L.dense_w8a8_forward(*fwd) == INV and L.dense_w8a8_backward(*bwd) == INV
    assert L.dense_w8a8_forward(p, p, 64, 80, 16, p, 4, p, 0, p, p, BIG, None) == INV   # K % 64 with an adapter
    assert L.dense_w8a8_forward(p, p, 64, 64, 0, None, 4, p, 0, p, p, 300, None) == WS
    # no rows: nothing to do
    assert L.fp8_quantize(0, 64, None, 0, None, None, None) == OK
    assert L.fp8_gemm(0, 64, 64, None, None, p, p, None, p, BIG, None) == OK
    assert L.dense_w8a8_forward(p, p, 64, 64, 0, None, 0, None, 0, None, p, BIG, None) == OK


@pytest.mark.parametrize("N,K", [(16, 16), (64, 7168), (7168, 64), (1104, 2064), (4096, 7168), (1040, 18432)])
def test_a_larger_batchs_workspace_serves_smaller_ones(L, N, K):
    rows = list(range(1, 700)) + [1000, 4096, 5000, 20000]
    for adapter in (False, True):
        b = [pmoe.dense_w8a8_ws_bytes(r, N, K, adapter) for r in rows]
        assert b[0] > 256 and all(x <= y for x, y in zip(b, b[1:]))


def test_linear_checks_its_tensors(monkeypatch):
    monkeypatch.setattr(pmoe, "moe_clear_status", lambda ws, stream=None: None)
    q, s = torch.zeros((64, 192), dtype=torch.uint8), torch.zeros((1, 2))
    make = lambda *a, **k: linear.DeviceLinearW8A8(*a, backward=False, **k)
    with pytest.raises(ValueError):
        make(q.T, s, 4)                                  # not contiguous
    with pytest.raises(TypeError):
        make(q.float(), s, 4)
    with pytest.raises(ValueError):
        make(q, torch.zeros((2, 1)), 4)
    with pytest.raises(ValueError):
        make(torch.zeros((64, 200), dtype=torch.uint8), s, 4)
    with pytest.raises(ValueError):
        make(q, s, 4, R=torch.zeros((3, 64, 32), dtype=BF16))
    with pytest.raises(ValueError):
        make(q, s, 4, R=torch.zeros((2, 64, 64), dtype=BF16))
    m = make(q, s, 4)
    X, Y = torch.zeros((4, 192), dtype=BF16), torch.zeros((4, 64), dtype=BF16)
    with pytest.raises(ValueError):
        m.forward(torch.zeros((5, 192), dtype=BF16), torch.zeros((5, 64), dtype=BF16))
    with pytest.raises(ValueError):
        m.forward(X, Y[:3])
    with pytest.raises(TypeError):
        m.forward(X.float(), Y)
    with pytest.raises(ValueError):
        m.forward(X[:, :64], Y)
    with pytest.raises(RuntimeError):
        m.backward(X, Y, X)                              # made without
    with pytest.raises(RuntimeError, match="GPU"):       # host memory
        m.forward(X, Y)
    m.qt = m.q
    with pytest.raises(RuntimeError, match="GPU"):
        m.backward(X, Y, X)


# ---------------------------------------------------------------- gradient list

def fill(L, *g, nbytes=None):
    n = len(g)
    arr = (pmoe.Grad * max(n, 1))(*[pmoe.Grad(*x) for x in g])
    nbytes = L.grad_list_bytes(n) if nbytes is None else nbytes
    lst = pmoe.GradListC()
    return L.grad_list_fill(n, arr, ctypes.create_string_buffer(max(nbytes, 1)), nbytes, ctypes.byref(lst)), lst


def test_grad_list(L):
    F, B = pmoe.GRAD_F32, pmoe.GRAD_BF16
    s, lst = fill(L)
    assert s == OK and lst.n == 0 and lst.chunks == 0
    s, lst = fill(L, (4096, 4096, 8192, F), (1 << 20, 1 << 22, 8193, F), (0, 0, 0, F), (1 << 24, 1 << 24, 16384, B))
    assert s == OK and lst.n == 4 and lst.chunks == 1 + 2 + 0 + 1 and not lst.table
    for bad in ((4096, 4096, 8, 2), (4096, 4096, -1, F), (None, 4096, 8, F), (4096, None, 8, F),
                (4100, 4096, 8, F), (4096, 4104, 8, F), (4096, 4096, (1 << 40) + 1, F)):
        assert fill(L, bad)[0] == INV, bad
    assert fill(L, (4096, 4096, 8, F), nbytes=16)[0] == WS
    # overlaps: the same gradient twice, a result on another's gradient, a result shifted on its own
    assert fill(L, (4096, 4096, 8, F), (4096, 4096, 8, F))[0] == INV
    assert fill(L, (4096, 8192, 8, F), (8192, 4096, 8, F))[0] == INV
    assert fill(L, (4096, 4112, 8, F))[0] == INV
    assert fill(L, (4096, 8192, 8, F), (4096, 8192 + 32, 8, F))[0] == OK      # one gradient, two results
    assert fill(L, (4096, 4096, 8, F), (4128, 4128, 8, F))[0] == OK           # neighbours
    assert fill(L, (4096, 4096, 9, F), (4128, 4128, 8, F))[0] == INV
    assert fill(L, (4096, 4096, 17, B), (4128, 4128, 8, F))[0] == INV
    assert L.grad_list_bytes(-1) == 0


def test_grad_calls_refused(L, p):
    lst = fill(L, (4096, 4096, 8, pmoe.GRAD_F32))[1]
    assert L.grad_norm(lst, p, p, BIG, None) == INV                           # no table
    assert L.grad_clip(lst, 1.0, p, p, BIG, None) == INV
    lst.table = p
    assert L.grad_norm(lst, None, p, BIG, None) == INV
    assert L.grad_norm(lst, p + 2, p, BIG, None) == INV
    assert L.grad_norm(lst, p, p, L.grad_ws_bytes() - 1, None) == WS
    assert L.grad_norm(lst, p, None, 0, None) == WS
    assert L.grad_norm(lst, p, p + 8, BIG, None) == WS
    for m in (0.0, -1.0, float("inf"), float("nan")):
        assert L.grad_clip(lst, m, p, p, BIG, None) == INV
    lst.table = p + 8
    assert L.grad_norm(lst, p, p, BIG, None) == INV


def test_grad_list_checks_its_tensors():
    a, b = torch.zeros(8), torch.zeros((2, 4))
    with pytest.raises(ValueError):
        grads.GradList([a, b], out=[a])
    with pytest.raises(TypeError):
        grads.GradList([a.double()])
    with pytest.raises(TypeError):
        grads.GradList([a], out=[a.to(BF16)])
    with pytest.raises(ValueError):
        grads.GradList([b.T])
    with pytest.raises(ValueError):
        grads.GradList([a], out=[torch.zeros(9)])
    with pytest.raises(pmoe.PmoeError):
        grads.GradList([a, a])
    with pytest.raises(pmoe.PmoeError):
        grads.GradList([torch.zeros(9)[1:]])                                  # not 16-byte aligned
    g = grads.GradList([a, b])
    with pytest.raises(TypeError):
        g.norm(torch.zeros(1, dtype=torch.float64))
    with pytest.raises(ValueError):
        g.clip(1.0, torch.zeros(2))
    with pytest.raises(RuntimeError, match="GPU"):                            # host memory
        g.clip(1.0, torch.zeros(1))
    with pytest.raises(RuntimeError, match="GPU"):
        g.norm(torch.zeros(1))


def test_calls_on_another_device_are_refused(monkeypatch):
    from precision_moe_adapter_gb300 import layer
    monkeypatch.setattr(pmoe, "moe_clear_status", lambda ws, stream=None: None)
    m = linear.DeviceLinearW8A8(torch.zeros((64, 192), dtype=torch.uint8), torch.zeros((1, 2)), 4, backward=False)
    g = grads.GradList([torch.zeros(8)])
    m.device = g.device = torch.device("cuda", 1)
    m.qt = m.q
    lay = layer.DeviceLayer.__new__(layer.DeviceLayer)
    lay.cfg, lay.device = None, torch.device("cuda", 1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for call in (lambda: m.forward(None, None), lambda: m.backward(None, None, None), m.status,
                 lambda: g.norm(None), lambda: g.clip(1.0, None),
                 lambda: lay.gate(None, None, None), lambda: lay.gate_backward(None, None, None, None, None)):
        with pytest.raises(RuntimeError, match="cuda:1"):
            call()
