"""The 8-bit layer's calls in one order on the host: the same refusals as the others."""
import ctypes

from precision_moe_adapter_gb300 import build, pmoe

INV, WS, OK = pmoe.PMOE_ERR_INVALID_ARG, pmoe.PMOE_ERR_WORKSPACE, pmoe.PMOE_OK
BIG = 1 << 40


def test_refusals():
    build.build()
    L = pmoe.lib()
    buf = ctypes.create_string_buffer(256)
    p = ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 16
    calls = ((L.fp8_gemm_one_order, [4, 64, 64, p, p, p, p, p, p, BIG, None], (3, 4, 5, 6, 7), 8),
             (L.dense_w8a8_forward_one_order, [p, p, 64, 64, 16, p, 4, p, 0, p, p, BIG, None], (0, 1, 7, 9), 10),
             (L.dense_w8a8_backward_one_order, [p, p, 64, 64, 16, p, 4, p, p, 0, p, p, p, BIG, None],
              (0, 1, 7, 8, 10, 11), 12))
    for f, args, where, ws in calls:
        for i in where:
            for bad in (None, args[i] + 4):
                assert f(*args[:i], bad, *args[i + 1:]) == INV, (f, i)
        assert f(*args[:ws], None, *args[ws + 1:]) == WS
        assert f(*args[:ws + 1], 255, None) == WS
    assert L.fp8_gemm_one_order(1 << 24, 64, 1 << 20, p, p, p, p, p, p, BIG, None) == INV
    assert L.fp8_gemm_one_order(0, 64, 64, None, None, p, p, None, p, BIG, None) == OK
    assert L.dense_w8a8_forward_one_order(p, p, 64, 64, 0, None, 0, None, 0, None, p, BIG, None) == OK
