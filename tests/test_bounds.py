"""Bounds on query tokens whose rows do not fit the kernels' 32-bit counts are
refused before anything is launched (made-up device addresses, no GPU)."""
import ctypes

import pytest

P = ctypes.c_void_p
OK = P(0x30000)
INT_MAX = 2 ** 31 - 1


def pools(lib):
    h8, h16 = P(), P()
    assert lib.pf_pool_create_e4m3(ctypes.byref(h8), P(0x10000), P(0x20000), P(0x40000), P(0x50000), 1, 64, 16, 2, 64) == 0
    assert lib.pf_pool_create(ctypes.byref(h16), P(0x10000), P(0x20000), 1, 64, 16, 2, 64, 1) == 0
    return h8, h16


@pytest.mark.parametrize("ws", [None, OK])
def test_cross_attention(pkv, ws):
    lib = pkv.lib()
    for pool in pools(lib):
        for bound, hq in ((INT_MAX, 2), (INT_MAX, 4), (INT_MAX // 2, 4), (1 << 28, 16), (INT_MAX - 100, 2)):
            rc = lib.pf_paged_cross_attention(pool, 0, OK, OK, 7, OK, OK, 4, bound, hq, ctypes.c_float(0.1), OK, 1, ws,
                                              1 << 30, None)
            assert rc == pkv.PF_ERR_INVALID and "query tokens" in pkv.pf_last_error(), (bound, hq)
        lib.pf_pool_destroy(pool)


@pytest.mark.parametrize("ws", [None, OK])
def test_causal_attention_over_a_table_as_large(pkv, ws):
    """A loose bound alone is none of the caller's errors; 2^28 tokens of 16 rows are."""
    lib = pkv.lib()
    for pool in pools(lib):
        rc = lib.pf_paged_prefill_attention(pool, 0, OK, OK, 1 << 24, OK, OK, 4, INT_MAX, 32, ctypes.c_float(0.1), OK, 1,
                                            ws, 1 << 30, None)
        assert rc == pkv.PF_ERR_INVALID and "query tokens" in pkv.pf_last_error()
        lib.pf_pool_destroy(pool)
