"""Bounds on query tokens: those whose rows do not fit the kernels' 32-bit counts
are refused before anything is launched, and a workspace made for a bound is
large enough for smaller ones (made-up device addresses, no GPU)."""
import ctypes

import pytest

P = ctypes.c_void_p
OK = P(0x30000)
INT_MAX = 2 ** 31 - 1


def pools(lib, B=16, H=2, D=64):
    h8, h16 = P(), P()
    assert lib.pf_pool_create_e4m3(ctypes.byref(h8), P(0x10000), P(0x20000), P(0x40000), P(0x50000), 1, 64, B, H, D) == 0
    assert lib.pf_pool_create(ctypes.byref(h16), P(0x10000), P(0x20000), 1, 64, B, H, D, 1) == 0
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


@pytest.mark.parametrize("B", [1, 16])
@pytest.mark.parametrize("H,group", [(12, 1), (8, 1), (8, 4), (5, 2), (1, 3)])
@pytest.mark.parametrize("D", [64, 128])
def test_workspace_of_more_tokens_is_no_smaller(pkv, B, H, group, D):
    """For as many tokens as take a workspace; 0 stands for calls without one."""
    lib = pkv.lib()
    for pool in pools(lib, B, H, D):
        for size in (lib.pf_prefill_workspace_bytes, lib.pf_cross_workspace_bytes):
            for blocks in (7, 4096 // B, 65536 // B):
                sizes = [size(pool, 4, H * group, blocks, n) for n in (*range(1, 18), 40, 100, 300)]
                some = [s for s in sizes if s]
                assert some[0] == sizes[0] > 0
                assert all(a <= b for a, b in zip(some, some[1:])), (blocks, sizes)
        lib.pf_pool_destroy(pool)
