"""Compaction of the host allocator against a plain model, and the refusals of
the 8-bit, cross attention and compaction calls (no GPU needed)."""
import ctypes

import numpy as np
import pytest


def _check(alloc, pkv, refs, src, dst, block_map):
    n = len(refs)
    live = sorted(b for b in range(n) if refs[b])
    want_src = [b for b in live if b >= len(live)]
    want_dst = [b for b in range(len(live)) if not refs[b]]
    assert src.tolist() == want_src and dst.tolist() == want_dst
    moved = dict(zip(want_src, want_dst))
    assert block_map.tolist() == [moved.get(b, b) for b in range(n)]
    new = [0] * n
    for b in live:
        new[moved.get(b, b)] = refs[b]
    assert [pkv.pf_alloc_refcount(alloc, b) for b in range(n)] == new
    assert pkv.pf_alloc_free_count(alloc) == n - len(live)
    return new


@pytest.mark.parametrize("n,seed", [(1, 0), (7, 3), (64, 0), (257, 11)])
def test_compact_after_churn(pkv, n, seed):
    alloc = pkv.pf_alloc_create(n, seed)
    rng = np.random.default_rng(seed)
    refs = [0] * n
    for _ in range(6):
        for _ in range(8):
            take = int(rng.integers(0, pkv.pf_alloc_free_count(alloc) + 1))
            for b in pkv.pf_alloc_blocks(alloc, take):
                refs[b] += 1
            live = np.flatnonzero(refs)
            share = rng.choice(live, int(rng.integers(0, live.size + 1)), replace=False) if live.size else live
            pkv.pf_alloc_share(alloc, share.astype(np.int32))
            for b in share:
                refs[b] += 1
            drop = rng.choice(live, int(rng.integers(0, live.size + 1)), replace=False) if live.size else live
            pkv.pf_free_blocks(alloc, drop.astype(np.int32))
            for b in drop:
                refs[b] -= 1
        refs = _check(alloc, pkv, refs, *pkv.pf_alloc_compact(alloc))
        again = pkv.pf_alloc_compact(alloc)
        assert again[0].size == 0 and again[2].tolist() == list(range(n))
    n_live = sum(1 for r in refs if r)
    rest = pkv.pf_alloc_blocks(alloc, n - n_live)
    assert rest.tolist() == list(range(n_live, n))       # the lowest free id first


def test_compact_empty_and_full(pkv):
    alloc = pkv.pf_alloc_create(5, 9)
    src, dst, m = pkv.pf_alloc_compact(alloc)
    assert src.size == dst.size == 0 and m.tolist() == [0, 1, 2, 3, 4]
    assert sorted(pkv.pf_alloc_blocks(alloc, 5).tolist()) == [0, 1, 2, 3, 4]
    assert pkv.pf_alloc_compact(alloc)[0].size == 0
    lib, P = pkv.lib(), ctypes.c_void_p
    n = ctypes.c_int()
    ids = (ctypes.c_int32 * 5)()
    assert lib.pf_alloc_compact(None, ids, ids, ids, ctypes.byref(n)) == pkv.PF_ERR_INVALID
    assert lib.pf_alloc_compact(alloc.handle, None, ids, ids, ctypes.byref(n)) == pkv.PF_ERR_INVALID
    assert lib.pf_alloc_compact(alloc.handle, ids, ids, P(0), ctypes.byref(n)) == pkv.PF_ERR_INVALID


P = ctypes.c_void_p
OK = P(0x30000)


def _pool8(lib, ks=0x40000, vs=0x50000, k=0x10000, B=16, H=12, D=64, L=1, N=64):
    h = P()
    rc = lib.pf_pool_create_e4m3(ctypes.byref(h), P(k), P(0x20000), P(ks), P(vs), L, N, B, H, D)
    return rc, h


def _pool16(lib):
    h = P()
    assert lib.pf_pool_create(ctypes.byref(h), P(0x10000), P(0x20000), 1, 64, 16, 12, 64, 1) == 0
    return h


def test_e4m3_pool_sizes_and_validation(pkv):
    lib = pkv.lib()
    assert pkv.pf_pool_bytes(3, 64, 16, 12, 64, dtype=pkv.PF_E4M3) == 3 * 64 * 16 * 12 * 64
    assert pkv.pf_scale_bytes(3, 64, 12) == 3 * 64 * 12 * 4
    assert pkv.pf_scale_bytes(3, 0, 12) == 0
    for bad in (dict(ks=0), dict(vs=0), dict(ks=0x40002), dict(k=0), dict(k=0x10004), dict(B=8), dict(D=32), dict(H=0),
                dict(N=0), dict(L=4096, N=65536)):
        rc, h = _pool8(lib, **bad)
        assert rc == pkv.PF_ERR_INVALID and not h.value, bad
    h = P()
    assert lib.pf_pool_create(ctypes.byref(h), OK, OK, 1, 64, 16, 12, 64, pkv.PF_E4M3) == pkv.PF_ERR_INVALID
    assert "pf_pool_create_e4m3" in pkv.pf_last_error()
    rc, h = _pool8(lib)
    assert rc == 0
    assert lib.pf_block_image_bytes(h) == 2 * (16 * 12 * 64 + 48)
    lib.pf_pool_destroy(h)


def test_append_refusals(pkv):
    lib = pkv.lib()
    rc, pool = _pool8(lib)
    f16 = _pool16(lib)
    call = lambda p=pool, layer=0, k=OK, v=OK, bt=OK, mb=7, lens=OK, cu=OK, n=4, mx=3: (   # noqa: E731
        lib.pf_append_kv(p, layer, k, v, bt, mb, lens, cu, n, mx, None))
    for bad in (dict(p=None), dict(layer=1), dict(layer=-1), dict(k=None), dict(v=P(0x30008)), dict(bt=None),
                dict(lens=None), dict(mb=0), dict(mb=1 << 27), dict(n=-1), dict(mx=-1), dict(cu=None, mx=2)):
        assert call(**bad) == pkv.PF_ERR_INVALID, bad
    assert call(p=f16) == pkv.PF_ERR_UNSUPPORTED and "pf_write_kv" in pkv.pf_last_error()
    assert call(n=0, k=None) == pkv.PF_OK and call(mx=0, k=None) == pkv.PF_OK
    assert lib.pf_write_kv(pool, 0, OK, OK, OK, 4, 7, OK, OK, 1, None) == pkv.PF_ERR_UNSUPPORTED
    assert "pf_append_kv" in pkv.pf_last_error()
    lib.pf_pool_destroy(pool)
    lib.pf_pool_destroy(f16)


def test_attention_refusals_on_e4m3_pools(pkv):
    lib = pkv.lib()
    rc, pool = _pool8(lib)
    dec = lambda hq=12, dt=1, scale=0.125, ws=1 << 30, split=0, w=OK: (   # noqa: E731
        lib.pf_paged_decode_attention(pool, 0, OK, OK, 7, OK, 4, hq, ctypes.c_float(scale), OK, dt, split, w, ws, None))
    for split in (-1, -2, 16):
        assert dec(split=split) == pkv.PF_ERR_UNSUPPORTED
        assert lib.pf_decode_workspace_bytes(pool, 4, 12, 7, split) == 0
    assert dec(hq=13) == pkv.PF_ERR_INVALID and dec(hq=12 * 17) == pkv.PF_ERR_UNSUPPORTED
    assert dec(dt=3) == pkv.PF_ERR_INVALID and dec(scale=0.0) == pkv.PF_ERR_INVALID
    assert dec(w=P(0x30008)) == pkv.PF_ERR_INVALID and dec(w=None) == pkv.PF_ERR_INVALID
    assert lib.pf_decode_workspace_bytes(pool, 4, 12 * 17, 7, 0) == 0
    ws = [lib.pf_decode_workspace_bytes(pool, 4, 12 * g, 7, 0) for g in (1, 2, 16)]
    assert 0 < ws[0] < ws[1] < ws[2]
    assert lib.pf_prefill_workspace_bytes(pool, 4, 12, 7, 16) == ws[2]
    assert lib.pf_prefill_workspace_bytes(pool, 4, 12, 7, 17) == 0
    lib.pf_pool_destroy(pool)
    rc, pool = _pool8(lib, B=1)
    assert lib.pf_prefill_workspace_bytes(pool, 4, 12, 7, 16) > 0       # any page size
    lib.pf_pool_destroy(pool)


def test_cross_refusals(pkv):
    lib = pkv.lib()
    for pool in (_pool8(lib)[1], _pool16(lib)):
        call = lambda p=pool, layer=0, q=OK, bt=OK, mb=7, lens=OK, cu=OK, n=4, mx=3, hq=12, scale=0.125, out=OK, dt=1, w=None, ws=0: (   # noqa: E731
            lib.pf_paged_cross_attention(p, layer, q, bt, mb, lens, cu, n, mx, hq, ctypes.c_float(scale), out, dt, w, ws, None))
        for bad in (dict(p=None), dict(layer=3), dict(q=None), dict(q=P(0x30002)), dict(bt=None), dict(mb=0),
                    dict(mb=1 << 27), dict(lens=None), dict(cu=None), dict(n=-1), dict(mx=-1), dict(hq=13), dict(hq=0),
                    dict(scale=-1.0), dict(scale=float("nan")), dict(out=None), dict(out=P(0x30004)), dict(dt=3),
                    dict(w=P(0x30008), ws=1 << 30)):
            assert call(**bad) == pkv.PF_ERR_INVALID, bad
        assert call(hq=12 * 17) == pkv.PF_ERR_UNSUPPORTED
        assert call(n=0, q=None) == pkv.PF_OK and call(mx=0, q=None) == pkv.PF_OK
        assert lib.pf_cross_workspace_bytes(pool, 4, 12, 7, 16) > 0
        assert lib.pf_cross_workspace_bytes(pool, 4, 12, 7, 17) == 0
        assert lib.pf_cross_workspace_bytes(pool, 4, 24, 7, 9) == 0
        assert lib.pf_cross_workspace_bytes(pool, 4, 13, 7, 1) == 0
        assert lib.pf_cross_workspace_bytes(None, 4, 12, 7, 1) == 0
        lib.pf_pool_destroy(pool)


def test_compact_blocks_refusals(pkv):
    lib = pkv.lib()
    pool = _pool16(lib)
    call = lambda p=pool, src=OK, dst=OK, n=2, m=OK, bt=OK, rows=3, mb=7, lens=OK: (   # noqa: E731
        lib.pf_compact_blocks(p, src, dst, n, m, bt, rows, mb, lens, None))
    for bad in (dict(p=None), dict(src=None), dict(dst=None), dict(n=-1), dict(rows=-1), dict(m=None), dict(bt=None),
                dict(mb=0), dict(lens=None)):
        assert call(**bad) == pkv.PF_ERR_INVALID, bad
    assert call(n=0, rows=0, m=None, bt=None, lens=None) == pkv.PF_OK
    lib.pf_pool_destroy(pool)
