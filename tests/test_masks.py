"""Masked attention without a GPU: what the calls refuse before anything is
launched, and their workspaces' sizes (made-up device addresses)."""
import ctypes
import math
from types import SimpleNamespace

import numpy as np
import pytest

from mask_util import pack, random_tree
from test_bounds import pools

P = ctypes.c_void_p
OK, ODD = P(0x30000), P(0x30008)
INT_MAX = 2 ** 31 - 1

GOOD = dict(layer=0, q=OK, bt=OK, width=7, lens=OK, cu=OK, n=4, most=5, hq=4, scale=0.1, window=9, sinks=2, tree=OK, words=1,
            out=OK, dtype=1, ws=None, bytes=0)


def window(lib, pool, **kw):
    a = {**GOOD, **kw}
    return lib.pf_paged_window_attention(pool, a["layer"], a["q"], a["bt"], a["width"], a["lens"], a["cu"], a["n"], a["most"],
                                         a["hq"], ctypes.c_float(a["scale"]), a["window"], a["sinks"], a["out"], a["dtype"],
                                         a["ws"], a["bytes"], None)


def tree(lib, pool, **kw):
    a = {**GOOD, **kw}
    return lib.pf_paged_tree_attention(pool, a["layer"], a["q"], a["bt"], a["width"], a["lens"], a["cu"], a["n"], a["most"],
                                       a["hq"], ctypes.c_float(a["scale"]), a["tree"], a["words"], a["out"], a["dtype"],
                                       a["ws"], a["bytes"], None)


COMMON = [
    (dict(layer=1), "layer"), (dict(n=-1), "negative"), (dict(most=-1), "negative"), (dict(q=None), "null"),
    (dict(bt=None), "null"), (dict(lens=None), "null"), (dict(out=None), "null"), (dict(q=ODD), "aligned"),
    (dict(out=ODD), "aligned"), (dict(dtype=3), "out_dtype"), (dict(hq=0), "n_q_heads"), (dict(hq=3), "n_q_heads"),
    (dict(width=0), "max_blocks"), (dict(width=1 << 27), "max_blocks"), (dict(scale=0.0), "scale"), (dict(scale=-1.0), "scale"),
    (dict(scale=math.nan), "scale"), (dict(ws=ODD, bytes=1 << 30), "aligned"),
]


@pytest.mark.parametrize("kw,word", COMMON + [(dict(window=0), "window"), (dict(window=-5), "window"), (dict(sinks=-1), "n_sinks"),
                                              (dict(cu=None), "max_new_tokens"), (dict(cu=None, most=0, window=0), "window")])
def test_window_refusals(pkv, kw, word):
    lib = pkv.lib()
    for pool in pools(lib):
        assert window(lib, pool, **kw) == pkv.PF_ERR_INVALID
        assert word in pkv.pf_last_error(), pkv.pf_last_error()
        lib.pf_pool_destroy(pool)


@pytest.mark.parametrize("kw,word", COMMON + [(dict(cu=None), "cu_q"), (dict(tree=None), "tree"), (dict(tree=P(0x30004)), "aligned"),
                                              (dict(words=0), "tree_words"), (dict(most=65), "tree_words"),
                                              (dict(most=INT_MAX, words=1 << 20), "tree_words")])
def test_tree_refusals(pkv, kw, word):
    lib = pkv.lib()
    for pool in pools(lib):
        assert tree(lib, pool, **kw) == pkv.PF_ERR_INVALID
        assert word in pkv.pf_last_error(), pkv.pf_last_error()
        lib.pf_pool_destroy(pool)


@pytest.mark.parametrize("call", [window, tree])
def test_nothing_to_do_and_not_built(pkv, call):
    lib = pkv.lib()
    for pool in pools(lib):
        assert call(lib, pool, hq=34) == pkv.PF_ERR_UNSUPPORTED
        assert call(lib, pool, n=0, q=None) == pkv.PF_OK
        assert call(lib, pool, most=0, q=None) == pkv.PF_OK
        # rows that do not fit 32 bits: only a table as large allows them
        assert call(lib, pool, most=INT_MAX, words=1 << 25, width=1 << 26, hq=32) == pkv.PF_ERR_INVALID
        assert "query tokens" in pkv.pf_last_error()
        lib.pf_pool_destroy(pool)
    assert call(lib, None) == pkv.PF_ERR_INVALID


@pytest.mark.parametrize("B", [1, 16])
@pytest.mark.parametrize("H,group", [(12, 1), (8, 4), (5, 2), (1, 3)])
@pytest.mark.parametrize("D", [64, 128])
def test_workspace_of_more_tokens_is_no_smaller(pkv, B, H, group, D):
    lib = pkv.lib()
    for pool in pools(lib, B, H, D):
        for size in (lambda *a: lib.pf_tree_workspace_bytes(pool, *a),
                     lambda *a: lib.pf_window_workspace_bytes(pool, *a, 64, 4),
                     lambda *a: lib.pf_window_workspace_bytes(pool, *a, 5000, 0),
                     lambda *a: lib.pf_window_workspace_bytes(pool, *a, INT_MAX, INT_MAX)):
            for blocks in (7, 4096 // B, 65536 // B):
                sizes = [size(4, H * group, blocks, n) for n in (*range(1, 18), 40, 100, 300)]
                some = [s for s in sizes if s]
                assert some[0] == sizes[0] > 0
                assert all(a <= b for a, b in zip(some, some[1:])), (blocks, sizes)
        lib.pf_pool_destroy(pool)


def test_workspace_refusals(pkv):
    lib = pkv.lib()
    for pool in pools(lib):
        for bad in ((-1, 4, 7, 3, 9, 0), (4, 4, 0, 3, 9, 0), (4, 4, 7, -1, 9, 0), (4, 4, 7, 3, 0, 0), (4, 4, 7, 3, 9, -1)):
            assert lib.pf_window_workspace_bytes(pool, *bad) == 0 and pkv.pf_last_error()
            if bad[4:] == (9, 0):
                assert lib.pf_tree_workspace_bytes(pool, *bad[:4]) == 0 and pkv.pf_last_error()
        lib.pf_pool_destroy(pool)
    assert lib.pf_tree_workspace_bytes(None, 4, 4, 7, 3) == 0 and lib.pf_window_workspace_bytes(None, 4, 4, 7, 3, 9, 0) == 0


def test_bindings_refuse_shapes(pkv, monkeypatch):
    import torch
    # (a host tensor's device is -1: as if that were the current one, every shape is looked at)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    pool = SimpleNamespace(handle=None, n_layers=1, n_blocks=8, block_size=16, n_kv_heads=2, head_dim=128, k_scale=None,
                           device=-1)
    q = torch.zeros((6, 4, 128), dtype=torch.float16)
    table, lens = torch.zeros((3, 2), dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    cu, bits = torch.arange(0, 8, 2, dtype=torch.int32), torch.zeros((6, 1), dtype=torch.int64)

    def both(word, q=q, table=table, lens=lens, cu=cu, out=None, bits=bits):
        out = q.clone() if out is None else out
        for call in (lambda: pkv.pf_paged_window_attention(pool, 0, q, table, lens, cu, 2, 0.1, 5, 1, out),
                     lambda: pkv.pf_paged_tree_attention(pool, 0, q, table, lens, cu, 2, 0.1, bits, out)):
            with pytest.raises(pkv.PagedKVError, match=word):
                call()
    for shape in ((6, 128), (6, 4, 64), (1, 6, 4, 128)):
        both("T_q", q=torch.zeros(shape, dtype=torch.float16))
    both("out", out=q[:5])
    both("float", out=q.double())
    both("block_tables", table=table[0])
    both("block_tables", lens=lens[:2])
    both("cu_q", cu=cu[:3])
    both("int32", table=table.long())
    both("int32", cu=cu.long())
    both("float16", q=q.float(), out=q)
    both("contiguous", q=q.transpose(0, 1).contiguous().transpose(0, 1))
    both("pool is null")
    with pytest.raises(pkv.PagedKVError, match="row per sequence"):
        pkv.pf_paged_window_attention(pool, 0, q, table, lens, None, 1, 0.1, 5, 1, q.clone())
    with pytest.raises(pkv.PagedKVError, match="cu_q"):
        pkv.pf_paged_tree_attention(pool, 0, q[:3], table, lens, None, 1, 0.1, bits[:3], q[:3].clone())
    with pytest.raises(pkv.PagedKVError, match="row per query"):
        pkv.pf_paged_tree_attention(pool, 0, q, table, lens, cu, 2, 0.1, bits[:5], q.clone())
    with pytest.raises(pkv.PagedKVError, match="int64"):
        pkv.pf_paged_tree_attention(pool, 0, q, table, lens, cu, 2, 0.1, bits.int(), q.clone())
    pool.device = 1
    both("current device")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    both("CUDA")


def test_packed_bits():
    """Bit j % 64 of word j / 64, whatever the sign."""
    rng = np.random.default_rng(0)
    sees = random_tree(rng, 130)
    words = pack([sees], 3).astype(np.uint64)
    for i in (0, 1, 63, 64, 100, 129):
        for j in range(130):
            assert bool((words[i, j // 64] >> np.uint64(j % 64)) & np.uint64(1)) == sees[i, j]
