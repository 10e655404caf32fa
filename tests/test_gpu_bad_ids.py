"""Block ids outside the pool where a query sees their tokens: every call flags
them, whatever the number, and other sequences' results are what they were;
entries of blocks that no query sees may hold any of them."""
import numpy as np
import pytest

from gpu_util import dev, host
from mask_util import pack, random_tree
from test_gpu_masks import Ctx, offsets

pytestmark = pytest.mark.gpu

IDS = [-1, -2, -3, -2 ** 31, 2 ** 31 - 1, None]     # None: one past the last


def calls(c, cu_dev, table_width):
    """(name, new tokens, call): the attention calls over a pool of two sequences, few rows and many."""
    import torch
    pkv, g = c.pkv, c.hq // c.h
    lens = dev(c.lens, c.device)

    def rows(n):
        return dev(np.random.default_rng(n).standard_normal((2 * n, c.hq, c.d)).astype(np.float16), c.device)
    q1 = rows(1)
    ws = pkv.make_workspace(c.pool, 2, c.hq, table_width, 0)
    yield "decode", 1, lambda t, o: pkv.pf_paged_decode_attention(c.pool, 1, q1, t, lens, c.scale, o, 0, ws)
    wws = pkv.make_window_workspace(c.pool, 2, c.hq, table_width, 1, 40, 3)
    yield "window step", 1, lambda t, o: pkv.pf_paged_window_attention(c.pool, 1, q1, t, lens, None, 1, c.scale, 40, 3, o, wws)
    for n in (3, 40):
        q, cu = rows(n), cu_dev(n)
        cws = pkv.make_cross_workspace(c.pool, 2, c.hq, table_width, n)
        pws, size = None, pkv.pf_prefill_workspace_bytes(c.pool, 2, c.hq, table_width, n)
        if size:
            pws = torch.empty(size, dtype=torch.uint8, device=c.device)
            pkv.pf_decode_workspace_init(pws)
        bits = dev(pack([random_tree(np.random.default_rng(i), n) for i in range(2)], 1), c.device)
        for w in (True, False):
            few = "few rows" if w and n * g <= 16 else "prompt"
            yield f"cross, {few}", n, lambda t, o, q=q, cu=cu, n=n, w=cws if w else None: pkv.pf_paged_cross_attention(
                c.pool, 1, q, t, lens, cu, n, c.scale, o, w)
            yield f"prefill, {few}", n, lambda t, o, q=q, cu=cu, n=n, w=pws if w else None: pkv.pf_paged_prefill_attention(
                c.pool, 1, q, t, lens, cu, n, c.scale, o, w)
            mws = pkv.make_window_workspace(c.pool, 2, c.hq, table_width, n, 40, 3) if w else None
            yield f"window, {few}", n, lambda t, o, q=q, cu=cu, n=n, w=mws: pkv.pf_paged_window_attention(
                c.pool, 1, q, t, lens, cu, n, c.scale, 40, 3, o, w)
            tws = pkv.make_tree_workspace(c.pool, 2, c.hq, table_width, n) if w else None
            yield f"tree, {few}", n, lambda t, o, q=q, cu=cu, n=n, b=bits, w=tws: pkv.pf_paged_tree_attention(
                c.pool, 1, q, t, lens, cu, n, c.scale, b, o, w)


@pytest.mark.parametrize("cache", ["f16", "e4m3"])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("h,g,d,page", [(2, 2, 64, 16), (2, 1, 128, 1), (1, 4, 128, 64), (3, 1, 64, 1), (2, 3, 64, 256)])
def test_bad_ids_are_flagged(pkv, cuda_dev, cache, f32, h, g, d, page):
    import torch
    L = 300
    c = Ctx(pkv, cuda_dev, cache, [L, L], h * g, h, d, page)
    width = c.table.shape[1]
    cu_dev = lambda n: dev(offsets([n, n]), cuda_dev)   # noqa: E731
    pkv.pf_device_status(reset=True)
    for name, n, call in calls(c, cu_dev, width):
        out = torch.empty((2 * n, h * g, d), dtype=torch.float32 if f32 else torch.float16, device=cuda_dev)
        good = dev(c.table, cuda_dev)
        call(good, out)
        assert pkv.pf_device_status(reset=True) == 0, name
        want = host(out).copy()
        # the second sequence's last block, its first (a window's sinks) and one that the window sees
        for entry in {(L - 1) // page, 0, (L - 20) // page}:
            for bad in IDS:
                t = c.table.copy()
                t[1, entry] = c.n_blocks if bad is None else bad
                call(dev(t, cuda_dev), out)
                assert pkv.pf_device_status(reset=True) == pkv.PF_DEV_BAD_BLOCK_ID, (name, entry, bad)
                assert np.array_equal(host(out)[:n], want[:n]), (name, entry, bad)
        # unseen: past the context, and between a window's sinks and its first token
        for bad in IDS:
            t = np.pad(c.table, ((0, 0), (0, 1)), constant_values=c.n_blocks if bad is None else bad)
            first = (L - n - 40) // page
            if name.startswith("window"):
                t[:, -(-3 // page):first] = t[0, -1]
            call(dev(t[:, :width + 1], cuda_dev), out)
            assert pkv.pf_device_status(reset=True) == 0, (name, bad)
