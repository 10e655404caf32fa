"""Attention under a window with sinks and under trees of drafts on the GPU,
against a plain 64-bit form: over fp16 and e4m3 pages, on the few-rows kernel
(with a workspace and at most 16 rows per kv-head) and on the prompt kernel,
contexts cut and whole."""
import numpy as np
import pytest

from e4m3_util import assert_within
from gpu_util import PagedCase, dev, host
from mask_util import masked64, pack, random_tree, tree_seen, window_seen
from test_gpu_e4m3 import F16, F32, Case

pytestmark = pytest.mark.gpu


class Ctx:
    """A pool of two layers (work in layer 1) of either type, its rows, and calls on it."""

    def __init__(self, pkv, device, cache, lens, hq, h, d, page, seed=9):
        self.pkv, self.device, self.cache = pkv, device, cache
        self.lens, self.hq, self.h, self.d, self.page = np.asarray(lens, np.int32), hq, h, d, page
        if cache == "f16":
            self.c = PagedCase(pkv, device, lens, hq, h, d, page, n_layers=2)
            self.table, self.n_blocks, self.k_host, self.v_host = self.c.bt, self.c.n_blocks, self.c.k_host, self.c.v_host
            # rows past a context's end hold what must not be read as numbers
            for s, L in enumerate(lens):
                t = np.arange(L, -(-L // page) * page)
                for x in (self.c.k_dev, self.c.v_dev):
                    x[1, dev(self.table[s, t // page].astype(np.int64), device), dev(t % page, device)] = float("nan")
        else:
            self.c = Case(pkv, device, lens, hq, h, d, page)
            self.c.fill()
            self.table, self.n_blocks = self.c.table, self.c.N
        self.pool = self.c.pool
        self.rng = np.random.default_rng(seed)
        self.scale = float(np.float32(1.0 / np.sqrt(d)))
        self.table = self.table.copy()

    def rows(self, s, L=None):
        L = int(self.lens[s]) if L is None else L
        t = np.arange(L)
        if self.cache == "f16":
            return [x[1][self.table_as_made(s)[t // self.page], t % self.page] for x in (self.k_host, self.v_host)]
        return [m.rows(self.table_as_made(s), L) for m in (self.c.km, self.c.vm)]

    def table_as_made(self, s):
        return (self.c.bt if self.cache == "f16" else self.c.table)[s]

    def forget(self, seen, poison):
        """What no query sees: rows hold no numbers; blocks of nothing else are gone, their entries
        hold anything (poison: they stay in the table, with scales that are no numbers)."""
        gone = []
        blk, at = [], []
        for s, x in enumerate(seen):
            L = int(self.lens[s])
            t = np.flatnonzero(~x.any(0)) if len(x) else np.arange(L)
            blk.append(self.table_as_made(s)[t // self.page])
            at.append(t % self.page)
        blk, at = (dev(np.concatenate(v).astype(np.int64), self.device) for v in (blk, at))
        if self.cache == "f16":
            for x in (self.c.k_dev, self.c.v_dev):
                x[1, blk, at] = float("nan")
        else:
            for x in (self.c.k, self.c.v):
                x.view(self.c.torch.uint8)[1, blk, at] = 0x7f
        for s, x in enumerate(seen):
            L = int(self.lens[s])
            any_row = x.any(0) if len(x) else np.zeros(L, bool)
            for j in range(-(-L // self.page)):
                if not any_row[j * self.page:(j + 1) * self.page].any():
                    gone.append(int(self.table[s, j]))
                    if not poison:
                        self.table[s, j] = 1 << 30
        if poison and gone:
            ids = dev(np.array(gone), self.device)
            if self.cache == "e4m3":
                for x in (self.c.ks, self.c.vs):
                    x[1, ids] = float("nan")
        return len(gone)

    def want(self, q, offs, seen, step, out_step):
        got = []
        for s, x in enumerate(seen):
            k, v = self.rows(s)
            got.append(masked64(q[offs[s]:offs[s + 1]], k, v, self.scale, x, step, out_step))
        out, tol = np.concatenate([o for o, _ in got]), np.concatenate([t for _, t in got])
        if self.cache == "e4m3" and len(out):
            tol = tol + np.where(out == 0, 0, self.c.small_terms(q, offs))
        return out, tol


def offsets(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def check(c, q, offs, seen, call, work, f32, what=""):
    """The call's result within its bound, twice, its rows alone, no flags."""
    import torch
    few = work is not None and (np.diff(offs).max(initial=0)) * (c.hq // c.h) <= 16
    step = 2.0 ** -21 if f32 and few else F16
    want, tol = c.want(q, offs, seen, step, F32 if f32 else F16)
    out = torch.full((len(q) + 1, c.hq, c.d), 7.0, dtype=torch.float32 if f32 else torch.float16, device=c.device)
    c.pkv.pf_device_status(reset=True)
    for _ in range(2):
        call(out[:-1], work)
        assert c.pkv.pf_device_status(reset=True) == 0, what
        assert_within(host(out)[:-1], want, tol, what)
    assert bool((out[-1] == 7.0).all())
    empty = np.concatenate([~x.any(1) if x.size else np.ones(len(x), bool) for x in seen]) if len(q) else np.zeros(0, bool)
    assert not host(out)[:-1][empty].any()


# ------------------------------------------------------------------ windows

WINDOWS = [
    # lengths, new tokens (None: a decode step without offsets), q-heads, kv-heads, head_dim, page, window, sinks
    ([200, 0, 17, 1, 64], None, 12, 12, 64, 16, 64, 4),
    ([2000, 130, 1024, 5], None, 14, 2, 64, 64, 100, 4),
    ([700, 513, 40], None, 5, 5, 128, 16, 257, 64),
    ([900, 64], None, 8, 4, 128, 1, 33, 3),
    ([3000], None, 16, 1, 64, 1, 1000, 0),
    ([3000, 10], None, 16, 1, 128, 256, 700, 300),
    ([500, 3], None, 3, 3, 64, 256, 1, 0),
    ([500, 31, 32, 33], None, 2, 2, 64, 16, 1, 1),
    ([300, 20], None, 2, 1, 128, 16, 1 << 30, 5),
    ([300, 20], None, 2, 1, 64, 16, 17, 1 << 30),
    ([300, 40, 0, 16], [3, 8, 0, 1], 12, 6, 64, 16, 30, 4),
    ([800, 90], [16, 2], 4, 4, 128, 64, 130, 70),
    ([800, 90], [5, 5], 3, 1, 64, 1, 10, 2),
    ([1500, 40], [5, 1], 9, 3, 128, 256, 600, 17),
    ([300, 129, 64, 1], [300, 100, 64, 1], 4, 2, 64, 16, 50, 4),
    ([1000, 700], [1000, 30], 2, 2, 128, 16, 200, 65),
    ([1000, 700], [600, 700], 8, 2, 128, 64, 64, 0),
    ([1300, 5], [1200, 3], 3, 3, 64, 64, 129, 129),
    ([700, 66], [520, 66], 6, 2, 64, 1, 100, 7),
    ([640, 300], [333, 300], 14, 2, 128, 1, 1, 1),
    ([900, 1100], [300, 20], 16, 1, 64, 256, 257, 1),
    ([2600], [40], 4, 1, 64, 16, 2000, 4),
    ([5000, 600], [33, 40], 2, 1, 128, 16, 3500, 300),
    ([4100, 900, 129], [70, 1, 129], 3, 1, 64, 64, 4000, 10),
    ([4500], [300], 4, 2, 64, 64, 2500, 700),
    ([3000, 100], [17, 100], 5, 1, 128, 1, 1111, 1),
    ([700], [500], 1, 1, 64, 16, 1 << 30, 0),
    ([257, 0], [256, 0], 1, 1, 128, 16, 5, 1 << 29),
]


def window_case(pkv, cuda_dev, cache, lens, new, hq, h, d, page, W, S, f32, ws, wide=False, poison=False):
    import torch
    c = Ctx(pkv, cuda_dev, cache, lens, hq, h, d, page)
    step = new is None
    new = [1] * len(lens) if step else new
    offs = offsets(new)
    q = c.rng.standard_normal((int(offs[-1]), hq, d)).astype(np.float16)
    seen = [window_seen(L, n, W, S) if L else np.zeros((n, 0), bool) for L, n in zip(lens, new)]
    c.forget(seen, poison)
    table = dev(c.table, cuda_dev)
    if wide:
        table = torch.nn.functional.pad(table, (0, 8192 // page), value=1 << 30)
    work = pkv.make_window_workspace(c.pool, len(lens), hq, table.shape[1], max(new), W, S) if ws else None
    assert work is not None or not ws or max(new) * (hq // h) > 16
    qd, ld, cu = dev(q, cuda_dev), dev(c.lens, cuda_dev), None if step else dev(offs, cuda_dev)
    check(c, q, offs, seen, lambda out, w: pkv.pf_paged_window_attention(c.pool, 1, qd, table, ld, cu, max(new), c.scale, W, S,
                                                                         out, w), work, f32)


@pytest.mark.parametrize("lens,new,hq,h,d,page,W,S", WINDOWS)
@pytest.mark.parametrize("cache", ["f16", "e4m3"])
@pytest.mark.parametrize("f32,ws", [(False, True), (True, True), (False, False)])
def test_window(pkv, cuda_dev, lens, new, hq, h, d, page, W, S, cache, f32, ws):
    window_case(pkv, cuda_dev, cache, lens, new, hq, h, d, page, W, S, f32, ws)


@pytest.mark.parametrize("lens,new,hq,h,d,page,W,S", WINDOWS)
@pytest.mark.parametrize("cache", ["f16", "e4m3"])
def test_window_wide_table(pkv, cuda_dev, lens, new, hq, h, d, page, W, S, cache):
    """Tables much wider than the contexts (more than a few rows: parts that have no tiles),
    and unseen blocks that are in the table but hold no numbers."""
    window_case(pkv, cuda_dev, cache, lens, new, hq, h, d, page, W, S, False, True, wide=True, poison=True)


def test_window_as_wide_as_the_context_is_causal(pkv, cuda_dev):
    """What pf_paged_prefill_attention gives, to the same bound (its tiles are others, so not bit for bit)."""
    import torch
    c = Ctx(pkv, cuda_dev, "f16", [300, 77], 4, 2, 64, 16)
    offs = offsets([200, 77])
    q = c.rng.standard_normal((277, 4, 64)).astype(np.float16)
    want, tol = c.want(q, offs, [window_seen(L, n, L, 0) for L, n in ((300, 200), (77, 77))], F16, F16)
    args = (c.pool, 1, dev(q, cuda_dev), dev(c.table, cuda_dev), dev(c.lens, cuda_dev), dev(offs, cuda_dev), 200, 0.125)
    for call in (lambda o: pkv.pf_paged_window_attention(*args, 300, 0, o), lambda o: pkv.pf_paged_prefill_attention(*args, o)):
        out = torch.empty((277, 4, 64), dtype=torch.float16, device=cuda_dev)
        call(out)
        assert_within(host(out), want, tol)


# -------------------------------------------------------------------- trees

def trees_for(rng, kind, new):
    out = []
    for n in new:
        x = random_tree(rng, n)
        if kind == "any":                                 # bits of no tree at all
            x = rng.random((n, n)) < 0.3
        elif kind == "empty":                             # some drafts see no draft
            x[::3] = False
        elif kind == "chain":
            x = np.tril(np.ones((n, n), bool))
        out.append(x)
    return out


TREES = [
    # lengths, drafts, q-heads, kv-heads, head_dim, page
    ([200, 9, 1, 30], [8, 9, 1, 0], 12, 12, 64, 16),
    ([600, 33, 2], [2, 2, 1], 14, 2, 64, 64),
    ([40, 90], [16, 3], 5, 5, 128, 1),
    ([20, 700], [4, 4], 12, 3, 128, 256),
    ([3000], [16], 1, 1, 64, 16),
    ([2500, 16], [7, 16], 2, 2, 64, 1),
    ([3000, 64], [1, 1], 16, 1, 128, 16),
    ([300, 64, 65, 100], [64, 64, 65, 37], 4, 2, 64, 16),
    ([500, 200], [200, 200], 3, 3, 128, 16),
    ([700, 33], [130, 33], 8, 2, 128, 64),
    ([260, 191], [129, 191], 2, 2, 64, 256),
    ([300, 20], [63, 18], 14, 2, 64, 1),
    ([5000, 600, 63], [33, 40, 17], 2, 1, 128, 16),
    ([9000], [64], 7, 1, 64, 64),
    ([9000], [200], 4, 2, 128, 64),
    ([4200, 65, 129], [70, 65, 3], 3, 1, 64, 1),
    ([300, 300], [300, 260], 1, 1, 64, 16),
    ([1500, 900], [700, 1], 2, 1, 128, 16),
]


def tree_case(pkv, cuda_dev, cache, lens, new, hq, h, d, page, kind, f32, ws, wide=False, extra_words=0):
    import torch
    c = Ctx(pkv, cuda_dev, cache, lens, hq, h, d, page)
    offs = offsets(new)
    q = c.rng.standard_normal((int(offs[-1]), hq, d)).astype(np.float16)
    trees = trees_for(c.rng, kind, new)
    seen = [tree_seen(L, x) for L, x in zip(lens, trees)]
    bits = dev(pack(trees, -(-max(new) // 64) + extra_words, c.rng), cuda_dev)
    table = dev(c.table, cuda_dev)
    if wide:
        table = torch.nn.functional.pad(table, (0, 8192 // page), value=1 << 30)
    work = pkv.make_tree_workspace(c.pool, len(lens), hq, table.shape[1], max(new)) if ws else None
    assert work is not None or not ws or max(new) * (hq // h) > 16
    qd, ld, cu = dev(q, cuda_dev), dev(c.lens, cuda_dev), dev(offs, cuda_dev)
    check(c, q, offs, seen, lambda out, w: pkv.pf_paged_tree_attention(c.pool, 1, qd, table, ld, cu, max(new), c.scale, bits, out,
                                                                       w), work, f32)


@pytest.mark.parametrize("lens,new,hq,h,d,page", TREES)
@pytest.mark.parametrize("cache", ["f16", "e4m3"])
@pytest.mark.parametrize("kind,f32,ws", [("tree", False, True), ("any", True, True), ("empty", False, False), ("empty", True, True)])
def test_tree(pkv, cuda_dev, lens, new, hq, h, d, page, cache, kind, f32, ws):
    tree_case(pkv, cuda_dev, cache, lens, new, hq, h, d, page, kind, f32, ws)


@pytest.mark.parametrize("lens,new,hq,h,d,page", TREES)
@pytest.mark.parametrize("cache", ["f16", "e4m3"])
def test_tree_wide_table(pkv, cuda_dev, lens, new, hq, h, d, page, cache):
    """Wide tables and rows of more words than the drafts need."""
    tree_case(pkv, cuda_dev, cache, lens, new, hq, h, d, page, "empty", False, True, wide=True, extra_words=2)


def test_a_chain_is_causal(pkv, cuda_dev):
    """Drafts in a row: the result of pf_paged_prefill_attention, to both calls' bounds."""
    import torch
    c = Ctx(pkv, cuda_dev, "e4m3", [300, 77], 4, 2, 64, 16)
    new = [150, 77]
    offs = offsets(new)
    q = c.rng.standard_normal((227, 4, 64)).astype(np.float16)
    trees = trees_for(c.rng, "chain", new)
    want, tol = c.want(q, offs, [tree_seen(L, x) for L, x in zip(c.lens, trees)], F16, F16)
    args = (c.pool, 1, dev(q, cuda_dev), dev(c.table, cuda_dev), dev(c.lens, cuda_dev), dev(offs, cuda_dev), 150, c.scale)
    for call in (lambda o: pkv.pf_paged_prefill_attention(*args, o),
                 lambda o: pkv.pf_paged_tree_attention(*args, dev(pack(trees, 3), cuda_dev), o)):
        out = torch.empty((227, 4, 64), dtype=torch.float16, device=cuda_dev)
        call(out)
        assert_within(host(out), want, tol)


# ------------------------------------------------------------------- common

def test_flags(pkv, cuda_dev):
    """Lengths past the table, more new tokens than the bound or the context, bad blocks that a query sees."""
    import torch
    c = Ctx(pkv, cuda_dev, "f16", [40, 40], 2, 2, 64, 16)
    bits = dev(np.full((40, 1), -1, np.int64), cuda_dev)
    bad = c.table.copy()
    bad[1, 2] = 10 ** 6
    for n in (3, 20):
        q = dev(np.zeros((2 * n, 2, 64), np.float16), cuda_dev)
        cu = dev(offsets([n, n]), cuda_dev)
        for ws in (True, False):
            work = pkv.make_window_workspace(c.pool, 2, 2, c.table.shape[1], n, 9, 2) if ws else None
            out = torch.empty_like(q)

            def both(table, lens, cu, most, flag):
                lens = dev(np.array(lens, np.int32), cuda_dev)
                for call in (lambda: pkv.pf_paged_window_attention(c.pool, 0, q, dev(table, cuda_dev), lens, cu, most, 0.125, 9, 2,
                                                                   out, work),
                             lambda: pkv.pf_paged_tree_attention(c.pool, 0, q, dev(table, cuda_dev), lens, cu, most, 0.125,
                                                                 bits[:2 * n], out, work)):
                    call()
                    assert pkv.pf_device_status(reset=True) == flag
            pkv.pf_device_status(reset=True)
            both(c.table, [40, 40], cu, n, 0)
            both(c.table, [40, 10 ** 6], cu, n, pkv.PF_DEV_BAD_LENGTH)
            both(c.table, [40, -1], cu, n, pkv.PF_DEV_BAD_LENGTH)
            both(c.table, [40, n - 1], cu, n, pkv.PF_DEV_BAD_LENGTH)
            both(c.table, [40, 40], cu, n - 1, pkv.PF_DEV_BAD_LENGTH)
            both(bad, [40, 40], cu, n, pkv.PF_DEV_BAD_BLOCK_ID)


@pytest.mark.parametrize("n", [3, 20])
def test_loose_bounds(pkv, cuda_dev, n):
    """The largest max_new_tokens there is: what the table holds."""
    import torch
    c = Ctx(pkv, cuda_dev, "f16", [60, 50], 4, 2, 64, 16)
    offs = offsets([n, n])
    q = c.rng.standard_normal((2 * n, 4, 64)).astype(np.float16)
    seen = [window_seen(L, n, 21, 3) for L in (60, 50)]
    want, tol = c.want(q, offs, seen, F16, F16)
    most = 2 ** 31 - 1
    ws = pkv.make_window_workspace(c.pool, 2, 4, c.table.shape[1], most, 21, 3)
    out = torch.empty((2 * n, 4, 64), dtype=torch.float16, device=cuda_dev)
    pkv.pf_paged_window_attention(c.pool, 1, dev(q, cuda_dev), dev(c.table, cuda_dev), dev(c.lens, cuda_dev), dev(offs, cuda_dev),
                                  most, c.scale, 21, 3, out, ws)
    assert_within(host(out), want, tol)


@pytest.mark.parametrize("cache", ["f16", "e4m3"])
def test_many_sequences(pkv, cuda_dev, cache):
    """More sequences than one launch of the few-rows kernel takes."""
    lens = [1 + (37 * i) % 80 for i in range(1500)]
    window_case(pkv, cuda_dev, cache, lens, None, 2, 2, 64, 16, 20, 2, False, True, wide=True)
    tree_case(pkv, cuda_dev, cache, lens, [min(L, 1 + i % 4) for i, L in enumerate(lens)], 2, 2, 64, 16, "empty", False, True,
              wide=True)


def test_far_blocks(pkv, cuda_dev):
    """Blocks past 2^32 bytes of the pool."""
    import torch
    n_blocks, B, H, D = 8600, 256, 8, 128
    k, v = (torch.empty((1, n_blocks, B, H, D), dtype=torch.float16, device=cuda_dev) for _ in range(2))
    pool = pkv.pf_pool_create(k, v)
    ids = [n_blocks - 1, n_blocks - 3, n_blocks - 2]
    rng = np.random.default_rng(3)
    rows = [rng.standard_normal((3, B, H, D)).astype(np.float16) for _ in range(2)]
    for x, r in zip((k, v), rows):
        x[0, dev(np.array(ids), cuda_dev)] = dev(r, cuda_dev)
    kk, vv = (r.reshape(3 * B, H, D) for r in rows)
    table, lens = dev(np.array([ids], np.int32), cuda_dev), dev(np.array([700], np.int32), cuda_dev)
    for n in (1, 40):
        q = rng.standard_normal((n, 16, D)).astype(np.float16)
        cu = dev(np.array([0, n], np.int32), cuda_dev)
        x = random_tree(rng, n)
        for seen, call in ((window_seen(700, n, 300, 5), lambda o, w: pkv.pf_paged_window_attention(
                pool, 0, dev(q, cuda_dev), table, lens, cu, n, 0.09, 300, 5, o, w)),
                           (tree_seen(700, x), lambda o, w: pkv.pf_paged_tree_attention(
                               pool, 0, dev(q, cuda_dev), table, lens, cu, n, 0.09, dev(pack([x], 1), cuda_dev), o, w))):
            want, tol = masked64(q, kk[:700], vv[:700], float(np.float32(0.09)), seen, F16, F16)
            for w in (None, pkv.make_tree_workspace(pool, 1, 16, 3, n)):
                out = torch.empty((n, 16, D), dtype=torch.float16, device=cuda_dev)
                call(out, w)
                assert_within(host(out), want, tol)


@pytest.mark.parametrize("hq,d", [(1, 64), (16, 128), (3, 128)])
@pytest.mark.parametrize("n", [1, 40])
def test_very_long_context(pkv, cuda_dev, hq, d, n):
    """A table that names the same eight pages over and over: a window of whole rounds of them and one
    round of sinks, or drafts that see nothing but the context, give what those pages give once."""
    import torch
    c = PagedCase(pkv, cuda_dev, [8 * 256], hq, 1, d, 256)
    rounds = 500
    table = dev(np.concatenate([np.tile(c.bt, (1, rounds)), c.bt[:, :1]], 1), cuda_dev)
    t = np.arange(8 * 256)
    k, v = (x[0][c.bt[0][t // 256], t % 256] for x in (c.k_host, c.v_host))
    rng = np.random.default_rng(1)
    q = rng.standard_normal((n, hq, d)).astype(np.float16)
    scale = float(np.float32(d ** -0.5))
    want, tol = masked64(q, k, v, scale, np.ones((n, len(t)), bool), F16, F16)
    # sums over 2^20 terms, not over the eight pages': at most 2^14 stages or tiles in order, each step off by
    # 2^-23 of the sum, then 2^8 parts at most
    tol = tol + np.abs(v.astype(np.float64)).mean() * 2 * (2.0 ** 14 + 2.0 ** 8) * 2.0 ** -23
    L = rounds * len(t)
    cu = dev(np.array([0, n], np.int32), cuda_dev)
    ws = pkv.make_tree_workspace(c.pool, 1, hq, table.shape[1], n)
    out = torch.empty((n, hq, d), dtype=torch.float16, device=cuda_dev)
    pkv.pf_device_status(reset=True)
    for w in (ws, None):
        pkv.pf_paged_window_attention(c.pool, 0, dev(q, cuda_dev), table, dev(np.array([L], np.int32), cuda_dev), cu, n, scale,
                                      400 * len(t), len(t), out, w)
        assert pkv.pf_device_status(reset=True) == 0
        assert_within(host(out), want, tol)
        bits = torch.zeros((n, 1), dtype=torch.int64, device=cuda_dev)
        pkv.pf_paged_tree_attention(c.pool, 0, dev(q, cuda_dev), table, dev(np.array([L + n], np.int32), cuda_dev), cu, n, scale,
                                    bits, out, w)
        assert pkv.pf_device_status(reset=True) == 0
        assert_within(host(out), want, tol)


def test_blocks_of_more_than_a_second(pkv, cuda_dev):
    """Six blocks of rows one after another for each SM, over 140 million tokens each (eight pages, over and over)."""
    import torch
    c = PagedCase(pkv, cuda_dev, [8 * 256], 16, 1, 128, 256)
    c.v_dev.fill_(0.75)
    rounds = 70000
    table = dev(c.bt, cuda_dev).repeat(1, rounds)
    n = 16 * torch.cuda.get_device_properties(cuda_dev).multi_processor_count * 5 + 16
    q = torch.randn((n, 16, 128), dtype=torch.float16, device=cuda_dev)
    out = torch.full_like(q, float("nan"))
    cu = dev(np.array([0, n], np.int32), cuda_dev)
    L = rounds * 8 * 256
    pkv.pf_device_status(reset=True)
    pkv.pf_paged_window_attention(c.pool, 0, q, table, dev(np.array([L], np.int32), cuda_dev), cu, n, 128 ** -0.5, L, 0, out)
    assert pkv.pf_device_status(reset=True) == 0
    # every row is there (sums of so many tokens in fp32 are not to be exact)
    assert bool((out > 0).all()) and bool((out < 1.5).all())


def test_two_calls_at_once(pkv, cuda_dev):
    """Calls on two streams over one pool, each with a workspace of its own."""
    import torch
    c = Ctx(pkv, cuda_dev, "e4m3", [3000, 500], 4, 2, 64, 16)
    table, lens = dev(c.table, cuda_dev), dev(c.lens, cuda_dev)
    jobs = []
    for n, W in ((1, 700), (60, 1500), (3, 40), (200, 100)):
        offs = offsets([n, n])
        q = c.rng.standard_normal((2 * n, 4, 64)).astype(np.float16)
        seen = [window_seen(L, n, W, 5) for L in c.lens]
        jobs.append((n, W, dev(q, cuda_dev), dev(offs, cuda_dev), torch.empty((2 * n, 4, 64), dtype=torch.float16, device=cuda_dev),
                     pkv.make_window_workspace(c.pool, 2, 4, table.shape[1], n, W, 5), torch.cuda.Stream(), *c.want(q, offs, seen, F16, F16)))
    torch.cuda.synchronize()
    for _ in range(20):
        for n, W, q, cu, out, ws, stream, _, _ in jobs:
            pkv.pf_paged_window_attention(c.pool, 1, q, table, lens, cu, n, c.scale, W, 5, out, ws, stream=stream)
    torch.cuda.synchronize()
    for n, W, q, cu, out, ws, stream, want, tol in jobs:
        assert_within(host(out), want, tol, f"{n} {W}")
    assert pkv.pf_device_status(reset=True) == 0


def test_replays_share_a_workspace(pkv, cuda_dev):
    """Captured calls of both kinds, few rows and many, over one workspace, replayed in turn on new inputs."""
    import torch
    c = Ctx(pkv, cuda_dev, "f16", [6000, 700], 4, 1, 64, 16)
    table, lens = dev(c.table, cuda_dev), dev(c.lens, cuda_dev)
    width = table.shape[1]
    ws = torch.empty(max(pkv.pf_window_workspace_bytes(c.pool, 2, 4, width, 40, 3000, 4),
                         pkv.pf_tree_workspace_bytes(c.pool, 2, 4, width, 40),
                         pkv.pf_tree_workspace_bytes(c.pool, 2, 4, width, 4)), dtype=torch.uint8, device=cuda_dev)
    pkv.pf_decode_workspace_init(ws)
    graphs = []
    for n in (2, 40):
        offs = offsets([n, n])
        q = torch.zeros((2 * n, 4, 64), dtype=torch.float16, device=cuda_dev)
        cu = dev(offs, cuda_dev)
        trees = trees_for(c.rng, "empty", [n, n])
        bits = dev(pack(trees, 1), cuda_dev)
        for call, seen in (
                (lambda o, q=q, cu=cu, n=n: pkv.pf_paged_window_attention(c.pool, 1, q, table, lens, cu, n, c.scale, 3000, 4, o, ws),
                 [window_seen(L, n, 3000, 4) for L in c.lens]),
                (lambda o, q=q, cu=cu, n=n, b=bits: pkv.pf_paged_tree_attention(c.pool, 1, q, table, lens, cu, n, c.scale, b, o, ws),
                 [tree_seen(L, x) for L, x in zip(c.lens, trees)])):
            out = torch.empty_like(q)
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                call(out)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                call(out)
            graphs.append((g, q, out, offs, seen))
    for i in range(12):
        g, q, out, offs, seen = graphs[(5 * i) % len(graphs)]
        qn = c.rng.standard_normal(tuple(q.shape)).astype(np.float16)
        q.copy_(dev(qn, cuda_dev))
        g.replay()
        torch.cuda.synchronize()
        assert_within(host(out), *c.want(qn, offs, seen, F16, F16), f"replay {i}")
    assert pkv.pf_device_status(reset=True) == 0


@pytest.mark.parametrize("cache", ["f16", "e4m3"])
def test_a_layer_with_drafts(pkv, cuda_dev, cache):
    """The calls together, as drafts are checked with them: the prompt rotated, written and attended under a
    window; drafts rotated for their depth, written and attended as a tree; the accepted path written again
    where it belongs; a decode step over the result."""
    import torch
    B, H, HQ, D, W, S, L, n = 16, 2, 4, 64, 40, 4, 100, 7
    rng = np.random.default_rng(2)
    parent = [-1, 0, 0, 1, 1, 2, 3]
    sees = np.zeros((n, n), bool)
    depth = np.zeros(n, np.int32)
    for i, p in enumerate(parent):
        if p >= 0:
            sees[i], depth[i] = sees[p], depth[p] + 1
        sees[i, i] = True
    path = [0, 1, 3]                                              # accepted
    alloc = pkv.pf_alloc_create(12, 5)
    row = np.zeros(10, np.int32)
    pkv.pf_seq_reserve(alloc, B, row, 0, L + n)
    table, seq = dev(row[None], cuda_dev), lambda m: dev(np.zeros(m, np.int32), cuda_dev)   # noqa: E731
    if cache == "f16":
        pool = pkv.pf_pool_create(*(torch.zeros((1, 12, B, H, D), dtype=torch.float16, device=cuda_dev) for _ in range(2)))
    else:
        pool = pkv.pf_pool_create(*(torch.zeros((1, 12, B, H, D), device=cuda_dev).to(torch.float8_e4m3fn) for _ in range(2)),
                                  *(torch.zeros((1, 12, H), device=cuda_dev) for _ in range(2)))
    angles = pkv.make_rope_angles(200, D, device=cuda_dev)
    w = torch.ones(D, device=cuda_dev)
    kept = []                                                     # rotated K and V rows as written, by slot

    def write(rows, slots, positions):
        """q of these rows, with K and V in the cache (slots: consecutive)."""
        x = dev(rows, cuda_dev)
        q, k, v = x[:, :HQ], x[:, HQ:HQ + H], x[:, HQ + H:]
        m = len(rows)
        q_out = torch.empty((m, HQ, D), dtype=torch.float16, device=cuda_dev)
        k_out = torch.empty((m, H, D), dtype=torch.float16, device=cuda_dev)
        rp = dev(positions.astype(np.int32), cuda_dev)
        common = dict(q_weight=w, k_weight=w, rope_pos=rp)
        if cache == "f16":
            pkv.pf_norm_rope_write(pool, 0, q, k, v, table, seq(m), dev(slots.astype(np.int32), cuda_dev), angles, q_out, k_out,
                                   **common)
        else:
            pkv.pf_norm_rope_write(pool, 0, q, k, None, None, None, None, angles, q_out, k_out, **common)
            pkv.pf_append_kv(pool, 0, k_out, v.contiguous(), table, dev(np.array([slots[-1] + 1], np.int32), cuda_dev),
                             dev(np.array([0, m], np.int32), cuda_dev), m)
        del kept[slots[0]:]
        kept.extend((host(k_out)[i], rows[i, HQ + H:]) for i in range(m))
        return q_out

    def cached():
        """The rows as attention reads them: gathered from the pages."""
        m = len(kept)
        got = [torch.empty((m, H, D), dtype=torch.float16, device=cuda_dev) for _ in range(2)]
        pkv.pf_gather_kv(pool, 0, table, dev(np.array([m], np.int32), cuda_dev), dev(np.zeros(1, np.int64), cuda_dev), *got)
        k, v = (host(x) for x in got)
        for have, put in ((k, [a for a, _ in kept]), (v, [b for _, b in kept])):
            put = np.stack(put).astype(np.float64)
            # e4m3: half a step of the value, or of its block's smallest step at a scale of 2^-7 and less
            assert np.all(np.abs(have - put) <= (0 if cache == "f16" else np.abs(put) * 2.0 ** -4 + 2.0 ** -10 * 8))
        return k, v

    def compare(out, q_out, seen, m):
        k, v = cached()
        want, tol = masked64(host(q_out), k, v, 0.125, seen, F16, F16)
        # (what the kernels read is code * scale: exact in fp16 but below 2^-14, off by 2^-25 there)
        more = 0 if cache == "f16" else 2.0 ** -25 * (1 + 2 * 0.125 * np.abs(host(q_out).astype(np.float64)).sum(-1).max() *
                                                      np.abs(v.astype(np.float64)).max()) * (1 + m)
        assert_within(host(out), want, tol + more)

    i32 = lambda *x: dev(np.array(x, np.int32), cuda_dev)         # noqa: E731
    pkv.pf_device_status(reset=True)
    prompt = rng.standard_normal((L, HQ + 2 * H, D)).astype(np.float16)
    q = write(prompt, np.arange(L), np.arange(L))
    out = torch.empty_like(q)
    pkv.pf_paged_window_attention(pool, 0, q, table, i32(L), i32(0, L), L, 0.125, W, S, out,
                                  pkv.make_window_workspace(pool, 1, HQ, 10, L, W, S))
    compare(out, q, window_seen(L, L, W, S), L)
    drafts = rng.standard_normal((n, HQ + 2 * H, D)).astype(np.float16)
    q = write(drafts, L + np.arange(n), L + depth)
    out = torch.empty_like(q)
    pkv.pf_paged_tree_attention(pool, 0, q, table, i32(L + n), i32(0, n), n, 0.125, dev(pack([sees], 1), cuda_dev), out,
                                pkv.make_tree_workspace(pool, 1, HQ, 10, n))
    compare(out, q, tree_seen(L + n, sees), L + n)
    accepted = host(out)[path[-1]]
    q = write(drafts[path], L + np.arange(len(path)), L + np.arange(len(path)))
    now = L + len(path)
    out = torch.empty((1, HQ, D), dtype=torch.float16, device=cuda_dev)
    last = q[-1:].contiguous()
    pkv.pf_paged_decode_attention(pool, 0, last, table, i32(now), 0.125, out, 0, pkv.make_workspace(pool, 1, HQ, 10, 0))
    k, v = cached()
    want, tol = masked64(host(last), k, v, 0.125, window_seen(now, 1, now, 0), F16, F16)
    assert_within(host(out), want, 2 * tol + (0 if cache == "f16" else 2.0 ** -17))
    # the accepted draft saw what the last token of the kept path sees
    if cache == "f16":
        assert_within(accepted[None], want, 2 * tol)
    assert pkv.pf_device_status(reset=True) == 0


def test_long_blocks_with_rows_for_one_query_tile(pkv, cuda_dev):
    """Two blocks of more than a second one after another on each SM, the first of 64 rows, so that half of the
    softmax warps wait as long as the others work; 205 million tokens, of whose pages three, the first, one in the
    middle and the last, hold values that are not 0, each in dims of its own.  All scores are 0, so an output
    is such a page's values over the number of tokens seen: sums of 256 times 60000 and of ones are exact in fp32
    (but for the last tile's ones, 2^-24), and the quotient is off by 2^-22 and its rounding."""
    import torch
    c = PagedCase(pkv, cuda_dev, [8 * 256], 16, 1, 128, 256)
    c.v_dev.zero_()
    ids = [int(x) for x in c.bt[0]]
    for i, page in enumerate(ids[:3]):
        c.v_dev[0, page, :, :, 32 * i:32 * i + 32] = 60000.0
    seqs = torch.cuda.get_device_properties(cuda_dev).multi_processor_count
    pages, n = 800001, 20
    row = torch.tensor(ids[3:], dtype=torch.int32, device=cuda_dev).repeat(pages // 5 + 1)[:pages]
    row[0], row[pages // 2], row[pages - 1] = ids[0], ids[1], ids[2]
    table = row.expand(seqs, pages).contiguous()
    L = 256 * (pages - 1) + 128
    q = torch.zeros((seqs * n, 16, 128), dtype=torch.float16, device=cuda_dev)
    out = torch.full_like(q, float("nan"))
    cu = dev(np.arange(seqs + 1, dtype=np.int32) * n, cuda_dev)
    pkv.pf_device_status(reset=True)
    pkv.pf_paged_window_attention(c.pool, 0, q, table, dev(np.full(seqs, L, np.int32), cuda_dev), cu, n, 128 ** -0.5, L, 0, out)
    assert pkv.pf_device_status(reset=True) == 0
    seen = L - n + 1 + np.arange(n)
    count = np.stack([np.full(n, 256), np.full(n, 256), seen - 256 * (pages - 1), np.zeros(n)], 1)      # of each page's
    want = np.tile(np.repeat(60000.0 * count / seen[:, None], 32, 1), (seqs, 1))[:, None]
    assert_within(host(out), np.broadcast_to(want, out.shape), np.broadcast_to(want * (F16 + 2.0 ** -21), out.shape))


@pytest.mark.parametrize("cache,d", [("f16", 64), ("e4m3", 128)])
def test_bounds_as_loose_as_there_are(pkv, cuda_dev, cache, d):
    """max_new_tokens as large as a table of 2^26 tokens (2 thousand million blocks of rows, nearly all of them
    empty) and drafts of up to 2^20: 480 (sequence, kv-head) pairs, some without tokens or without new ones."""
    import torch
    page, seqs, h, g = 256, 60, 8, 16
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(0, 500, seqs)]
    new = [min(L, int(n)) for L, n in zip(lens, rng.integers(0, 24, seqs))]
    lens[7] = new[7] = new[20] = 0
    c = Ctx(pkv, cuda_dev, cache, lens, h * g, h, d, page)
    offs = offsets(new)
    q = c.rng.standard_normal((int(offs[-1]), h * g, d)).astype(np.float16)
    table = torch.nn.functional.pad(dev(c.table, cuda_dev), (0, 2 ** 26 // page - c.table.shape[1]), value=1 << 30)
    qd, ld, cu = dev(q, cuda_dev), dev(c.lens, cuda_dev), dev(offs, cuda_dev)
    check(c, q, offs, [window_seen(L, n, 90, 5) for L, n in zip(lens, new)],
          lambda out, w: pkv.pf_paged_window_attention(c.pool, 1, qd, table, ld, cu, 2 ** 31 - 1, c.scale, 90, 5, out, w), None, False)
    trees = trees_for(c.rng, "empty", new)
    bits = torch.nn.functional.pad(dev(pack(trees, 1), cuda_dev), (0, 2 ** 14 - 1), value=-1)
    check(c, q, offs, [tree_seen(L, x) for L, x in zip(lens, trees)],
          lambda out, w: pkv.pf_paged_tree_attention(c.pool, 1, qd, table, ld, cu, 2 ** 20, c.scale, bits, out, w), None, False)


class Marked:
    """A long context of one sequence: eight pages of zeros over and over, but for `marked` entries of its table,
    each a page of its own with values in dims of its own.  Weights of the zero rows are all alike, so a few
    thousand tokens and a count give the 64-bit result, and a marked page or token read in the wrong place shows.
    All numbers are e4m3's, so that both pool types hold the same."""

    def __init__(self, device, cache, hq, d, pages, marked, loud, pkv, seed=11):
        import torch
        rng = np.random.default_rng(seed)
        self.d, self.hq, self.marked, B = d, hq, np.asarray(marked), 256
        k, v = np.zeros((8 + len(marked), B, 1, d), np.float32), np.zeros((8 + len(marked), B, 1, d), np.float32)
        k[8:] = rng.choice([-3.0, -2.0, -1.5, -1.0, 1.0, 1.5, 2.0, 3.0], k[8:].shape)
        own = d // len(marked)
        for i, entry in enumerate(marked):
            v[8 + i, :, 0, own * i:own * (i + 1)] = rng.choice([5.0, 6.0, 7.0], (B, own))
            for t in loud:                                # tokens at a border: 64 times as much
                if t // B == entry:
                    v[8 + i, t % B] *= 64
        to = torch.float16 if cache == "f16" else torch.float8_e4m3fn
        pools = [dev(x, device)[None].to(to) for x in (k, v)]
        scales = [] if cache == "f16" else [torch.ones((1, len(k), 1), device=device) for _ in range(2)]
        self.keep = pools + scales
        self.pool = pkv.pf_pool_create(*pools, *scales)
        table = np.resize(np.arange(8, dtype=np.int32), pages)
        table[self.marked] = 8 + np.arange(len(marked))
        self.table = dev(table[None], device)
        self.at = (self.marked[:, None] * B + np.arange(B)).reshape(-1)      # marked tokens, and their rows
        self.k, self.v = (x[8:].astype(np.float64).reshape(-1, d) for x in (k, v))
        self.scale = float(np.float32(d ** -0.5))

    def want(self, q, seen, total, tiles):
        """seen [n, marked tokens], total [n]: tokens seen of all.  The bound is masked64's, with fp32 sums of the
        weights over `tiles` steps, each off by 2^-24 of the sum (twice: the products' too)."""
        q = q.astype(np.float64)
        z = np.where(seen[:, None], np.einsum("nhd,td->nht", q, self.k) * self.scale, -np.inf)
        size = np.einsum("nhd,td->nht", np.abs(q), np.abs(self.k)).max(-1) * self.scale
        zeros = (total - seen.sum(-1))[:, None].astype(np.float64)
        assert (zeros > 0).all()
        m = np.maximum(z.max(-1), 0.0)
        w = np.exp(z - m[..., None])
        sum_w = w.sum(-1) + zeros * np.exp(-m)
        out, A = (np.einsum("nht,td->nhd", w, x) / sum_w[..., None] for x in (self.v, np.abs(self.v)))
        e = size * (self.d + 4) * 2.0 ** -23 + (np.maximum(m, np.where(seen[:, None], np.abs(z), 0).max(-1)) + 16) * 2.0 ** -22
        tol = A * (2 * e[..., None] + F16 + tiles * 2.0 ** -23)
        small = np.einsum("nt,td->nd", seen.astype(np.float64), np.abs(self.v)) * 2.0 ** -25
        return out, tol + small[:, None] / sum_w[..., None] + np.abs(out) * F16 + 2.0 ** -25


@pytest.mark.parametrize("cache", ["f16", "e4m3"])
@pytest.mark.parametrize("hq,d", [(1, 64), (16, 128), (3, 128)])
@pytest.mark.parametrize("n", [1, 40, 200])
def test_places_in_a_very_long_context(pkv, cuda_dev, cache, hq, d, n):
    """A million tokens: sinks, what lies behind them, both sides of the window's border, its middle and the end,
    each a page of its own; every border lies inside a page."""
    import torch
    pages, first, S = 4000, 1500, 100
    L = 256 * pages - 90
    W = L - n + 1 - (256 * first + 77)                    # the first query sees tokens from 77 of page `first` on
    loud = [*range(S - 4, S + 4), *range(256 * first + 70, 256 * first + 90), *range(L - n - 4, L)]
    c = Marked(cuda_dev, cache, hq, d, pages, [0, 1, first - 1, first, 2700, pages - 2, pages - 1], loud, pkv)
    q = np.random.default_rng(n).standard_normal((n, hq, d)).astype(np.float16)
    p = np.arange(L - n, L)[:, None]
    lens, cu = dev(np.array([L], np.int32), cuda_dev), dev(np.array([0, n], np.int32), cuda_dev)
    qd, out = dev(q, cuda_dev), torch.empty((n, hq, d), dtype=torch.float16, device=cuda_dev)
    pkv.pf_device_status(reset=True)
    seen = (c.at <= p) & ((c.at > p - W) | (c.at < S))
    ws = pkv.make_window_workspace(c.pool, 1, hq, pages, n, W, S)
    want = c.want(q, seen, (np.minimum(W, p + 1) + np.minimum(S, np.maximum(0, p - W + 1)))[:, 0], 2 ** 14 + 2 ** 8)
    for w in (ws, None):
        pkv.pf_paged_window_attention(c.pool, 0, qd, c.table, lens, cu, n, c.scale, W, S, out, w)
        assert pkv.pf_device_status(reset=True) == 0
        assert_within(host(out), *want)
    sees = random_tree(np.random.default_rng(n), n)
    bits = dev(pack([sees], -(-n // 64)), cuda_dev)
    draft = c.at - (L - n)
    seen = np.where(draft < 0, True, sees[:, np.clip(draft, 0, n - 1)] & (draft < n))
    ws = pkv.make_tree_workspace(c.pool, 1, hq, pages, n)
    want = c.want(q, seen, L - n + sees.sum(1), 2 ** 14 + 2 ** 8)
    for w in (ws, None):
        pkv.pf_paged_tree_attention(c.pool, 0, qd, c.table, lens, cu, n, c.scale, bits, out, w)
        assert pkv.pf_device_status(reset=True) == 0
        assert_within(host(out), *want)


@pytest.mark.parametrize("cache", ["f16", "e4m3"])
@pytest.mark.parametrize("lens,n,hq,h,d", [([3000, 40, 700], 1, 14, 2, 64), ([6000, 5], 3, 8, 2, 128), ([9000], 30, 7, 1, 64),
                                           ([900, 1200, 300], 60, 8, 2, 128), ([2000] * 40, 20, 8, 8, 64)])
def test_the_same_bits_again(pkv, cuda_dev, cache, lens, n, hq, h, d):
    """Contexts cut over the SMs are joined in one order: a call gives the same bits every time, also between others."""
    import torch
    c = Ctx(pkv, cuda_dev, cache, lens, hq, h, d, 16)
    new = [min(n, L) for L in lens]
    offs = offsets(new)
    table, ld, cu = dev(c.table, cuda_dev), dev(c.lens, cuda_dev), dev(offs, cuda_dev)
    q = dev(c.rng.standard_normal((int(offs[-1]), hq, d)).astype(np.float16), cuda_dev)
    bits = dev(pack(trees_for(c.rng, "empty", new), 1), cuda_dev)
    win, tre = (make(c.pool, len(lens), hq, table.shape[1], n, *more) for make, more in (
        (pkv.make_window_workspace, (800, 4)), (pkv.make_tree_workspace, ())))
    jobs = []
    for dtype in (torch.float16, torch.float32):
        jobs.append((lambda o: pkv.pf_paged_window_attention(c.pool, 1, q, table, ld, cu, n, c.scale, 800, 4, o, win), dtype))
        jobs.append((lambda o: pkv.pf_paged_tree_attention(c.pool, 1, q, table, ld, cu, n, c.scale, bits, o, tre), dtype))
    first = []
    for i in range(6):
        for j, (call, dtype) in enumerate(jobs):
            out = torch.empty(q.shape, dtype=dtype, device=cuda_dev)
            call(out)
            if i == 0:
                first.append(out)
            else:
                assert torch.equal(out, first[j]), (i, j)
