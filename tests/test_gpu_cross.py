"""Cross attention on the GPU against a plain 64-bit form: queries that see
the whole of a context whose length is its own, over fp16 and e4m3 pages, on
the few-rows kernel (with a workspace) and on the prompt kernel."""
import numpy as np
import pytest

from e4m3_util import assert_within, attention64
from gpu_util import PagedCase, dev, host
from test_gpu_e4m3 import F16, F32, Case

pytestmark = pytest.mark.gpu

CASES = [
    # context lengths, query tokens, q-heads, kv-heads, head_dim, page, workspace
    ([100, 0, 17, 1], [1, 2, 0, 3], 12, 12, 64, 16, True),
    ([600, 33, 1], [2, 2, 1], 14, 2, 64, 64, True),
    ([40, 90], [16, 3], 5, 5, 128, 1, True),
    ([1, 700], [4, 4], 12, 3, 128, 256, True),
    ([3000], [1], 2, 1, 128, 16, True),
    ([2000], [5], 3, 1, 64, 16, True),
    ([50, 0, 7], [5, 2, 0], 4, 4, 64, 16, False),             # few rows, no workspace
    ([0, 129, 1, 64], [130, 300, 140, 0], 2, 2, 64, 16, True),  # more queries than context
    ([512, 65], [100, 257], 8, 2, 128, 16, False),
    ([200, 31], [64, 40], 6, 2, 64, 1, False),
    ([700], [33], 4, 4, 128, 256, True),
]


@pytest.mark.parametrize("lens,new,hq,h,d,page,ws", CASES)
@pytest.mark.parametrize("cache", ["f16", "e4m3"])
@pytest.mark.parametrize("f32", [False, True])
def test_cross(pkv, cuda_dev, lens, new, hq, h, d, page, ws, cache, f32):
    _cross(pkv, cuda_dev, lens, new, hq, h, d, page, ws, cache, f32, False)


MANY = [([3 + 7 * i % 90 for i in range(40)], [1 + i % 3 for i in range(40)], 25, 5, 64, 16, True),
        ([3 + 7 * i % 90 for i in range(40)], [1 + i % 3 for i in range(40)], 20, 5, 128, 1, True)]


@pytest.mark.parametrize("lens,new,hq,h,d,page,ws", CASES[:6] + MANY)
@pytest.mark.parametrize("cache", ["f16", "e4m3"])
def test_cross_wide_table(pkv, cuda_dev, lens, new, hq, h, d, page, ws, cache):
    """Tables with room for 4096 more tokens: fp16 results from the few-rows kernel as well."""
    _cross(pkv, cuda_dev, lens, new, hq, h, d, page, ws, cache, False, True)


@pytest.mark.parametrize("lens,new,hq,h,d,page", [
    ([5000, 0, 600, 63], [33, 40, 17, 3], 2, 1, 128, 16),       # a part per context, several, none
    ([9000], [300], 4, 2, 64, 64),                             # two blocks of rows, the last one short
    ([1, 1024, 2047], [20, 20, 19], 3, 3, 64, 256),
    ([700, 1300], [6, 9], 12, 4, 128, 1),
    ([4100, 64, 65, 129], [129, 1, 128, 100], 1, 1, 64, 16),   # contexts of one and two tiles beside a cut one
])
@pytest.mark.parametrize("cache", ["f16", "e4m3"])
@pytest.mark.parametrize("f32", [False, True])
def test_cross_cut_contexts(pkv, cuda_dev, lens, new, hq, h, d, page, cache, f32):
    """Few blocks of many rows over long contexts: cut into parts, which are merged."""
    _cross(pkv, cuda_dev, lens, new, hq, h, d, page, True, cache, f32, False)


def _cross(pkv, cuda_dev, lens, new, hq, h, d, page, ws, cache, f32, wide):
    import torch
    offs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    rng = np.random.default_rng(9)
    q = rng.standard_normal((int(offs[-1]), hq, d)).astype(np.float16)
    scale = float(np.float32(1.0 / np.sqrt(d)))
    work_small = ws and max(new) * (hq // h) <= 16
    step = 2.0 ** -21 if f32 and work_small else F16
    if cache == "f16":
        c = PagedCase(pkv, cuda_dev, lens, hq, h, d, page, n_layers=2)
        pool, table, lens_dev = c.pool, c.bt_dev, c.lens_dev
        # rows past a context's end hold what must not be read as numbers
        for s, L in enumerate(lens):
            for t in range(L, -(-L // page) * page):
                for x in (c.k_dev, c.v_dev):
                    x[1, c.bt[s, t // page], t % page] = float("nan")

        def rows(x, s, L):
            t = np.arange(L)
            return x[1][c.bt[s][t // page], t % page]
        got = [attention64(q[offs[s]:offs[s + 1]], rows(c.k_host, s, L), rows(c.v_host, s, L), scale, False, step,
                           F32 if f32 else F16) for s, L in enumerate(lens)]
        want, tol = np.concatenate([o for o, _ in got]), np.concatenate([t for _, t in got])
    else:
        c = Case(pkv, cuda_dev, lens, hq, h, d, page)
        c.fill()
        pool, table, lens_dev = c.pool, c.table_dev, dev(c.lens, cuda_dev)
        want, tol = c.want(q, offs, False, step, F32 if f32 else F16)
        tol = tol + 2.0 ** -25 + 2 * 2.0 ** -25 * scale * np.abs(q.astype(np.float64)).sum(-1).max() * 64
    if wide:
        table = torch.nn.functional.pad(table, (0, 4096 // page), value=1 << 30)
    out = torch.full((int(offs[-1]) + 1, hq, d), 7.0, dtype=torch.float32 if f32 else torch.float16, device=cuda_dev)
    work = pkv.make_cross_workspace(pool, len(lens), hq, table.shape[1], max(new)) if ws else None
    step_tokens = 128 if d == 64 else 64
    blocks = len(lens) * h * -(-max(new) * (hq // h) // 256)
    cut = ws and min(torch.cuda.get_device_properties(cuda_dev).multi_processor_count // blocks,
                     -(-table.shape[1] * page // step_tokens) // 4) >= 2
    assert (work is not None) == (work_small or cut)
    pkv.pf_device_status(reset=True)
    for _ in range(2):
        pkv.pf_paged_cross_attention(pool, 1, dev(q, cuda_dev), table, lens_dev, dev(offs, cuda_dev), max(new), scale,
                                     out[:-1], work)
        assert pkv.pf_device_status(reset=True) == 0
        assert_within(host(out)[:-1], want, tol)
    assert bool((out[-1] == 7.0).all())


def test_one_query_is_decode_attention(pkv, cuda_dev):
    """A single query per sequence: the result of pf_paged_decode_attention, to the fp32 output's bound."""
    import torch
    c = PagedCase(pkv, cuda_dev, [300, 40, 1], 8, 4, 64, 16)
    plain = host(c.attention(0.125, out_dtype=torch.float32)).astype(np.float64)
    out = torch.empty((3, 8, 64), dtype=torch.float32, device=cuda_dev)
    ws = pkv.make_cross_workspace(c.pool, 3, 8, c.bt.shape[1], 1)
    pkv.pf_paged_cross_attention(c.pool, 0, c.q_dev, c.bt_dev, c.lens_dev, dev(np.arange(4, dtype=np.int32), cuda_dev),
                                 1, 0.125, out, ws)
    assert np.abs(host(out) - plain).max() <= 2e-5    # each within 1e-5 of the exact result


def test_rows_of_shared_pages(pkv, cuda_dev):
    """Several hypotheses of one input: table rows that name the same pages."""
    import torch
    c = PagedCase(pkv, cuda_dev, [200], 4, 4, 64, 16)
    table = np.repeat(c.bt, 5, axis=0)
    lens = np.full(5, 200, np.int32)
    q = np.random.default_rng(1).standard_normal((5, 4, 64)).astype(np.float16)
    out = torch.empty((5, 4, 64), dtype=torch.float16, device=cuda_dev)
    ws = pkv.make_cross_workspace(c.pool, 5, 4, table.shape[1], 1)
    pkv.pf_paged_cross_attention(c.pool, 0, dev(q, cuda_dev), dev(table, cuda_dev), dev(lens, cuda_dev),
                                 dev(np.arange(6, dtype=np.int32), cuda_dev), 1, 0.125, out, ws)
    t = np.arange(200)
    k, v = (x[0][c.bt[0][t // 16], t % 16] for x in (c.k_host, c.v_host))
    got = [attention64(q[i:i + 1], k, v, 0.125, False, F16, F16) for i in range(5)]
    assert_within(host(out), np.concatenate([o for o, _ in got]), np.concatenate([t for _, t in got]))


def test_flags(pkv, cuda_dev):
    import torch
    c = PagedCase(pkv, cuda_dev, [40, 40], 2, 2, 64, 16)
    q = dev(np.zeros((6, 2, 64), np.float16), cuda_dev)
    cu = dev(np.array([0, 3, 6], np.int32), cuda_dev)
    ws = pkv.make_cross_workspace(c.pool, 2, 2, c.bt.shape[1], 3)
    for work in (ws, None):
        out = torch.empty_like(q)
        pkv.pf_device_status(reset=True)
        pkv.pf_paged_cross_attention(c.pool, 0, q, c.bt_dev, dev(np.array([40, 10 ** 6], np.int32), cuda_dev), cu, 3,
                                     0.125, out, work)
        assert pkv.pf_device_status(reset=True) == pkv.PF_DEV_BAD_LENGTH
        pkv.pf_paged_cross_attention(c.pool, 0, q, c.bt_dev, c.lens_dev, cu, 2, 0.125, out, work)
        assert pkv.pf_device_status(reset=True) == pkv.PF_DEV_BAD_LENGTH
        bad = c.bt.copy()
        bad[1, 1] = 10 ** 6
        pkv.pf_paged_cross_attention(c.pool, 0, q, dev(bad, cuda_dev), c.lens_dev, cu, 3, 0.125, out, work)
        assert pkv.pf_device_status(reset=True) == pkv.PF_DEV_BAD_BLOCK_ID


@pytest.mark.parametrize("hq,d,tokens", [(1, 64, 1 << 20), (16, 128, 1 << 19), (3, 128, 40000)])
@pytest.mark.parametrize("f32", [False, True])
def test_very_long_context(pkv, cuda_dev, hq, d, tokens, f32):
    """One long context over all SMs, its parts merged by CTA and then over the
    CTAs: a table that names the same eight pages over and over, so the result
    is that of those pages once."""
    import torch
    c = PagedCase(pkv, cuda_dev, [8 * 256], hq, 1, d, 256)
    reps = tokens // (8 * 256)
    table = np.tile(c.bt, (1, reps))
    lens = dev(np.array([reps * 8 * 256], np.int32), cuda_dev)
    q = np.random.default_rng(1).standard_normal((1, hq, d)).astype(np.float16)
    out = torch.empty((1, hq, d), dtype=torch.float32 if f32 else torch.float16, device=cuda_dev)
    ws = pkv.make_cross_workspace(c.pool, 1, hq, table.shape[1], 1)
    scale = float(np.float32(d ** -0.5))
    table, cu = dev(table, cuda_dev), dev(np.array([0, 1], np.int32), cuda_dev)
    t = np.arange(8 * 256)
    k, v = (x[0][c.bt[0][t // 256], t % 256] for x in (c.k_host, c.v_host))
    want, tol = attention64(q, k, v, scale, False, 2.0 ** -21 if f32 else F16, F32 if f32 else F16)
    # sums over `tokens` terms, not over the eight pages': a warp adds its stages' products to its part in
    # order (at most 2^9 of them here, each step off by 2^-23 of the sum), then 2^8 parts at most
    tol = tol + np.abs(v.astype(np.float64)).mean() * 2 * (2.0 ** 9 + 2.0 ** 8) * 2.0 ** -23
    for _ in range(2):
        pkv.pf_paged_cross_attention(c.pool, 0, dev(q, cuda_dev), table, lens, cu, 1, scale, out, ws)
        assert pkv.pf_device_status(reset=True) == 0
        assert_within(host(out), want, tol)


@pytest.mark.parametrize("lens,new,ws", [([3000, 700], [2, 1], True), ([300, 64], [140, 130], False)])
def test_captured_and_replayed(pkv, cuda_dev, lens, new, ws):
    """Two captured calls that share a workspace, replayed in turn on new inputs."""
    import torch
    c = PagedCase(pkv, cuda_dev, lens, 4, 2, 64, 16)
    offs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    cu = dev(offs, cuda_dev)
    work = pkv.make_cross_workspace(c.pool, 2, 4, c.bt.shape[1], max(new)) if ws else None
    q = torch.zeros((int(offs[-1]), 4, 64), dtype=torch.float16, device=cuda_dev)
    outs = [torch.empty_like(q) for _ in range(2)]
    call = lambda o: pkv.pf_paged_cross_attention(c.pool, 0, q, c.bt_dev, c.lens_dev, cu, max(new), 0.125, o, work)   # noqa: E731
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(outs[0])
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, o in zip(graphs, outs):
        with torch.cuda.graph(g):
            call(o)
    rng = np.random.default_rng(2)
    rows = [[x[0][c.bt[s][np.arange(L) // 16], np.arange(L) % 16] for x in (c.k_host, c.v_host)] for s, L in enumerate(lens)]
    for i in range(4):
        qn = rng.standard_normal(tuple(q.shape)).astype(np.float16)
        q.copy_(dev(qn, cuda_dev))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        got = [attention64(qn[offs[s]:offs[s + 1]], *rows[s], 0.125, False, F16, F16) for s in range(2)]
        assert_within(host(outs[i % 2]), np.concatenate([o for o, _ in got]), np.concatenate([t for _, t in got]))
