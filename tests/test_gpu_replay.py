"""Captured calls, replayed: nothing that one replay leaves in the workspace may
count as the next one's."""
import numpy as np
import pytest

from e4m3_util import assert_within, attention64
from gpu_util import PagedCase, dev, host
from test_gpu_e4m3 import F16, Case, wide_table

pytestmark = pytest.mark.gpu

RECORDS = 33280   # first byte behind the workspace's front


def captured(call):
    import torch
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    return g


def want(c, q, lens, offs=None, causal=False):
    offs = np.arange(len(lens) + 1) if offs is None else offs
    got = []
    for s, L in enumerate(lens):
        rows = [x[0][c.bt[s][np.arange(L) // c.B], np.arange(L) % c.B] for x in (c.k_host, c.v_host)]
        got.append(attention64(q[offs[s]:offs[s + 1]], *rows, 0.125, causal, F16, F16))
    # (this kernel sums the rounded weights, which is as far off again at most)
    return np.concatenate([o for o, _ in got]), 2 * np.concatenate([t for _, t in got])


@pytest.mark.parametrize("split", [64, 16])
def test_chunks_of_an_earlier_replay_are_not_merged_again(pkv, cuda_dev, split):
    """A context of many chunks in one replay, of a single one in the next: its merge of the first replay
    must not run again over the result."""
    import torch
    c = PagedCase(pkv, cuda_dev, [1000, 400, 70], 4, 4, 64, 16)
    ws = pkv.make_workspace(c.pool, 3, 4, c.bt.shape[1], split)
    q, lens = torch.zeros_like(c.q_dev), c.lens_dev.clone()
    out = torch.empty_like(q)
    g = captured(lambda: pkv.pf_paged_decode_attention(c.pool, 0, q, c.bt_dev, lens, 0.125, out, split, ws))
    rng = np.random.default_rng(1)
    for now in ([1000, 400, 70], [10, 0, 16], [1000, 5, 1], [64, 400, 2]):
        qn = rng.standard_normal(tuple(q.shape)).astype(np.float16)
        q.copy_(dev(qn, cuda_dev))
        lens.copy_(dev(np.array(now, np.int32), cuda_dev))
        g.replay()
        torch.cuda.synchronize()
        assert_within(host(out), *want(c, qn, now), f"{now}")


@pytest.mark.parametrize("call", ["decode", "cuda_cores", "step", "append"])
def test_parts_of_an_earlier_replay_are_not_taken_for_this_one_s(pkv, cuda_dev, call):
    """Parts of a cut context count when each of their 64-bit words carries the launch's stamp (the upper
    half).  Two replays of one graph have to stamp differently: with one stamp a merge may find the
    words of the replay before, and not wait for its own."""
    import torch
    lens = [3000, 700, 31]
    c = PagedCase(pkv, cuda_dev, lens, 4, 4, 64, 16)
    n = 2 if call == "append" else 1
    offs = np.arange(4, dtype=np.int32) * n
    q = torch.zeros((3 * n, 4, 64), dtype=torch.float16, device=cuda_dev)
    out = torch.empty_like(q)
    if call == "append":
        ws = pkv.make_prefill_workspace(c.pool, 3, 4, c.bt.shape[1], n)
        cu = dev(offs, cuda_dev)
        run = lambda: pkv.pf_paged_prefill_attention(c.pool, 0, q, c.bt_dev, c.lens_dev, cu, n, 0.125, out, ws)   # noqa: E731
    else:
        split = -2 if call == "cuda_cores" else 0
        ws = pkv.make_workspace(c.pool, 3, 4, c.bt.shape[1], split)
        if call == "step":   # the newest rows once more
            new = [dev(np.stack([x[0][c.bt[s][(L - 1) // 16], (L - 1) % 16] for s, L in enumerate(lens)]), cuda_dev)
                   for x in (c.k_host, c.v_host)]
            run = lambda: pkv.pf_decode_step(c.pool, 0, q, *new, c.bt_dev, c.lens_dev, 0.125, out, split, ws,   # noqa: E731
                                             flags=pkv.PF_STEP_OVERLAP_PREVIOUS)
        else:
            run = lambda: pkv.pf_paged_decode_attention(c.pool, 0, q, c.bt_dev, c.lens_dev, 0.125, out, split, ws)   # noqa: E731
    g = captured(run)
    rng = np.random.default_rng(1)
    before = None
    for i in range(4):
        qn = rng.standard_normal(tuple(q.shape)).astype(np.float16)
        q.copy_(dev(qn, cuda_dev))
        g.replay()
        torch.cuda.synchronize()
        assert_within(host(out), *want(c, qn, lens, offs, call == "append"), f"replay {i}")
        words = host(ws[RECORDS:].view(torch.int64))
        stamps = (words >> 32) & 0xffffffff
        assert np.count_nonzero(words) > 64
        if before is not None:
            again = (words != 0) & (stamps == before)
            assert not again.any(), f"replay {i}: {again.sum()} words have the stamp of the replay before"
        before = stamps
        if i == 1:
            run()            # a plain call in between
            torch.cuda.synchronize()
            before = (host(ws[RECORDS:].view(torch.int64)) >> 32) & 0xffffffff


def test_two_graphs_and_plain_calls_share_a_workspace(pkv, cuda_dev):
    import torch
    lens = [2500, 900]
    c = PagedCase(pkv, cuda_dev, lens, 8, 4, 64, 16)
    ws = pkv.make_workspace(c.pool, 2, 8, c.bt.shape[1], 0)
    q = torch.zeros_like(c.q_dev)
    outs = [torch.empty_like(q) for _ in range(3)]
    call = lambda o: pkv.pf_paged_decode_attention(c.pool, 0, q, c.bt_dev, c.lens_dev, 0.125, o, 0, ws)   # noqa: E731
    graphs = [captured(lambda o=o: call(o)) for o in outs[:2]]
    rng = np.random.default_rng(4)
    for i in range(6):
        qn = rng.standard_normal(tuple(q.shape)).astype(np.float16)
        q.copy_(dev(qn, cuda_dev))
        o = outs[i % 3]
        if i % 3 < 2:
            graphs[i % 3].replay()
        else:
            call(o)
        torch.cuda.synchronize()
        assert_within(host(o), *want(c, qn, lens), f"call {i}")


@pytest.mark.parametrize("call", ["decode", "step", "cross"])
def test_few_rows_replays_count_themselves(pkv, cuda_dev, call):
    """The few-rows kernel's flags carry the launch's stamp.  A replay takes its own from the count of
    launches at byte 256 of the workspace, 2^16 for each: with one stamp for all replays, a flag set
    after the wait for it had run out would pass for the next replay's."""
    import torch
    lens = [3000, 700, 31]
    c = Case(pkv, cuda_dev, lens, 4, 4, 64, 16)
    c.fill()
    table, lens_dev = dev(wide_table(c), cuda_dev), dev(c.lens, cuda_dev)
    q = torch.zeros((3, 4, 64), dtype=torch.float16, device=cuda_dev)
    out = torch.empty_like(q)
    ws = pkv.make_workspace(c.pool, 3, 4, table.shape[1], 0)
    cu = dev(np.arange(4, dtype=np.int32), cuda_dev)
    last = [dev(np.stack([m.rows(c.table[s], L)[-1] for s, L in enumerate(lens)]).astype(np.float16), cuda_dev)
            for m in (c.km, c.vm)]            # the newest rows once more: their codes stay
    run = {"decode": lambda: pkv.pf_paged_decode_attention(c.pool, 1, q, table, lens_dev, c.scale(), out, 0, ws),
           "step": lambda: pkv.pf_decode_step(c.pool, 1, q, *last, table, lens_dev, c.scale(), out, 0, ws),
           "cross": lambda: pkv.pf_paged_cross_attention(c.pool, 1, q, table, lens_dev, cu, 1, c.scale(), out, ws)}[call]
    g = captured(run)
    count = lambda: int(host(ws[256:264].view(torch.int64))[0])   # noqa: E731
    offs = np.arange(4)
    for i in range(4):
        qn = c.rng.standard_normal((3, 4, 64)).astype(np.float16)
        q.copy_(dev(qn, cuda_dev))
        assert count() == i << 16
        g.replay()
        torch.cuda.synchronize()
        want, tol = c.want(qn, offs, False, F16, F16)
        assert_within(host(out), want, tol + c.small_terms(qn, offs), f"replay {i}")
        run()                                 # a plain call takes the host's stamp
        torch.cuda.synchronize()
        assert_within(host(out), want, tol + c.small_terms(qn, offs), f"after replay {i}")
        assert count() == (i + 1) << 16
    assert not host(ws[512:33280]).any()
    assert pkv.pf_device_status(reset=True) == 0
