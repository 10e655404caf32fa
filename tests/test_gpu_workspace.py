"""One workspace under calls of every kind: the kernels share its layout, a
front of 33,280 bytes (reserved bytes, then from byte 512 the few-rows
kernel's flags) and records behind it; and under calls of fewer tokens than it
was made for."""
import numpy as np
import pytest

from e4m3_util import assert_within, attention64
from gpu_util import PagedCase, dev, host
from test_gpu_e4m3 import F16, F32, Case, wide_table

pytestmark = pytest.mark.gpu

FLAGS = slice(512, 33280)


def test_flags_hold_nothing_but_flags(pkv, cuda_dev):
    """A flag is a word equal to its launch's stamp, so no call may leave anything else there: calls of
    both pool types, of 1, 3, 12 and 40 rows, fp16 and fp32 results, balanced and in fixed chunks, in
    turn on one workspace.  Each gives its result and leaves every flag word zero."""
    import torch
    c = Case(pkv, cuda_dev, [3000, 700], 4, 4, 64, 16)
    c.fill()
    f = PagedCase(pkv, cuda_dev, [3000, 700], 4, 4, 64, 16)
    table, lens = dev(wide_table(c), cuda_dev), dev(c.lens, cuda_dev)
    sizes = [f.pkv.pf_decode_workspace_bytes(f.pool, 2, 4, f.bt.shape[1], split) for split in (0, 64)]
    sizes += [pkv.pf_prefill_workspace_bytes(c.pool, 2, 4, table.shape[1], n) for n in (1, 3, 12, 40)]
    sizes += [pkv.pf_cross_workspace_bytes(f.pool, 2, 4, f.bt.shape[1], n) for n in (1, 12, 40)]
    ws = torch.zeros(max(sizes), dtype=torch.uint8, device=cuda_dev)
    pkv.pf_decode_workspace_init(ws)
    kv = [[x[0][f.bt[s][np.arange(L) // 16], np.arange(L) % 16] for x in (f.k_host, f.v_host)]
          for s, L in enumerate(f.lens)]

    def e4m3(n, dtype):
        offs = np.array([0, n, 2 * n], np.int32)
        q = c.rng.standard_normal((2 * n, 4, 64)).astype(np.float16)
        out = torch.empty((2 * n, 4, 64), dtype=dtype, device=cuda_dev)
        pkv.pf_paged_prefill_attention(c.pool, 1, dev(q, cuda_dev), table, lens, dev(offs, cuda_dev), n, c.scale(), out, ws)
        want, tol = c.want(q, offs, True, F16, F16)
        assert_within(host(out), want, tol + c.small_terms(q, offs), f"e4m3 {n}")

    def cross(n, dtype):
        offs = np.array([0, n, 2 * n], np.int32)
        q = c.rng.standard_normal((2 * n, 4, 64)).astype(np.float16)
        out = torch.empty((2 * n, 4, 64), dtype=dtype, device=cuda_dev)
        pkv.pf_paged_cross_attention(f.pool, 0, dev(q, cuda_dev), f.bt_dev, f.lens_dev, dev(offs, cuda_dev), n, 0.125, out, ws)
        got = [attention64(q[offs[s]:offs[s + 1]], *kv[s], 0.125, False, F16, F16) for s in range(2)]
        assert_within(host(out), np.concatenate([o for o, _ in got]), np.concatenate([t for _, t in got]), f"cross {n}")

    def decode(split, dtype):
        got = [attention64(f.q[s:s + 1], *kv[s], 0.125, False, F16, F16) for s in range(2)]
        # (the fp16 pools' kernel sums the rounded weights: as far off again at most)
        assert_within(host(f.attention(0.125, split=split, out_dtype=dtype, ws=ws)), np.concatenate([o for o, _ in got]),
                      2 * np.concatenate([t for _, t in got]), f"decode {split}")

    calls = [lambda t, n=n: e4m3(n, t) for n in (1, 3, 12, 40)] + [lambda t, n=n: cross(n, t) for n in (1, 12, 40)]
    calls += [lambda t, s=s: decode(s, t) for s in (0, 64)]
    for dtype in (torch.float16, torch.float32):
        for i in np.random.default_rng(3).permutation(np.repeat(np.arange(len(calls)), 2)):
            calls[i](dtype)
            assert not host(ws[FLAGS]).any(), f"call {i}"
    assert pkv.pf_device_status(reset=True) == 0


@pytest.mark.parametrize("made_for", [9, 12, 16, 40])
@pytest.mark.parametrize("h,d", [(12, 64), (4, 128)])
@pytest.mark.parametrize("kind", ["e4m3", "f16", "cross"])
def test_workspace_made_for_more_tokens(pkv, cuda_dev, made_for, h, d, kind):
    """A program sizes its workspace for the most tokens of a step; steps of fewer use the same."""
    import torch
    lens = [900, 60]
    scale = float(np.float32(d ** -0.5))
    if kind == "e4m3":
        c = Case(pkv, cuda_dev, lens, h, h, d, 16)
        c.fill()
        pool, layer, table = c.pool, 1, dev(wide_table(c), cuda_dev)
    else:
        c = PagedCase(pkv, cuda_dev, lens, h, h, d, 16)
        pool, layer, table = c.pool, 0, c.bt_dev
    make = pkv.make_cross_workspace if kind == "cross" else pkv.make_prefill_workspace
    call = pkv.pf_paged_cross_attention if kind == "cross" else pkv.pf_paged_prefill_attention
    ws = make(pool, 2, h, table.shape[1], made_for)
    for n in (1, 4, 7, 8, 9, 12, 16, 40):
        if n > made_for:
            break
        offs = np.array([0, n, 2 * n], np.int32)
        q = np.random.default_rng(n).standard_normal((2 * n, h, d)).astype(np.float16)
        for dtype in (torch.float16, torch.float32):
            out = torch.empty((2 * n, h, d), dtype=dtype, device=cuda_dev)
            call(pool, layer, dev(q, cuda_dev), table, dev(np.array(lens, np.int32), cuda_dev), dev(offs, cuda_dev), n,
                 scale, out, ws)
            if kind == "e4m3":
                want, tol = c.want(q, offs, True, F16, F16)
                tol = tol + c.small_terms(q, offs)
            else:
                got = []
                for s, L in enumerate(lens):
                    rows = [x[0][c.bt[s][np.arange(L) // 16], np.arange(L) % 16] for x in (c.k_host, c.v_host)]
                    got.append(attention64(q[offs[s]:offs[s + 1]], *rows, scale, kind != "cross", F16, F16))
                # (the fp16 pools' kernels may sum the rounded weights: as far off again at most)
                want, tol = np.concatenate([o for o, _ in got]), 2 * np.concatenate([t for _, t in got])
            assert_within(host(out), want, tol, f"{n} tokens")
    assert pkv.pf_device_status(reset=True) == 0


@pytest.mark.parametrize("kind", ["decode", "step", "cross"])
def test_more_sequences_than_a_launch_takes(pkv, cuda_dev, kind):
    """2,500 sequences, some of them empty: consecutive launches over one workspace."""
    import torch
    rng = np.random.default_rng(12)
    lens = rng.integers(0, 40, 2500).astype(np.int32)
    c = Case(pkv, cuda_dev, lens, 4, 2, 64, 16)
    n = len(lens)
    if kind == "step":
        c.append(np.maximum(lens - 1, 0))
    else:
        c.fill()
    q = rng.standard_normal((n, 4, 64)).astype(np.float16)
    out = torch.full((n + 1, 4, 64), 7.0, dtype=torch.float32, device=cuda_dev)
    ws = pkv.make_workspace(c.pool, n, 4, c.table.shape[1], 0)
    args = (c.table_dev, dev(c.lens, cuda_dev))
    pkv.pf_device_status(reset=True)
    for _ in range(2):
        if kind == "decode":
            pkv.pf_paged_decode_attention(c.pool, 1, dev(q, cuda_dev), *args, c.scale(), out[:-1], 0, ws)
        elif kind == "cross":
            pkv.pf_paged_cross_attention(c.pool, 1, dev(q, cuda_dev), *args, dev(np.arange(n + 1, dtype=np.int32), cuda_dev),
                                         1, c.scale(), out[:-1], ws)
        elif c.at.sum() < lens.sum():
            k, v = c.rows(n), c.rows(n)
            pkv.pf_decode_step(c.pool, 1, dev(q, cuda_dev), dev(k, cuda_dev), dev(v, cuda_dev), *args, c.scale(),
                               out[:-1], 0, ws)
            one = np.concatenate([[0], np.cumsum(lens > 0)])     # an empty context takes no row
            c.km.append(k[lens > 0], c.table, c.lens, one)
            c.vm.append(v[lens > 0], c.table, c.lens, one)
            c.at = c.lens.copy()
            c.check_pool()
        want, tol = c.want(q, np.arange(n + 1), False, 2.0 ** -21, F32)
        assert_within(host(out)[:-1], want, tol)
    assert bool((out[-1] == 7.0).all())
    assert pkv.pf_device_status(reset=True) == 0
