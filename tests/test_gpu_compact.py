"""Compaction on the GPU: contents and tables move together, for both pool
types, and a serving loop goes on over the packed pool."""
import numpy as np
import pytest

from e4m3_util import assert_within, attention64
from gpu_util import dev, host
from test_gpu_e4m3 import F16

pytestmark = pytest.mark.gpu


def _bits(t):
    import torch
    return host(t.view(torch.uint8))


@pytest.mark.parametrize("cache", ["f16", "e4m3"])
@pytest.mark.parametrize("layers,page,heads,dim", [(3, 16, 12, 64), (1, 1, 1, 64), (2, 256, 5, 128), (12, 64, 2, 64)])
def test_moves_and_tables(pkv, cuda_dev, cache, layers, page, heads, dim):
    import torch
    n = 40
    rng = np.random.default_rng(3)
    shape = (layers, n, page, heads, dim)
    alloc = pkv.pf_alloc_create(n, 5)
    ids = pkv.pf_alloc_blocks(alloc, 30)
    pkv.pf_free_blocks(alloc, ids[::2].copy())
    rows = [ids[1:13:2], ids[13:29:2], ids[:0]]                 # 6, 8 and 0 pages
    lens = np.array([6 * page - page // 2, 8 * page, 0], np.int32)
    table = np.full((3, 9), 10 ** 6, np.int32)                  # entries past a context are never read
    for s, r in enumerate(rows):
        table[s, :r.size] = r
    pkv.pf_free_blocks(alloc, ids[29:30])
    raw = [torch.from_numpy(rng.integers(0, 256, (*shape, 2 if cache == "f16" else 1), dtype=np.uint8)).to(cuda_dev)
           for _ in range(2)]
    if cache == "f16":
        k, v = (x.view(torch.float16).squeeze(-1) for x in raw)
        tensors, pool = [k, v], pkv.pf_pool_create(k, v)
    else:
        k, v = (x.squeeze(-1).view(torch.float8_e4m3fn) for x in raw)
        ks, vs = (torch.rand((layers, n, heads), device=cuda_dev) for _ in range(2))
        tensors, pool = [k, v, ks, vs], pkv.pf_pool_create(k, v, ks, vs)
    was = [_bits(t).copy() for t in tensors]
    src, dst, block_map = pkv.pf_alloc_compact(alloc)
    assert src.size > 0
    t_dev = dev(table, cuda_dev)
    pkv.pf_device_status(reset=True)
    for _ in range(2):                                          # a second call finds nothing to change
        pkv.pf_compact_blocks(pool, dev(src, cuda_dev), dev(dst, cuda_dev), dev(block_map, cuda_dev), t_dev,
                              dev(lens, cuda_dev))
    assert pkv.pf_device_status(reset=True) == 0
    for t, w in zip(tensors, was):
        w[:, dst] = w[:, src]
        assert np.array_equal(_bits(t), w)
    want = table.copy()
    for s, r in enumerate(rows):
        want[s, :r.size] = block_map[r]
    assert np.array_equal(host(t_dev), want)
    assert sorted(want[want < n]) == list(range(14))


def test_bad_ids_and_map_entries(pkv, cuda_dev):
    import torch
    k = torch.randn((1, 8, 16, 2, 64), device=cuda_dev).half()
    v = torch.randn_like(k)
    pool = pkv.pf_pool_create(k, v)
    was = k.clone()
    table = dev(np.array([[1, 2, 99], [3, 0, 0]], np.int32), cuda_dev)
    lens = dev(np.array([48, -5], np.int32), cuda_dev)
    m = np.arange(8, dtype=np.int32)
    m[1], m[2] = 4, 77
    pkv.pf_device_status(reset=True)
    pkv.pf_compact_blocks(pool, dev(np.array([8, 5], np.int32), cuda_dev), dev(np.array([0, -1], np.int32), cuda_dev),
                          dev(m, cuda_dev), table, lens)
    assert pkv.pf_device_status(reset=True) == pkv.PF_DEV_BAD_BLOCK_ID | pkv.PF_DEV_BAD_LENGTH
    assert bool((k == was).all())
    assert host(table).tolist() == [[4, 2, 99], [3, 0, 0]]


def test_serving_over_an_8_bit_pool(pkv, cuda_dev):
    """Prompts, decode steps, a finished sequence, a fork with copy-on-write,
    compaction, cross attention of another head over the same cache, more
    steps: checked against a dense fp64 history of what the pool holds."""
    import torch
    B, H, Hq, D, N, W = 16, 2, 6, 64, 48, 12
    k = torch.empty((1, N, B, H, D), dtype=torch.float8_e4m3fn, device=cuda_dev)
    v = torch.empty_like(k)
    ks, vs = (torch.empty((1, N, H), device=cuda_dev) for _ in range(2))
    pool = pkv.pf_pool_create(k, v, ks, vs)
    alloc = pkv.pf_alloc_create(N, 3)
    rng = np.random.default_rng(0)
    scale = float(np.float32(D ** -0.5))
    table, lens = np.zeros((4, W), np.int32), np.zeros(4, np.int32)
    pkv.pf_device_status(reset=True)

    def held(s):
        """fp64 rows of sequence s as the pool holds them."""
        t = np.arange(lens[s])
        blk = table[s][t // B]
        return [x.float().cpu().numpy().astype(np.float64)[0][blk, t % B] * sc.cpu().numpy()[0][blk][..., None]
                for x, sc in ((k, ks), (v, vs))]

    def step(new):
        """Append `new[s]` tokens to every sequence, then attend causally."""
        new = np.asarray(new, np.int32)
        for s in range(4):
            if new[s]:
                pkv.pf_seq_reserve(alloc, B, table[s], int(lens[s]), int(lens[s] + new[s]))
                first, last = lens[s] // B, (lens[s] + new[s] - 1) // B
                for j in range(first, last + 1):
                    pair = pkv.pf_alloc_cow(alloc, table[s], j)
                    if pair:
                        pkv.pf_copy_blocks(pool, *(dev(np.array([x], np.int32), cuda_dev) for x in pair))
        lens[:] += new
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = int(cu[-1])
        kn, vn = (rng.standard_normal((T, H, D)).astype(np.float16) for _ in range(2))
        q = rng.standard_normal((T, Hq, D)).astype(np.float16)
        args = dev(table, cuda_dev), dev(lens, cuda_dev), dev(cu, cuda_dev), int(new.max())
        pkv.pf_append_kv(pool, 0, dev(kn, cuda_dev), dev(vn, cuda_dev), *args)
        out = torch.empty((T, Hq, D), dtype=torch.float16, device=cuda_dev)
        ws = pkv.make_prefill_workspace(pool, 4, Hq, W, int(new.max()))
        pkv.pf_paged_prefill_attention(pool, 0, dev(q, cuda_dev), *args, scale, out, ws)
        for s in range(4):
            hk, hv = held(s)
            # what was appended, within a half step of e4m3 (and the smallest code's half)
            for x, h in ((kn, hk), (vn, hv)):
                if new[s]:
                    a = x[cu[s]:cu[s + 1]].astype(np.float64)
                    amax = np.abs(a).max()
                    assert np.all(np.abs(h[lens[s] - new[s]:] - a) <= np.abs(a) * 2.0 ** -4 + amax * 2.0 ** -16)
            want, tol = attention64(q[cu[s]:cu[s + 1]], hk, hv, scale, True, F16, F16)
            assert_within(host(out)[cu[s]:cu[s + 1]], want, tol + 2.0 ** -20, f"sequence {s}")

    step([40, 100, 7, 0])
    step([1, 1, 1, 0])
    pkv.pf_seq_release(alloc, B, table[1], int(lens[1]))
    table[1], lens[1] = 0, 0
    pkv.pf_seq_fork(alloc, B, table[0], int(lens[0]), table[3])
    lens[3] = lens[0]
    step([1, 0, 1, 1])
    src, dst, block_map = pkv.pf_alloc_compact(alloc)
    t_dev = dev(table, cuda_dev)
    before = [held(s) for s in range(4)]
    pkv.pf_compact_blocks(pool, dev(src, cuda_dev), dev(dst, cuda_dev), dev(block_map, cuda_dev), t_dev, dev(lens, cuda_dev))
    used = np.arange(W)[None, :] * B < lens[:, None]
    table = np.where(used, block_map[table], table)
    assert np.array_equal(host(t_dev), table)
    assert table[used].max() == N - pkv.pf_alloc_free_count(alloc) - 1
    for s in range(4):
        for a, b in zip(before[s], held(s)):
            assert np.array_equal(a, b)
    q = rng.standard_normal((8, Hq, D)).astype(np.float16)
    cu = np.array([0, 2, 4, 6, 8], np.int32)
    out = torch.empty((8, Hq, D), dtype=torch.float16, device=cuda_dev)
    pkv.pf_paged_cross_attention(pool, 0, dev(q, cuda_dev), t_dev, dev(lens, cuda_dev), dev(cu, cuda_dev), 2, scale, out,
                                 pkv.make_cross_workspace(pool, 4, Hq, W, 2))
    for s in range(4):
        want, tol = attention64(q[cu[s]:cu[s + 1]], *held(s), scale, False, F16, F16)
        assert_within(host(out)[cu[s]:cu[s + 1]], want, tol + 2.0 ** -20)
    step([1, 30, 1, 1])
    step([20, 1, 0, 3])
    assert pkv.pf_device_status(reset=True) == 0
