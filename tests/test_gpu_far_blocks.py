"""Blocks whose bytes lie past 2^32 from the pool's base: every call over them
gives what it gives over the same blocks of a small pool, bit for bit."""
import numpy as np
import pytest

from gpu_util import dev, host

pytestmark = pytest.mark.gpu

B, H, D, HQ, NEAR = 256, 8, 128, 16, 12


def pools(pkv, device, dtype, n_blocks):
    import torch
    k, v = (torch.empty((1, n_blocks, B, H, D), dtype=dtype, device=device) for _ in range(2))
    assert n_blocks == NEAR or k.numel() * k.element_size() > 2 ** 32 + NEAR * B * H * D * 2
    if dtype == torch.float16:
        return pkv.pf_pool_create(k, v)
    return pkv.pf_pool_create(k, v, *(torch.empty((1, n_blocks, H), device=device) for _ in range(2)))


@pytest.mark.parametrize("cache", ["e4m3", "f16"])
def test_far_blocks(pkv, cuda_dev, cache):
    import torch
    dtype = torch.float8_e4m3fn if cache == "e4m3" else torch.float16
    far = 17000 if cache == "e4m3" else 8600
    rng = np.random.default_rng(8)
    lens = np.array([700, 300, 0, 257], np.int32)
    table = np.full((4, 3), 1 << 30, np.int32)
    order = rng.permutation(NEAR - 2)
    for s, i in zip((0, 1, 3), (0, 3, 5)):
        n = -(-int(lens[s]) // B)
        table[s, :n] = order[i:i + n]
    offs = np.concatenate([[0], np.cumsum(lens)])
    rows = [rng.standard_normal((int(lens.sum()), H, D)).astype(np.float16) for _ in range(2)]
    few, many = (np.array(x, np.int32) for x in ([0, 2, 3, 3, 5], [0, 130, 200, 200, 457]))
    q = rng.standard_normal((457, HQ, D)).astype(np.float16)
    got = []
    for n_blocks in (NEAR, far):
        pool = pools(pkv, cuda_dev, dtype, n_blocks)
        shift = n_blocks - NEAR
        bt = dev(np.where(table < NEAR, table + shift, table).astype(np.int32), cuda_dev)
        ln = dev(lens, cuda_dev)
        kn, vn = (dev(x, cuda_dev) for x in rows)
        if cache == "e4m3":
            pkv.pf_append_kv(pool, 0, kn, vn, bt, ln, dev(offs.astype(np.int32), cuda_dev), int(lens.max()))
        else:
            seq = np.repeat(np.arange(4), lens).astype(np.int32)
            pos = np.concatenate([np.arange(L) for L in lens]).astype(np.int32)
            pkv.pf_write_kv(pool, 0, kn, vn, bt, dev(seq, cuda_dev), dev(pos, cuda_dev))
        # the last block of sequence 3 moves to the pool's end
        src = dev(np.array([table[3, 1] + shift], np.int32), cuda_dev)
        dst = dev(np.array([n_blocks - 1], np.int32), cuda_dev)
        ident = np.arange(n_blocks, dtype=np.int32)
        ident[table[3, 1] + shift] = n_blocks - 1
        pkv.pf_compact_blocks(pool, src, dst, dev(ident, cuda_dev), bt, ln)
        outs = []
        for dt in (torch.float16, torch.float32):
            new = lambda n: torch.full((n, HQ, D), 7.0, dtype=dt, device=cuda_dev)   # noqa: E731
            qd = dev(q, cuda_dev)
            wide = torch.nn.functional.pad(bt, (0, 16), value=1 << 30)
            for t in (bt, wide):
                ws = pkv.make_workspace(pool, 4, HQ, t.shape[1], 0)
                o = new(4)
                pkv.pf_paged_decode_attention(pool, 0, qd[:4], t, ln, 0.09, o, 0, ws)
                outs.append(o)
                for cu in (few, many):
                    most, n = int(np.diff(cu).max()), int(cu[-1])
                    ws = pkv.make_prefill_workspace(pool, 4, HQ, t.shape[1], most)
                    o = new(n)
                    pkv.pf_paged_prefill_attention(pool, 0, qd[:n], t, ln, dev(cu, cuda_dev), most, 0.09, o, ws)
                    outs.append(o)
                    ws = pkv.make_cross_workspace(pool, 4, HQ, t.shape[1], most)
                    o = new(n)
                    pkv.pf_paged_cross_attention(pool, 0, qd[:n], t, ln, dev(cu, cuda_dev), most, 0.09, o, ws)
                    outs.append(o)
        back = [torch.zeros((int(lens.sum()), H, D), dtype=torch.float16, device=cuda_dev) for _ in range(2)]
        pkv.pf_gather_kv(pool, 0, bt, ln, dev(offs[:4].astype(np.int64), cuda_dev), *back)
        got.append([host(o) for o in outs + back])
        assert pkv.pf_device_status(reset=True) == 0
        del pool
        torch.cuda.empty_cache()
    for i, (a, b) in enumerate(zip(*got)):
        assert np.all(np.isfinite(a)) and np.array_equal(a, b), i
