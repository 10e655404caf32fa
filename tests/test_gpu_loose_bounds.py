"""max_new_tokens is an upper bound: a loose one, up to the type's largest,
changes nothing but the launch."""
import numpy as np
import pytest

from e4m3_util import assert_within, attention64
from gpu_util import PagedCase, dev, host
from test_gpu_e4m3 import F16, Case

pytestmark = pytest.mark.gpu

INT_MAX = 2 ** 31 - 1


@pytest.mark.parametrize("page,h,d", [(16, 2, 64), (1, 1, 128), (256, 1, 64)])
@pytest.mark.parametrize("bound", [1 << 20, INT_MAX])
def test_append(pkv, cuda_dev, page, h, d, bound):
    """Pages far past the context are not touched, whatever the bound."""
    c = Case(pkv, cuda_dev, [300, 17, 0, 256], h, h, d, page)
    pkv.pf_device_status(reset=True)
    for new in ([200, 17, 0, 255], [100, 0, 0, 1]):
        new = np.array(new, np.int32)
        c.at = c.at + new
        offs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        k, v = c.rows(int(offs[-1])), c.rows(int(offs[-1]))
        pkv.pf_append_kv(c.pool, 1, dev(k, cuda_dev), dev(v, cuda_dev), c.table_dev, dev(c.at, cuda_dev),
                         dev(offs, cuda_dev), bound)
        c.km.append(k, c.table, c.at, offs)
        c.vm.append(v, c.table, c.at, offs)
        c.check_pool()
    assert pkv.pf_device_status(reset=True) == 0


@pytest.mark.parametrize("lens,new", [([300, 17, 40], [200, 17, 3]), ([5, 1, 0], [2, 1, 0])])
@pytest.mark.parametrize("cache", ["f16", "e4m3"])
@pytest.mark.parametrize("ws", [False, True])
def test_causal_attention(pkv, cuda_dev, lens, new, cache, ws):
    """The largest bound, 2 q-heads per kv-head: the rows that it allows do not fit 32 bits, those of the table do."""
    import torch
    offs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(offs[-1])
    q = np.random.default_rng(2).standard_normal((T, 4, 64)).astype(np.float16)
    if cache == "f16":
        c = PagedCase(pkv, cuda_dev, lens, 4, 2, 64, 16)
        pool, layer, table = c.pool, 0, c.bt_dev
        got = []
        for s, L in enumerate(lens):
            rows = [x[0][c.bt[s][np.arange(L) // 16], np.arange(L) % 16] for x in (c.k_host, c.v_host)]
            got.append(attention64(q[offs[s]:offs[s + 1]], *rows, 0.125, True, F16, F16))
        # (the kernel of few rows sums the rounded weights: as far off again at most)
        want, tol = np.concatenate([o for o, _ in got]), 2 * np.concatenate([t for _, t in got])
    else:
        c = Case(pkv, cuda_dev, lens, 4, 2, 64, 16)
        c.fill()
        pool, layer, table = c.pool, 1, c.table_dev
        want, tol = c.want(q, offs, True, F16, F16)
        tol = tol + c.small_terms(q, offs)
    out = torch.full((T + 1, 4, 64), 7.0, dtype=torch.float16, device=cuda_dev)
    work = torch.zeros(1 << 24, dtype=torch.uint8, device=cuda_dev) if ws else None
    pkv.pf_device_status(reset=True)
    pkv.pf_paged_prefill_attention(pool, layer, dev(q, cuda_dev), table, dev(np.array(lens, np.int32), cuda_dev),
                                   dev(offs, cuda_dev), INT_MAX, 0.125, out[:-1], work)
    assert pkv.pf_device_status(reset=True) == 0
    assert_within(host(out)[:-1], want, tol)
    assert bool((out[-1] == 7.0).all())
