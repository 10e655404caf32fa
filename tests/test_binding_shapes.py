"""Queries of another shape than the pool's rows are refused by the bindings by
that shape, before a pointer is taken (tensors of the host, no GPU)."""
from types import SimpleNamespace

import pytest


@pytest.fixture
def pool():
    return SimpleNamespace(handle=None, n_layers=1, n_blocks=8, block_size=16, n_kv_heads=2, head_dim=128, k_scale=None,
                           device=0)


@pytest.mark.parametrize("shape", [(3, 4, 64), (3, 4, 256)])
def test_decode_head_dim(pkv, pool, shape):
    """A kernel for 128 values per head must not read rows of 64."""
    import torch
    q = torch.zeros(shape, dtype=torch.float16)
    table, lens, ws = torch.zeros((3, 2), dtype=torch.int32), torch.ones(3, dtype=torch.int32), torch.zeros(1024)
    k = torch.zeros((3, 2, shape[2]), dtype=torch.float16)
    for call in (lambda: pkv.pf_paged_decode_attention(pool, 0, q, table, lens, 0.1, q.clone(), 0, ws),
                 lambda: pkv.pf_paged_decode_attention_noalloc(pool, 0, q, table, lens, 0.1, q.clone(), 0),
                 lambda: pkv.pf_decode_step(pool, 0, q, k, k, table, lens, 0.1, q.clone(), 0, ws)):
        with pytest.raises(pkv.PagedKVError, match="head_dim"):
            call()


@pytest.mark.parametrize("shape", [(6, 128), (6, 4, 64), (1, 6, 4, 128), (6, 128, 1)])
def test_tokens(pkv, pool, shape, monkeypatch):
    """[tokens, values] is no [tokens, heads, values], although its last dimension fits."""
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    q = torch.zeros(shape, dtype=torch.float16)
    table, lens = torch.zeros((3, 2), dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    cu = torch.arange(0, 8, 2, dtype=torch.int32)
    for call in (pkv.pf_paged_prefill_attention, pkv.pf_paged_cross_attention):
        with pytest.raises(pkv.PagedKVError, match="n_q_heads, head_dim|T_q"):
            call(pool, 0, q, table, lens, cu, 2, 0.1, q.clone())
