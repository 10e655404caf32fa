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


def host_is_current(monkeypatch):
    """A host tensor's device is -1: as if that were the current one, every argument is looked at."""
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)


@pytest.mark.parametrize("make", [lambda t: t.tolist(), lambda t: t.numpy(), lambda t: 3])
def test_what_is_no_tensor_is_a_type_error(pkv, pool, monkeypatch, make):
    """By the argument's name, in whatever place."""
    import torch
    host_is_current(monkeypatch)
    pool.device = -1
    q, k = torch.zeros((3, 4, 128), dtype=torch.float16), torch.zeros((3, 2, 128), dtype=torch.float16)
    i3, table, w = torch.zeros(3, dtype=torch.int32), torch.zeros((3, 2), dtype=torch.int32), torch.zeros(128)
    rope = dict(q=q, k=k, v=k, block_tables=table, seq_idx=i3, pos=i3, angles=torch.zeros((9, 128)), q_out=q.clone(),
                k_out=k.clone(), q_weight=w, k_weight=w, rope_pos=i3)
    common = dict(q=q, block_tables=table, context_lens=i3, cu_q=torch.arange(4, dtype=torch.int32), out=q.clone(),
                  workspace=torch.zeros(1024, dtype=torch.uint8))
    bits = torch.zeros((3, 1), dtype=torch.int64)
    for call, args in (
            (lambda **a: pkv.pf_norm_rope_write(pool, 0, **a), rope),
            (lambda **a: pkv.pf_paged_window_attention(pool, 0, max_new_tokens=2, scale=0.1, window=5, n_sinks=1, **a), common),
            (lambda **a: pkv.pf_paged_tree_attention(pool, 0, max_draft_tokens=2, scale=0.1, **a), dict(common, tree=bits))):
        for name, t in args.items():
            with pytest.raises(TypeError, match=f"^{name} must be a torch tensor$"):
                call(**{**args, name: make(t)})
        with pytest.raises(pkv.PagedKVError, match="pool is null"):
            call(**args)
