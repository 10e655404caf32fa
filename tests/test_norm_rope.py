"""The rotated cache write without a GPU: what it refuses before anything is
launched (made-up device addresses), and its table of angles."""
import ctypes
import math
from types import SimpleNamespace

import numpy as np
import pytest

P = ctypes.c_void_p
OK, ODD = P(0x30000), P(0x30008)


def make(lib, e4m3=False):
    h = P()
    if e4m3:
        assert lib.pf_pool_create_e4m3(ctypes.byref(h), P(0x10000), P(0x20000), P(0x40000), P(0x50000), 1, 64, 16, 2, 64) == 0
    else:
        assert lib.pf_pool_create(ctypes.byref(h), P(0x10000), P(0x20000), 1, 64, 16, 2, 64, 1) == 0
    return h


GOOD = dict(layer=0, q=OK, qs=512, k=OK, ks=512, v=OK, vs=512, n=3, hq=4, qw=OK, kw=OK, eps=1e-6, angles=OK, positions=9,
            rot=64, flags=0, rope_pos=None, table=OK, rows=4, width=7, seq=OK, pos=OK, q_out=OK, qos=256, k_out=None, kos=0)


def call(lib, pool, **kw):
    a = {**GOOD, **kw}
    return lib.pf_norm_rope_write(pool, a["layer"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["n"], a["hq"],
                                  a["qw"], a["kw"], ctypes.c_float(a["eps"]), a["angles"], a["positions"], a["rot"],
                                  a["flags"], a["rope_pos"], a["table"], a["rows"], a["width"], a["seq"], a["pos"],
                                  a["q_out"], a["qos"], a["k_out"], a["kos"], None)


@pytest.mark.parametrize("kw,word", [
    (dict(layer=1), "layer"), (dict(layer=-1), "layer"), (dict(n=-1), "n_tokens"), (dict(flags=2), "flags"),
    (dict(q=None, k=None), "neither"), (dict(hq=0), "n_q_heads"), (dict(hq=-4), "n_q_heads"), (dict(hq=1 << 20), "n_q_heads"),
    (dict(q_out=None), "q_out"), (dict(q=None), "without q"), (dict(q=None, hq=0), "without q"),
    (dict(q=None, hq=0, q_out=None), "without q"), (dict(k=None), "without k"), (dict(k=None, table=None, k_out=OK), "without k"),
    (dict(k=None, table=None), "without k"), (dict(table=None), "k_out"), (dict(v=None), "v, seq_idx"),
    (dict(seq=None), "v, seq_idx"), (dict(pos=None), "v, seq_idx"), (dict(rows=0), "n_table_rows"), (dict(width=0), "n_table_rows"),
    (dict(q=ODD), "aligned"), (dict(k=ODD), "aligned"), (dict(v=ODD), "aligned"), (dict(q_out=ODD), "aligned"),
    (dict(k_out=ODD, kos=128), "aligned"), (dict(qw=ODD), "aligned"), (dict(kw=ODD), "aligned"), (dict(angles=ODD), "aligned"),
    (dict(qs=4), "strides"), (dict(ks=-8), "strides"), (dict(vs=1 << 41), "strides"), (dict(qos=248), "overlap"),
    (dict(qos=0), "overlap"), (dict(k_out=OK, kos=120), "overlap"), (dict(eps=-1.0), "eps"), (dict(eps=math.nan), "eps"),
    (dict(eps=math.inf), "eps"), (dict(rot=-16), "rot_dim"), (dict(rot=80), "rot_dim"), (dict(angles=None), "angles"),
    (dict(positions=0), "angles"), (dict(table=None, k_out=OK, kos=128, pos=None), "rope_pos"),
])
def test_refusals(pkv, kw, word):
    lib = pkv.lib()
    pool = make(lib)
    assert call(lib, pool, **kw) == pkv.PF_ERR_INVALID
    assert word in pkv.pf_last_error() and "pf_norm_rope_write" in pkv.pf_last_error(), pkv.pf_last_error()
    lib.pf_pool_destroy(pool)


def test_not_built(pkv):
    lib = pkv.lib()
    pool, pool8 = make(lib), make(lib, True)
    for rot in (8, 24, 63):
        assert call(lib, pool, rot=rot) == pkv.PF_ERR_UNSUPPORTED and "multiple of 16" in pkv.pf_last_error()
    assert call(lib, pool8) == pkv.PF_ERR_UNSUPPORTED and "pf_append_kv" in pkv.pf_last_error()
    assert call(lib, None) == pkv.PF_ERR_INVALID
    for p in (pool, pool8):
        assert call(lib, p, n=0, q=None, k=None) == pkv.PF_OK     # nothing to do
        lib.pf_pool_destroy(p)


def test_binding_refuses_shapes(pkv, monkeypatch):
    import torch
    # (a host tensor's device is -1: as if that were the current one, every shape is looked at)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    pool = SimpleNamespace(handle=None, n_layers=1, n_blocks=8, block_size=16, n_kv_heads=2, head_dim=64, k_scale=None,
                           device=-1)
    q, k = torch.zeros((3, 4, 64), dtype=torch.float16), torch.zeros((3, 2, 64), dtype=torch.float16)
    i3, table, ang = torch.zeros(3, dtype=torch.int32), torch.zeros((2, 2), dtype=torch.int32), torch.zeros((9, 64))
    good = dict(q=q, k=k, v=k, block_tables=table, seq_idx=i3, pos=i3, angles=ang, q_out=q.clone())
    for kw, word in ((dict(q=None, k=None), "neither"), (dict(k=k[:2]), "rows"), (dict(v=k[:2]), "rows"),
                     (dict(q_out=None), "q_out"), (dict(q=None), "q_out"), (dict(q=q[0], k=None, v=None, q_out=q), "n_tokens"),
                     (dict(v=k[0]), "rows"), (dict(q_out=q[:2]), "rows"), (dict(q=q.float()), "float16"),
                     (dict(k=k.transpose(0, 1).contiguous().transpose(0, 1)), "contiguous"), (dict(k_out=q), "rows"),
                     (dict(pos=i3.long()), "int32"),
                     (dict(seq_idx=i3[:2]), "seq_idx"), (dict(pos=i3[:2]), "pos"), (dict(rope_pos=i3[:2]), "rope_pos"),
                     (dict(block_tables=i3), "block_tables"), (dict(angles=ang[0]), "angles"),
                     (dict(q_weight=ang[0, :32]), "q_weight"), (dict(k_weight=ang), "k_weight"),
                     (dict(q=q[..., :32]), "64"), (dict(), "pool is null")):
        with pytest.raises(pkv.PagedKVError, match=word):
            pkv.pf_norm_rope_write(pool, 0, **{**good, **kw})
    pool.device = 1
    with pytest.raises(pkv.PagedKVError, match="current device"):
        pkv.pf_norm_rope_write(pool, 0, **good)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(pkv.PagedKVError, match="CUDA"):
        pkv.pf_norm_rope_write(pool, 0, **good)


@pytest.mark.parametrize("rot,theta", [(64, 10000.0), (16, 500000.0), (128, 10000.0)])
def test_angles(pkv, rot, theta):
    """Against powers by repeated multiplication in numpy's longer type, to fp32's rounding."""
    n = 70000
    got = pkv.make_rope_angles(n, rot, theta, device="cpu").numpy()
    assert got.shape == (n, rot) and got.dtype == np.float32
    p = np.array([0, 1, 2, 1000, 65535, n - 1])
    step = np.longdouble(theta) ** (np.longdouble(-2) / rot)
    f = np.ones(rot // 2, np.longdouble)
    for j in range(1, rot // 2):
        f[j] = f[j - 1] * step
    a = p[:, None] * f
    want = np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float64)
    # an angle below 2^17 in 64 bits is off by a few 2^-36, then one rounding of a value of at most 1
    assert np.abs(got[p].astype(np.float64) - want).max() <= 2.0 ** -25 + 2.0 ** -33
