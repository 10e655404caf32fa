"""8-bit (e4m3) pools on the GPU against plain 64-bit forms: the quantising
append code for code, decode and append attention, the fused step, the gather,
block copies and swapping."""
import numpy as np
import pytest

import synth_inputs as si
from e4m3_util import TABLE, Model, assert_within, attention64
from gpu_util import dev, host

pytestmark = pytest.mark.gpu

F16, F32 = 2.0 ** -11, 2.0 ** -24


class Case:
    """An 8-bit pool of two layers (work in layer 1), its fp64 model and tables."""

    def __init__(self, pkv, device, lens, n_q_heads, heads, dim, block_size, seed=5, spare=3, width=None):
        import torch
        self.pkv, self.device, self.torch = pkv, device, torch
        self.lens = np.asarray(lens, dtype=np.int32)
        self.Hq, self.H, self.D, self.B = n_q_heads, heads, dim, block_size
        need = sum(si.pages_for(L, block_size) for L in self.lens)
        self.N = need + spare
        self.table = si.block_tables(self.lens, block_size, self.N, 7, max_blocks=width)
        shape = (2, self.N, block_size, heads, dim)
        # unwritten memory: NaN codes and wild scales
        self.k = torch.full(shape, 0x7f, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
        self.v = torch.full(shape, 0xff, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
        self.ks = torch.full((2, self.N, heads), 3.0e38, device=device)
        self.vs = torch.full((2, self.N, heads), float("nan"), device=device)
        self.pool = pkv.pf_pool_create(self.k, self.v, self.ks, self.vs)
        self.km, self.vm = Model(self.N, block_size, heads, dim), Model(self.N, block_size, heads, dim)
        self.table_dev = dev(self.table, device)
        self.rng = np.random.default_rng(seed)
        self.at = np.zeros_like(self.lens)

    def rows(self, n, spread=True):
        """fp16 rows whose size differs by token, so that scales grow on the way."""
        x = self.rng.standard_normal((n, self.H, self.D))
        if spread:
            x *= np.exp2(self.rng.integers(-6, 5, (n, 1, 1)))
        return x.astype(np.float16)

    def append(self, new, k=None, v=None, cu=True):
        """The next `new[s]` tokens of every sequence."""
        new = np.asarray(new, dtype=np.int32)
        self.at = self.at + new
        offs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        k = self.rows(int(offs[-1])) if k is None else k
        v = self.rows(int(offs[-1])) if v is None else v
        if cu:
            self.pkv.pf_append_kv(self.pool, 1, dev(k, self.device), dev(v, self.device), self.table_dev,
                                  dev(self.at, self.device), dev(offs, self.device), max(1, int(new.max())))
        else:
            rows = np.zeros((len(new), self.H, self.D), np.float16)   # row s, unused where nothing is appended
            rk, rv = rows.copy(), rows.copy()
            rk[new > 0], rv[new > 0] = k, v
            self.pkv.pf_append_kv(self.pool, 1, dev(rk, self.device), dev(rv, self.device), self.table_dev,
                                  dev(np.where(new > 0, self.at, 0).astype(np.int32), self.device), None)
        self.km.append(k, self.table, self.at, offs)
        self.vm.append(v, self.table, self.at, offs)

    def fill(self):
        """The contexts up to their lengths, in a few ragged appends."""
        left = self.lens.copy()
        first = left // 3
        self.append(first)
        self.append(np.minimum(left - first, 1))
        self.append(self.lens - self.at)

    def check_pool(self):
        """Written codes and scales equal the model's; everything else is as it was."""
        for dev_codes, dev_scales, m, fresh in ((self.k, self.ks, self.km, 0x7f), (self.v, self.vs, self.vm, 0xff)):
            codes = host(dev_codes.view(self.torch.uint8))
            written = ~np.isnan(m.code)
            assert np.array_equal(TABLE[codes[1]][written], m.code[written])
            assert np.all(codes[1][~written] == fresh)
            assert np.all(codes[0] == fresh)
            scales = host(dev_scales)
            known = ~np.isnan(m.scale)
            assert np.array_equal(scales[1][known].astype(np.float64), m.scale[known])

    def want(self, q, offs, causal, weight_step, out_step):
        outs = [attention64(q[offs[s]:offs[s + 1]], self.km.rows(self.table[s], L), self.vm.rows(self.table[s], L),
                            self.scale(), causal, weight_step, out_step) for s, L in enumerate(self.lens)]
        return np.concatenate([o for o, _ in outs]), np.concatenate([t for _, t in outs])

    def small_terms(self, q, offs):
        """What want() leaves out, on either kernel.

        Weights stored as subnormal fp16 (below 2^-14) are off by 2^-25 instead
        of 2^-11 relative.  The prompt kernel stores w / w_max times at least 1,
        so that moves the mean by at most 2^-25 |v| for each token, sum w / w_max
        being at least 1.  The few-rows kernel stores 2^7 w / w_max times a V
        scale over the largest V scale S met, and takes it times code * S: at most
        2^-32 |code| S for each token.
        The prompt kernel's dequantised values may be off by 2^-25 where they are
        below 2^-14: V's move the mean by as much, K's a score by at most
        e = 2^-25 * scale * sum |q|, and the mean by 2 e times the largest |v|."""
        out = []
        for s, L in enumerate(self.lens):
            t = np.arange(L)
            blk = self.table[s][t // self.B]
            code = np.abs(self.vm.code[blk, t % self.B])                                 # [L, H, D]
            v = code * self.vm.scale[blk][:, :, None]
            top = self.vm.scale[blk].max(0)[:, None] if L else 0.0                      # [H, 1]
            x = np.maximum(2.0 ** -32 * code.sum(0) * top, 2.0 ** -25 * v.sum(0)) + 2.0 ** -25
            big = v.max(0) if L else x
            e = 2.0 ** -25 * self.scale() * np.abs(q[offs[s]:offs[s + 1]].astype(np.float64)).sum(-1)
            wide = lambda y: np.repeat(y, self.Hq // self.H, 0)[None]   # noqa: E731
            out.append(wide(x) + 2 * e[:, :, None] * wide(big))
        return np.concatenate(out)

    def scale(self):
        return float(np.float32(1.0 / np.sqrt(self.D)))


@pytest.mark.parametrize("block_size", [1, 16, 64, 256])
@pytest.mark.parametrize("heads,dim", [(12, 64), (5, 128), (1, 64)])
def test_append_codes_and_scales(pkv, cuda_dev, block_size, heads, dim):
    c = Case(pkv, cuda_dev, [1, 0, 40, 300, 17, 64, 257], heads, heads, dim, block_size)
    pkv.pf_device_status(reset=True)
    c.append([1, 0, 7, 130, 16, 1, 256])
    c.append([0, 0, 1, 100, 0, 63, 1])
    c.check_pool()
    for _ in range(5):   # decode steps, one token per growing sequence
        c.append([0, 0, 1, 1, 0, 0, 0], cu=False)
    c.append([0, 0, 27, 65, 1, 0, 0])
    assert np.array_equal(c.at, c.lens)
    c.check_pool()
    assert pkv.pf_device_status(reset=True) == 0


def test_append_extreme_values(pkv, cuda_dev):
    """The type's largest and smallest values, zeros, and pages whose scale
    grows by the whole range."""
    c = Case(pkv, cuda_dev, [48], 2, 2, 64, 16)
    tiny = np.zeros((16, 2, 64), np.float16)
    tiny[::2] = np.float16(2.0 ** -24)
    tiny[1, 0] = np.float16(2.0 ** -14)
    zero = np.zeros((8, 2, 64), np.float16)
    big = np.full((8, 2, 64), np.float16(65504.0))
    big[1::2] = np.float16(-65504.0)
    big[:, :, ::3] = np.float16(448.0)
    pkv.pf_device_status(reset=True)
    for x in (tiny, zero, big, big[:4], tiny[:12]):
        c.append([len(x)], k=x, v=-x)
    c.check_pool()
    assert pkv.pf_device_status(reset=True) == 0


def test_append_nonfinite_is_flagged_and_held_finite(pkv, cuda_dev):
    c = Case(pkv, cuda_dev, [20, 20], 2, 2, 64, 16)
    x = c.rows(40, spread=False)
    x[3, 0, 5], x[4, 1, 63], x[7, 0, 0], x[30] = np.inf, -np.inf, np.nan, np.nan
    pkv.pf_device_status(reset=True)
    c.append([20, 20], k=x, v=c.rows(40))
    assert pkv.pf_device_status(reset=True) == pkv.PF_DEV_NONFINITE
    c.check_pool()


def test_append_bad_values_are_flagged(pkv, cuda_dev):
    c = Case(pkv, cuda_dev, [16, 16], 2, 2, 64, 16)
    k = dev(c.rows(4), cuda_dev)
    before = host(c.k.view(c.torch.uint8)).copy()
    cu = dev(np.array([0, 2, 4], np.int32), cuda_dev)
    lens = dev(np.array([2, 2], np.int32), cuda_dev)
    pkv.pf_device_status(reset=True)
    bad = c.table.copy()
    bad[:, 0] = [c.N, -1]
    pkv.pf_append_kv(c.pool, 1, k, k, dev(bad, cuda_dev), lens, cu, 2)
    assert pkv.pf_device_status(reset=True) == pkv.PF_DEV_BAD_BLOCK_ID
    pkv.pf_append_kv(c.pool, 1, k, k, c.table_dev, dev(np.array([-3, 0], np.int32), cuda_dev), cu, 2)
    assert pkv.pf_device_status(reset=True) == pkv.PF_DEV_BAD_LENGTH
    assert np.array_equal(host(c.k.view(c.torch.uint8)), before)


CASES = [
    # lens, q-heads, kv-heads, head_dim, page
    ([1, 100, 17, 0, 64, 33], 12, 12, 64, 16),
    ([700, 1, 0, 255, 256, 257], 14, 2, 64, 64),
    ([90, 513], 8, 4, 128, 16),
    ([31, 32, 33], 10, 5, 128, 1),
    ([5, 1000], 3, 3, 64, 256),
    ([300], 16, 1, 128, 16),
    ([129, 64], 9, 1, 64, 1),
    ([4000], 1, 1, 64, 16),          # one context cut over many teams
    ([2500, 2], 4, 4, 128, 64),
]


@pytest.mark.parametrize("lens,hq,h,d,page", CASES)
@pytest.mark.parametrize("f32", [False, True])
def test_decode(pkv, cuda_dev, lens, hq, h, d, page, f32):
    import torch
    c = Case(pkv, cuda_dev, lens, hq, h, d, page, width=max(si.pages_for(max(lens), page), 2))
    c.fill()
    q = c.rng.standard_normal((len(lens), hq, d)).astype(np.float16)
    out = torch.full((len(lens) + 1, hq, d), 7.0, dtype=torch.float32 if f32 else torch.float16, device=cuda_dev)
    ws = pkv.make_workspace(c.pool, len(lens), hq, c.table.shape[1], 0)
    pkv.pf_device_status(reset=True)
    for _ in range(2):   # the workspace is ready for the next call
        pkv.pf_paged_decode_attention(c.pool, 1, dev(q, cuda_dev), c.table_dev, dev(c.lens, cuda_dev), c.scale(),
                                      out[:-1], 0, ws)
        assert pkv.pf_device_status(reset=True) == 0
        want, tol = c.want(q, np.arange(len(lens) + 1), False, 2.0 ** -21 if f32 else F16, F32 if f32 else F16)
        assert_within(host(out)[:-1], want, tol)
    assert bool((out[-1] == 7.0).all())      # the row behind the last sequence


def wide_table(c):
    """The table with room for 4096 more tokens, whose entries name no block:
    fp16 results then come from the few-rows kernel as well."""
    return np.pad(c.table, ((0, 0), (0, 4096 // c.B)), constant_values=1 << 30)


@pytest.mark.parametrize("lens,hq,h,d,page", CASES)
def test_decode_wide_table(pkv, cuda_dev, lens, hq, h, d, page):
    import torch
    c = Case(pkv, cuda_dev, lens, hq, h, d, page, width=max(si.pages_for(max(lens), page), 2))
    c.fill()
    table = dev(wide_table(c), cuda_dev)
    q = c.rng.standard_normal((len(lens), hq, d)).astype(np.float16)
    out = torch.full((len(lens) + 1, hq, d), 7.0, dtype=torch.float16, device=cuda_dev)
    ws = pkv.make_workspace(c.pool, len(lens), hq, table.shape[1], 0)
    pkv.pf_device_status(reset=True)
    for _ in range(2):
        pkv.pf_paged_decode_attention(c.pool, 1, dev(q, cuda_dev), table, dev(c.lens, cuda_dev), c.scale(),
                                      out[:-1], 0, ws)
        assert pkv.pf_device_status(reset=True) == 0
        want, tol = c.want(q, np.arange(len(lens) + 1), False, F16, F16)
        assert_within(host(out)[:-1], want, tol + c.small_terms(q, np.arange(len(lens) + 1)))
    assert bool((out[-1] == 7.0).all())


@pytest.mark.parametrize("lens,hq,h,d,page", [([100, 0, 300], 12, 12, 64, 16), ([1, 2000], 8, 2, 128, 64),
                                                ([900, 3, 0], 16, 1, 128, 16),    # 122 blocks' records, the prompt kernel
                                                ([40] * 160, 16, 1, 128, 16)])   # 41 blocks' records
def test_decode_noalloc(pkv, cuda_dev, lens, hq, h, d, page):
    """Without a workspace, tight table and wide: both kernels, the built-in scratch used twice."""
    import torch
    c = Case(pkv, cuda_dev, lens, hq, h, d, page)
    c.fill()
    q = c.rng.standard_normal((len(lens), hq, d)).astype(np.float16)
    want, tol = c.want(q, np.arange(len(lens) + 1), False, F16, F16)
    tol = tol + c.small_terms(q, np.arange(len(lens) + 1))
    for table in (c.table, wide_table(c), wide_table(c)):
        out = torch.full((len(lens), hq, d), 7.0, dtype=torch.float16, device=cuda_dev)
        pkv.pf_paged_decode_attention_noalloc(c.pool, 1, dev(q, cuda_dev), dev(table, cuda_dev), dev(c.lens, cuda_dev),
                                              c.scale(), out, 0)
        assert_within(host(out), want, tol)


def test_decode_step_wide_table(pkv, cuda_dev):
    """Steps whose attention sets out while the append runs, then contexts that are all empty."""
    import torch
    lens = [33, 1, 16, 900, 0, 2000]
    c = Case(pkv, cuda_dev, lens, 8, 4, 128, 16)
    c.append(np.maximum(c.lens - 1, 0))
    table, n = wide_table(c), len(lens)
    q = c.rng.standard_normal((n, 8, 128)).astype(np.float16)
    out = torch.empty((n, 8, 128), dtype=torch.float16, device=cuda_dev)
    ws = pkv.make_workspace(c.pool, n, 8, table.shape[1], 0)
    k, v = c.rows(n), c.rows(n)
    args = (dev(q, cuda_dev), dev(k, cuda_dev), dev(v, cuda_dev), dev(table, cuda_dev))
    pkv.pf_decode_step(c.pool, 1, *args, dev(c.lens, cuda_dev), c.scale(), out, 0, ws)
    one = np.concatenate([[0], np.cumsum(c.lens > 0)])     # the empty context takes no row
    c.km.append(k[c.lens > 0], c.table, c.lens, one)
    c.vm.append(v[c.lens > 0], c.table, c.lens, one)
    c.check_pool()
    want, tol = c.want(q, np.arange(n + 1), False, F16, F16)
    assert_within(host(out), want, tol + c.small_terms(q, np.arange(n + 1)))
    pkv.pf_decode_step(c.pool, 1, *args, dev(np.zeros(n, np.int32), cuda_dev), c.scale(), out, 0, ws)
    assert not host(out).any()
    c.check_pool()
    assert pkv.pf_device_status(reset=True) == 0


@pytest.mark.parametrize("lens,new,hq,h,d,page,ws", [
    ([40, 17, 3, 300], [3, 1, 3, 0], 12, 12, 64, 16, True),
    ([40, 500, 16], [2, 2, 1], 14, 2, 64, 64, True),          # 14 rows per kv-head
    ([100, 33], [16, 2], 5, 5, 128, 1, True),
    ([100, 33], [5, 2], 5, 5, 128, 1, False),                 # few rows, no workspace
    ([300, 7, 0, 129], [300, 7, 0, 128], 4, 4, 64, 16, True),  # tcgen05 kernel
    ([200, 513, 64], [150, 400, 1], 8, 2, 128, 16, True),
    ([70, 90], [70, 33], 6, 2, 64, 1, False),
    ([257, 600], [256, 130], 2, 1, 128, 256, False),
    ([65, 128], [65, 128], 3, 3, 128, 64, False),
    # few blocks of rows: contexts cut into parts, the last of which some rows do not see
    ([5000, 64, 700], [33, 64, 17], 2, 1, 128, 16, True),
    ([6000], [700], 2, 2, 64, 64, True),
    ([1100, 515], [1030, 20], 1, 1, 64, 256, True),
    ([900, 1], [300, 1], 4, 2, 128, 1, True),
    ([2000, 130, 127, 128], [128, 128, 100, 33], 1, 1, 64, 16, True),
])
@pytest.mark.parametrize("f32", [False, True])
def test_append_attention(pkv, cuda_dev, lens, new, hq, h, d, page, ws, f32):
    import torch
    c = Case(pkv, cuda_dev, lens, hq, h, d, page)
    c.fill()
    offs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = c.rng.standard_normal((int(offs[-1]), hq, d)).astype(np.float16)
    out = torch.full((int(offs[-1]) + 1, hq, d), 7.0, dtype=torch.float32 if f32 else torch.float16, device=cuda_dev)
    work = pkv.make_prefill_workspace(c.pool, len(lens), hq, c.table.shape[1], max(new)) if ws else None
    pkv.pf_device_status(reset=True)
    pkv.pf_paged_prefill_attention(c.pool, 1, dev(q, cuda_dev), c.table_dev, dev(c.lens, cuda_dev),
                                   dev(offs, cuda_dev), max(new), c.scale(), out[:-1], work)
    assert pkv.pf_device_status(reset=True) == 0
    # the prompt kernel rounds weights to fp16 whatever the output's type; its dequantised values may be off
    # by 2^-25 where they are below 2^-14 (rows of K: that times the sum of |q|)
    fine = f32 and work is not None and max(new) * (hq // h) <= 16
    want, tol = c.want(q, offs, True, 2.0 ** -21 if fine else F16, F32 if f32 else F16)
    tol = tol + 2.0 ** -25 + 2 * 2.0 ** -25 * c.scale() * np.abs(q.astype(np.float64)).sum(-1).max() * 64
    assert_within(host(out)[:-1], want, tol)
    assert bool((out[-1] == 7.0).all())


@pytest.mark.parametrize("lens,new,hq,h,d,page", [
    ([40, 17, 3, 300], [3, 1, 3, 0], 12, 12, 64, 16),
    ([40, 500, 16], [2, 2, 1], 14, 2, 64, 64),                # 14 rows per kv-head
    ([100, 33], [16, 2], 5, 5, 128, 1),
    ([1000, 16], [4, 4], 8, 2, 128, 256),
    # 9 to 16 rows: with more than a block per SM on the few-rows kernel
    ([3 + 7 * i % 90 for i in range(40)], [1 + i % 3 for i in range(40)], 25, 5, 64, 16),
    ([3 + 7 * i % 90 for i in range(40)], [1 + i % 3 for i in range(40)], 20, 5, 128, 16),
    ([3 + 7 * i % 90 for i in range(80)], [1 + i % 3 for i in range(80)], 8, 2, 128, 1),
    ([2000], [5], 9, 3, 64, 16),                                # ... with fewer on the prompt kernel, cut
])
def test_append_attention_wide_table(pkv, cuda_dev, lens, new, hq, h, d, page):
    import torch
    c = Case(pkv, cuda_dev, lens, hq, h, d, page)
    c.fill()
    offs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = c.rng.standard_normal((int(offs[-1]), hq, d)).astype(np.float16)
    out = torch.full((int(offs[-1]) + 1, hq, d), 7.0, dtype=torch.float16, device=cuda_dev)
    table = dev(wide_table(c), cuda_dev)
    work = pkv.make_prefill_workspace(c.pool, len(lens), hq, table.shape[1], max(new))
    pkv.pf_device_status(reset=True)
    pkv.pf_paged_prefill_attention(c.pool, 1, dev(q, cuda_dev), table, dev(c.lens, cuda_dev), dev(offs, cuda_dev),
                                   max(new), c.scale(), out[:-1], work)
    assert pkv.pf_device_status(reset=True) == 0
    want, tol = c.want(q, offs, True, F16, F16)
    assert_within(host(out)[:-1], want, tol + c.small_terms(q, offs))
    assert bool((out[-1] == 7.0).all())


@pytest.mark.parametrize("wide", [False, True])
def test_wide_range_of_value_scales(pkv, cuda_dev, wide):
    """Pages whose V scales differ by 2^20: an outlier page of little weight
    must not cost the others their precision."""
    import torch
    c = Case(pkv, cuda_dev, [64], 1, 1, 64, 16)
    k = np.zeros((64, 1, 64), np.float16)
    v = c.rows(64, spread=False)
    k[16:32, :, 0] = -100.0                       # the outlier page: weight e^-12.5 of the others
    v[16:32] *= np.float16(1024.0)
    v[32:48] *= np.float16(2.0 ** -6)
    c.append([64], k=k, v=v)
    q = np.zeros((1, 1, 64), np.float16)
    q[:, :, 0] = 1.0
    for f32 in (False, True):
        out = torch.empty((1, 1, 64), dtype=torch.float32 if f32 else torch.float16, device=cuda_dev)
        table = wide_table(c) if wide else c.table
        ws = pkv.make_workspace(c.pool, 1, 1, table.shape[1], 0)
        pkv.pf_paged_decode_attention(c.pool, 1, dev(q, cuda_dev), dev(table, cuda_dev), dev(c.lens, cuda_dev),
                                      c.scale(), out, 0, ws)
        want, tol = c.want(q, [0, 1], False, 2.0 ** -21 if f32 else F16, F32 if f32 else F16)
        assert_within(host(out), want, tol)


@pytest.mark.parametrize("page", [16, 1])
def test_decode_step_appends_then_attends(pkv, cuda_dev, page):
    import torch
    lens = [33, 1, 16, 200]
    c = Case(pkv, cuda_dev, lens, 8, 4, 64, page)
    c.append(c.lens - 1)
    k, v = c.rows(4), c.rows(4)
    q = c.rng.standard_normal((4, 8, 64)).astype(np.float16)
    out = torch.empty((4, 8, 64), dtype=torch.float16, device=cuda_dev)
    ws = pkv.make_workspace(c.pool, 4, 8, c.table.shape[1], 0)
    pkv.pf_decode_step(c.pool, 1, dev(q, cuda_dev), dev(k, cuda_dev), dev(v, cuda_dev), c.table_dev,
                       dev(c.lens, cuda_dev), c.scale(), out, 0, ws)
    one = np.arange(5)
    c.km.append(k, c.table, c.lens, one)
    c.vm.append(v, c.table, c.lens, one)
    c.check_pool()
    want, tol = c.want(q, one, False, F16, F16)
    assert_within(host(out), want, tol)
    assert pkv.pf_device_status(reset=True) == 0


@pytest.mark.parametrize("page,h,d", [(16, 12, 64), (1, 3, 128), (256, 1, 64)])
def test_gather_widens(pkv, cuda_dev, page, h, d):
    import torch
    lens = [70, 0, 1, 300]
    c = Case(pkv, cuda_dev, lens, h, h, d, page)
    c.fill()
    off = np.array([2, 0, 75, 80], np.int64)
    outs = [torch.full((400, h, d), 7.0, dtype=torch.float16, device=cuda_dev) for _ in range(2)]
    pkv.pf_gather_kv(c.pool, 1, c.table_dev, dev(c.lens, cuda_dev), dev(off, cuda_dev), *outs)
    for out, m in zip(outs, (c.km, c.vm)):
        want = np.full((400, h, d), 7.0)
        for s, L in enumerate(lens):
            want[off[s]:off[s] + L] = m.rows(c.table[s], L)
        assert np.array_equal(host(out), want.astype(np.float16))


def test_copy_blocks_and_swap(pkv, cuda_dev):
    """Codes and scales of every layer move together, bit for bit."""
    import torch
    for h, page in ((3, 16), (12, 64), (1, 1)):
        c = Case(pkv, cuda_dev, [page * 4], h, h, 64, page, spare=6)
        c.append([page * 4])
        src, dst = c.table[0][:3].copy(), np.setdiff1d(np.arange(c.N), c.table[0])[:3].astype(np.int32)
        snap = [host(t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t.view(torch.int32)).copy()
                for t in (c.k, c.v, c.ks, c.vs)]
        now = lambda: [host(t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t.view(torch.int32))   # noqa: E731
                       for t in (c.k, c.v, c.ks, c.vs)]
        pkv.pf_copy_blocks(c.pool, dev(src, cuda_dev), dev(dst, cuda_dev))
        for was, is_ in zip(snap, now()):
            was[:, dst] = was[:, src]
            assert np.array_equal(was, is_)
        n = pkv.pf_block_image_bytes(c.pool)
        assert n == 2 * 2 * (page * h * 64 + (4 * h + 15) // 16 * 16)
        buf = torch.zeros(3 * n, dtype=torch.uint8).pin_memory()
        pkv.pf_swap_out(c.pool, dev(src, cuda_dev), buf)
        torch.cuda.synchronize()
        for t in (c.k, c.v):
            t.view(torch.uint8)[:, torch.from_numpy(src).long().to(cuda_dev)] = 0
        back = dst[::-1].copy()
        pkv.pf_swap_in(c.pool, buf, dev(back, cuda_dev))
        for was, is_, codes in zip(snap, now(), (1, 1, 0, 0)):
            was[:, back] = was[:, src]
            if codes:
                was[:, src] = 0
            assert np.array_equal(was, is_)


def test_captured_and_replayed(pkv, cuda_dev):
    """A decode step captured into two graphs that share a workspace: replays
    with other inputs give what the plain call gives."""
    import torch
    c = Case(pkv, cuda_dev, [700, 1300, 64], 4, 4, 64, 16)
    c.append(c.lens - 1)
    ws = pkv.make_workspace(c.pool, 3, 4, c.table.shape[1], 0)
    lens = dev(c.lens, cuda_dev)
    q, k, v = (torch.zeros((3, 4, 64), dtype=torch.float16, device=cuda_dev) for _ in range(3))
    outs = [torch.empty_like(q) for _ in range(2)]
    call = lambda o: pkv.pf_decode_step(c.pool, 1, q, k, v, c.table_dev, lens, c.scale(), o, 0, ws)   # noqa: E731
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(outs[0])
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, o in zip(graphs, outs):
        with torch.cuda.graph(g):
            call(o)
    before = (c.km.code.copy(), c.km.scale.copy(), c.vm.code.copy(), c.vm.scale.copy())
    codes = [t.clone() for t in (c.k.view(torch.uint8), c.v.view(torch.uint8), c.ks, c.vs)]
    for i in range(4):
        kn, vn = c.rows(3, spread=False), c.rows(3, spread=False)
        qn = c.rng.standard_normal((3, 4, 64)).astype(np.float16)
        for t, x in ((q, qn), (k, kn), (v, vn)):
            t.copy_(dev(x, cuda_dev))
        for t, x in zip((c.k.view(torch.uint8), c.v.view(torch.uint8), c.ks, c.vs), codes):
            t.copy_(x)
        c.km.code, c.km.scale, c.vm.code, c.vm.scale = (x.copy() for x in before)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        c.km.append(kn, c.table, c.lens, np.arange(4))
        c.vm.append(vn, c.table, c.lens, np.arange(4))
        want, tol = c.want(qn, np.arange(4), False, F16, F16)
        # (the first call, before the capture, may have rounded the earlier rows to zero rows' scale: none grows)
        assert_within(host(outs[i % 2]), want, tol, f"replay {i}")


def test_two_streams_with_their_own_workspaces(pkv, cuda_dev):
    import torch
    c = Case(pkv, cuda_dev, [1500, 900], 6, 6, 64, 16)
    c.fill()
    q = c.rng.standard_normal((2, 6, 64)).astype(np.float16)
    qd, lens = dev(q, cuda_dev), dev(c.lens, cuda_dev)
    ws = [pkv.make_workspace(c.pool, 2, 6, c.table.shape[1], 0) for _ in range(2)]
    outs = [torch.empty_like(qd) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, o, w in zip(streams, outs, ws):
            pkv.pf_paged_decode_attention(c.pool, 1, qd, c.table_dev, lens, c.scale(), o, 0, w, stream=st)
    torch.cuda.synchronize()
    want, tol = c.want(q, np.arange(3), False, F16, F16)
    for o in outs:
        assert_within(host(o), want, tol)


def test_workspace_shared_with_an_fp16_pool(pkv, cuda_dev):
    """One workspace, calls of both pool types in turn."""
    import torch
    from gpu_util import PagedCase, assert_close_to_oracle
    import oracle
    oracle.build()
    c = Case(pkv, cuda_dev, [1500, 900], 6, 6, 64, 16)
    c.fill()
    f = PagedCase(pkv, cuda_dev, [1500, 900], 6, 6, 64, 16)
    q = c.rng.standard_normal((2, 6, 64)).astype(np.float16)
    qd, lens = dev(q, cuda_dev), dev(c.lens, cuda_dev)
    ws = max((pkv.make_workspace(p, 2, 6, f.bt.shape[1], 0) for p in (c.pool, f.pool)), key=lambda t: t.numel())
    want, tol = c.want(q, np.arange(3), False, F16, F16)
    for _ in range(3):
        out = torch.empty_like(qd)
        pkv.pf_paged_decode_attention(c.pool, 1, qd, c.table_dev, lens, c.scale(), out, 0, ws)
        assert_within(host(out), want, tol)
        assert_close_to_oracle(host(f.attention(0.125, ws=ws)), f.oracle(oracle, 0.125))


def test_tensors_elsewhere_are_refused(pkv, cuda_dev):
    """Tensors of the host, of another type or not contiguous: an error that names the argument, nothing launched."""
    import torch
    c = Case(pkv, cuda_dev, [33, 5], 4, 4, 64, 16)
    c.fill()
    q = torch.zeros((2, 4, 64), dtype=torch.float16, device=cuda_dev)
    out, lens = torch.full_like(q, 7.0), dev(c.lens, cuda_dev)
    ws = pkv.make_workspace(c.pool, 2, 4, c.table.shape[1], 0)
    good = [q, c.table_dev, lens, c.scale(), out, 0, ws]
    for i, bad, name in ((0, q.cpu(), "q"), (1, c.table_dev.cpu(), "block_tables"), (2, lens.long(), "context_lens"),
                         (4, out.cpu(), "out"), (6, ws.cpu(), "workspace"),
                         (0, q.transpose(0, 1).contiguous().transpose(0, 1), "q")):
        args = list(good)
        args[i] = bad
        with pytest.raises(pkv.PagedKVError, match=name):
            pkv.pf_paged_decode_attention(c.pool, 1, *args)
    with pytest.raises(pkv.PagedKVError, match="k_new"):
        pkv.pf_append_kv(c.pool, 1, q.cpu(), q, c.table_dev, lens, None)
    with pytest.raises(pkv.PagedKVError, match="block_map"):
        ids = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
        pkv.pf_compact_blocks(c.pool, ids, ids, torch.zeros(c.N, dtype=torch.int32), c.table_dev, lens)
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("hq,h,new", [(16, 1, 1), (2, 2, 1), (2, 1, 4), (2, 1, 40)])
def test_workspace_of_a_larger_batch(pkv, cuda_dev, hq, h, new):
    """A workspace made for the largest batch serves smaller ones, whose contexts are cut further;
    with one that is too small a call of many rows cuts less."""
    import torch
    c = Case(pkv, cuda_dev, [3000], hq, h, 128, 16)
    c.fill()
    offs = np.array([0, new], np.int32)
    q = c.rng.standard_normal((new, hq, 128)).astype(np.float16)
    want, tol = c.want(q, offs, True, F16, F16)
    out = torch.empty((new, hq, 128), dtype=torch.float16, device=cuda_dev)
    lens, table, qd = dev(c.lens, cuda_dev), c.table_dev, dev(q, cuda_dev)
    for n in (500, 40, 1):
        ws = pkv.make_prefill_workspace(c.pool, n, hq, table.shape[1], new)
        pkv.pf_paged_prefill_attention(c.pool, 1, qd, table, lens, dev(offs, cuda_dev), new, c.scale(), out, ws)
        assert_within(host(out), want, tol + c.small_terms(q, offs), f"made for {n}")
        if new == 1:
            ws = pkv.make_workspace(c.pool, n, hq, table.shape[1], 0)
            pkv.pf_paged_decode_attention(c.pool, 1, qd, table, lens, c.scale(), out, 0, ws)
            assert_within(host(out), want, tol + c.small_terms(q, offs), f"decode, made for {n}")
    if new == 40:
        for kb in (16, 600):                      # no part fits; four do
            ws = torch.zeros(kb * 1024, dtype=torch.uint8, device=cuda_dev)
            pkv.pf_paged_prefill_attention(c.pool, 1, qd, table, lens, dev(offs, cuda_dev), new, c.scale(), out, ws)
            assert_within(host(out), want, tol + c.small_terms(q, offs), f"{kb} KiB")


def test_cut_contexts_captured_and_replayed(pkv, cuda_dev):
    """Two captured calls of cut contexts that share a workspace, replayed with other lengths and queries."""
    import torch
    c = Case(pkv, cuda_dev, [5000, 1500], 4, 2, 64, 16)
    c.fill()
    new, offs = [20, 30], np.array([0, 20, 50], np.int32)
    ws = pkv.make_prefill_workspace(c.pool, 2, 4, c.table.shape[1], 30)
    qd = torch.zeros((50, 4, 64), dtype=torch.float16, device=cuda_dev)
    lens, cu = dev(c.lens, cuda_dev), dev(offs, cuda_dev)
    outs = [torch.empty_like(qd) for _ in range(2)]
    call = lambda o: pkv.pf_paged_prefill_attention(c.pool, 1, qd, c.table_dev, lens, cu, max(new), c.scale(), o, ws)   # noqa: E731
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(outs[0])
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, o in zip(graphs, outs):
        with torch.cuda.graph(g):
            call(o)
    full = c.lens
    for i, now in enumerate(([5000, 1500], [400, 30], [2049, 1024], [20, 1500])):
        q = c.rng.standard_normal((50, 4, 64)).astype(np.float16)
        c.lens = np.array(now, np.int32)
        qd.copy_(dev(q, cuda_dev))
        lens.copy_(dev(c.lens, cuda_dev))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        want, tol = c.want(q, offs, True, F16, F16)
        assert_within(host(outs[i % 2]), want, tol + c.small_terms(q, offs), f"replay {i}")
    c.lens = full
