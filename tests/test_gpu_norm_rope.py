"""Norms, rotation and cache write (pf_norm_rope_write) on the GPU against a
plain 64-bit form; every byte of the pools is compared."""
import numpy as np
import pytest

from e4m3_util import assert_within
from gpu_util import PagedCase, dev, host
from test_gpu_e4m3 import Case

pytestmark = pytest.mark.gpu


def rotated64(x, weight, eps, angles, p, interleaved):
    """fp64 rows and how far fp32 arithmetic and one rounding to fp16 may be off.

    The sum of D squares is off by at most D 2^-24 relative (its root by half),
    eps and the mean by 2^-23, the reciprocal root by 2^-22, two products by
    2^-23: a normed value by e = (D / 2 + 10) 2^-24.  A turned one is a sum of two
    products of it: (|a c| + |b s|) (e + 2^-23).  The result is rounded to
    fp16 (2^-11 relative, or 2^-25)."""
    x = x.astype(np.float64)
    D = x.shape[-1]
    e = 0.0
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps))) * weight.astype(np.float64)
        e = (D / 2 + 10) * 2.0 ** -24
    size = np.abs(x)
    out = x.copy()
    if angles is not None:
        rot = angles.shape[1]
        c, s = (y[:, None].astype(np.float64) for y in np.split(angles[p], 2, axis=1))
        i = np.arange(rot // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
        size[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
        size[..., b] = np.abs(x[..., b] * c) + np.abs(x[..., a] * s)
    return out, size * (e + 2.0 ** -23) + np.abs(out) * 2.0 ** -11 + 2.0 ** -25


class Rows:
    """New rows of the last `new` tokens of each context, as slices of one projection or apart."""

    def __init__(self, pkv, device, lens, new, hq, h, d, page, packed=False, norm=True, rot=None, theta=10000.0, seed=3,
                 layers=2):
        import torch
        self.c = PagedCase(pkv, device, lens, hq, h, d, page, n_layers=layers)
        rng = np.random.default_rng(seed)
        T = int(sum(new))
        self.packed_host = (rng.standard_normal((T, hq + 2 * h, d)) * 2).astype(np.float16)
        self.q, self.k, self.v = np.split(self.packed_host, [hq, hq + h], axis=1)
        x = dev(self.packed_host, device)
        self.qd, self.kd, self.vd = x[:, :hq], x[:, hq:hq + h], x[:, hq + h:]
        if not packed:
            self.qd, self.kd, self.vd = self.qd.contiguous(), self.kd.contiguous(), self.vd.contiguous()
        self.qw, self.kw = ((1 + 0.2 * rng.standard_normal(d)).astype(np.float32) for _ in range(2)) if norm else (None, None)
        self.seq = np.repeat(np.arange(len(lens)), new).astype(np.int32)
        self.pos = np.concatenate([np.arange(L - n, L) for L, n in zip(lens, new)]).astype(np.int32)
        rot = d if rot is None else rot
        self.angles_dev = pkv.make_rope_angles(max(1, max(lens)), rot, theta, device=device) if rot else None
        self.angles = host(self.angles_dev) if rot else None
        self.weights = {n: None if w is None else dev(w, device) for n, w in (("q_weight", self.qw), ("k_weight", self.kw))}
        self.out = torch.full((T + 1, hq, d), 7.0, dtype=torch.float16, device=device)
        self.ids = [dev(x, device) for x in (self.seq, self.pos)]

    def slots(self):
        B = self.c.B
        return self.c.bt[self.seq, self.pos // B], self.pos % B

    def check_cache(self, layer, k64, ktol, rows=slice(None), v=None):
        """K within its bound, V bit for bit, everything else as it was."""
        blk, at = (x[rows] for x in self.slots())
        for t, was, new in ((self.c.k_dev, self.c.k_host, None), (self.c.v_dev, self.c.v_host, self.v if v is None else v)):
            got = host(t)
            if new is None:
                assert_within(got[layer, blk, at], k64[rows], ktol[rows], "k")
                new = got[layer, blk, at]
            else:
                new = new[rows]
            want = was.copy()
            want[layer, blk, at] = new
            assert np.array_equal(got.view(np.uint16), want.view(np.uint16))


CASES = [
    # lengths, new tokens, q-heads, kv-heads, head_dim, page
    ([40, 1, 17, 300], [1, 1, 1, 1], 12, 12, 64, 16),
    ([40, 0, 17, 300], [23, 0, 17, 3], 14, 2, 64, 64),
    ([100, 65], [100, 1], 40, 40, 128, 16),
    ([700, 3], [70, 2], 32, 8, 128, 256),
    ([50, 9], [50, 9], 5, 5, 128, 1),
    ([33], [1], 1, 1, 64, 16),
    ([33], [5], 16, 1, 128, 1),
]


@pytest.mark.parametrize("lens,new,hq,h,d,page", CASES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm,rot,packed", [(True, None, False), (False, None, True), (True, 0, True), (True, 16, False),
                                             (False, 32, False), (True, 48, True), (False, 0, False)])
def test_rows(pkv, cuda_dev, lens, new, hq, h, d, page, interleaved, norm, rot, packed):
    r = Rows(pkv, cuda_dev, lens, new, hq, h, d, page, packed, norm, rot)
    pkv.pf_device_status(reset=True)
    for _ in range(2):
        pkv.pf_norm_rope_write(r.c.pool, 1, r.qd, r.kd, r.vd, r.c.bt_dev, *r.ids, r.angles_dev, r.out[:-1], eps=1e-5,
                               interleaved=interleaved, **r.weights)
        assert pkv.pf_device_status(reset=True) == 0
        want, tol = rotated64(r.q, r.qw, 1e-5, r.angles, r.pos, interleaved)
        assert_within(host(r.out)[:-1], want, tol, "q")
        r.check_cache(1, *rotated64(r.k, r.kw, 1e-5, r.angles, r.pos, interleaved))
    assert bool((r.out[-1] == 7.0).all())


@pytest.mark.parametrize("d,hq,h", [(64, 6, 2), (128, 3, 3)])
def test_without_a_cache(pkv, cuda_dev, d, hq, h):
    """Keys into k_out, in place too, and then quantised into an 8-bit pool; only queries; only keys."""
    import torch
    lens, new = [60, 5, 31], [33, 5, 1]
    r = Rows(pkv, cuda_dev, lens, new, hq, h, d, 16, packed=True)
    c8 = Case(pkv, cuda_dev, lens, hq, h, d, 16)
    rope_pos = np.random.default_rng(1).integers(0, max(lens), len(r.pos)).astype(np.int32)
    rp = dev(rope_pos, cuda_dev)
    k_out = torch.empty((len(r.pos), h, d), dtype=torch.float16, device=cuda_dev)
    args = (None, None, None, r.angles_dev)
    pkv.pf_device_status(reset=True)
    pkv.pf_norm_rope_write(c8.pool, 1, r.qd, r.kd, None, *args, r.out[:-1], k_out, rope_pos=rp, **r.weights)
    wq, wk = (rotated64(x, w, 1e-6, r.angles, rope_pos, False) for x, w in ((r.q, r.qw), (r.k, r.kw)))
    assert_within(host(r.out)[:-1], *wq)
    assert_within(host(k_out), *wk)
    both = [host(r.out).copy(), host(k_out).copy()]
    c8.append([lens[s] - new[s] for s in range(3)])
    c8.append(new, host(k_out), r.v)
    c8.check_pool()
    # one at a time, and into another layout
    wide = torch.zeros((len(r.pos), h + 1, d), dtype=torch.float16, device=cuda_dev)
    pkv.pf_norm_rope_write(c8.pool, 0, r.qd, None, None, *args, r.out[:-1], rope_pos=rp, q_weight=r.weights["q_weight"])
    pkv.pf_norm_rope_write(c8.pool, 0, None, r.kd, None, *args, None, wide[:, 1:], rope_pos=rp, k_weight=r.weights["k_weight"])
    assert np.array_equal(host(r.out), both[0]) and np.array_equal(host(wide)[:, 1:], both[1]) and not host(wide)[:, 0].any()
    # in place: the slices of the projection take the results, V stays
    pkv.pf_norm_rope_write(c8.pool, 0, r.qd, r.kd, None, *args, r.qd, r.kd, rope_pos=rp, **r.weights)
    assert np.array_equal(host(r.qd), both[0][:-1]) and np.array_equal(host(r.kd), both[1]) and np.array_equal(host(r.vd), r.v)
    assert pkv.pf_device_status(reset=True) == 0


def test_k_out_beside_the_cache(pkv, cuda_dev):
    """Rotation positions apart from the slots', as drafts have them; the same bits in k_out and in the pages."""
    import torch
    r = Rows(pkv, cuda_dev, [90, 40], [12, 7], 4, 2, 64, 16)
    rope_pos = (r.pos - np.arange(len(r.pos)) % 3).astype(np.int32)
    k_out = torch.empty((len(r.pos), 2, 64), dtype=torch.float16, device=cuda_dev)
    pkv.pf_norm_rope_write(r.c.pool, 0, r.qd, r.kd, r.vd, r.c.bt_dev, *r.ids, r.angles_dev, r.out[:-1], k_out,
                           rope_pos=dev(rope_pos, cuda_dev), **r.weights)
    r.check_cache(0, *rotated64(r.k, r.kw, 1e-6, r.angles, rope_pos, False))
    assert np.array_equal(host(r.c.k_dev)[(0, *r.slots())], host(k_out))
    assert_within(host(r.out)[:-1], *rotated64(r.q, r.qw, 1e-6, r.angles, rope_pos, False))


def test_keys_alone_into_the_cache(pkv, cuda_dev):
    """Without queries, and with a norm of one kind only."""
    r = Rows(pkv, cuda_dev, [90, 40], [12, 7], 4, 2, 64, 16)
    pkv.pf_norm_rope_write(r.c.pool, 1, None, r.kd, r.vd, r.c.bt_dev, *r.ids, r.angles_dev, None)
    r.check_cache(1, *rotated64(r.k, None, 0, r.angles, r.pos, False))
    r = Rows(pkv, cuda_dev, [90, 40], [12, 7], 4, 2, 64, 16, packed=True)
    pkv.pf_norm_rope_write(r.c.pool, 1, r.qd, r.kd, r.vd, r.c.bt_dev, *r.ids, r.angles_dev, r.out[:-1],
                           k_weight=r.weights["k_weight"], eps=0.0)
    r.check_cache(1, *rotated64(r.k, r.kw, 0.0, r.angles, r.pos, False))
    assert_within(host(r.out)[:-1], *rotated64(r.q, None, 0, r.angles, r.pos, False))


def test_broadcast_rows(pkv, cuda_dev):
    """One token's rows for all positions (a stride of 0 between tokens)."""
    import torch
    r = Rows(pkv, cuda_dev, [30], [9], 3, 3, 128, 16)
    one = r.qd[:1].expand(9, 3, 128)
    out = torch.empty((9, 3, 128), dtype=torch.float16, device=cuda_dev)
    pkv.pf_norm_rope_write(r.c.pool, 0, one, r.kd[:1].expand(9, 3, 128), r.vd, r.c.bt_dev, *r.ids, r.angles_dev, out)
    want, tol = rotated64(np.repeat(r.q[:1], 9, 0), None, 0, r.angles, r.pos, False)
    assert_within(host(out), want, tol)
    with pytest.raises(pkv.PagedKVError, match="overlap"):
        pkv.pf_norm_rope_write(r.c.pool, 0, r.qd, None, None, None, None, None, r.angles_dev, one, rope_pos=r.ids[1])


def test_flags(pkv, cuda_dev):
    """Bad positions and blocks are flagged; their rows stay as they were, all others are written."""
    pkv.pf_device_status(reset=True)
    for what in ("angle", "negative angle", "sequence", "position", "negative position", "block", "negative block"):
        r = Rows(pkv, cuda_dev, [40, 33], [6, 5], 4, 2, 64, 16)
        seq, pos, rope_pos, bt = r.seq.copy(), r.pos.copy(), r.pos.copy(), r.c.bt.copy()
        bad = 7
        if what.endswith("angle"):
            rope_pos[bad] = -1 if what[0] == "n" else len(r.angles)
        elif what == "sequence":
            seq[bad] = 2
        elif what.endswith("position"):
            pos[bad] = -1 if what[0] == "n" else bt.shape[1] * 16
        else:
            bt[1, 1] = -1 if what[0] == "n" else r.c.n_blocks
        pkv.pf_norm_rope_write(r.c.pool, 0, r.qd, r.kd, r.vd, dev(bt, cuda_dev), dev(seq, cuda_dev), dev(pos, cuda_dev),
                               r.angles_dev, r.out[:-1], rope_pos=dev(rope_pos, cuda_dev), **r.weights)
        flag = pkv.PF_DEV_BAD_BLOCK_ID if what.endswith("block") else pkv.PF_DEV_BAD_POSITION
        assert pkv.pf_device_status(reset=True) == flag, what
        good = np.ones(len(pos), bool)
        good[bad] = False
        if what.endswith("block"):
            good &= (r.seq != 1) | (r.pos // 16 != 1)
        rows = good.copy()
        want, tol = rotated64(r.q, r.qw, 1e-6, r.angles, r.pos, False)
        if what.endswith("angle"):
            assert np.all(host(r.out)[bad] == 7.0)
        else:
            good[:] = True
        assert_within(host(r.out)[:-1][good], want[good], tol[good], what)
        if what.endswith("angle"):                    # V does not turn: it is written
            blk, at = r.slots()
            assert np.array_equal(host(r.c.v_dev)[0, blk, at], r.v)
            k64, ktol = rotated64(r.k, r.kw, 1e-6, r.angles, r.pos, False)
            got = host(r.c.k_dev)[0, blk, at]
            assert_within(got[rows], k64[rows], ktol[rows])
            assert np.array_equal(got[bad], r.c.k_host[0, blk, at][bad])
        else:
            r.check_cache(0, *rotated64(r.k, r.kw, 1e-6, r.angles, r.pos, False), rows=rows)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_non_finite_values_stay_in_their_rows(pkv, cuda_dev, norm, interleaved):
    r = Rows(pkv, cuda_dev, [20], [9], 6, 2, 128, 16, norm=norm, rot=64)
    bad = r.q.copy()
    bad[3, 1, 5], bad[4, 2, 100], bad[5, 5, 40] = np.nan, np.inf, 0
    bad[6, 0], bad[7, 0] = 0, 65504
    pkv.pf_norm_rope_write(r.c.pool, 0, dev(bad, cuda_dev), r.kd, r.vd, r.c.bt_dev, *r.ids, r.angles_dev, r.out[:-1],
                           interleaved=interleaved, **r.weights)
    got = host(r.out)[:-1].astype(np.float64)
    with np.errstate(all="ignore"):
        want, tol = rotated64(bad, r.qw, 1e-6, r.angles, r.pos, interleaved)
    rows = np.ones((9, 6), bool)
    rows[3, 1] = rows[4, 2] = rows[7, 0] = False
    assert_within(got[rows], want[rows], tol[rows])
    assert not got[6, 0].any()
    if norm:
        assert np.all(np.isnan(got[3, 1])) and np.isnan(got[4, 2, 100])
        assert_within(got[7, 0], want[7, 0], tol[7, 0])
    else:
        i = np.arange(128)
        pair = {5, 4} if interleaved else {5, 37}
        assert np.all(np.isnan(got[3, 1, list(pair)])) and np.all(np.isfinite(got[3, 1, [x for x in i if x not in pair]]))
        assert got[4, 2, 100] == np.inf and np.all(np.isfinite(got[4, 2, i != 100]))


def test_other_stream_and_replays(pkv, cuda_dev):
    """A call on a side stream, and two captured ones replayed in turn on new inputs."""
    import torch
    r = Rows(pkv, cuda_dev, [200, 17], [90, 17], 8, 2, 64, 16)
    outs = [torch.empty_like(r.qd) for _ in range(2)]
    call = lambda o, layer: pkv.pf_norm_rope_write(   # noqa: E731
        r.c.pool, layer, r.qd, r.kd, r.vd, r.c.bt_dev, *r.ids, r.angles_dev, o, **r.weights)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(outs[0], 0)
    side.synchronize()
    assert_within(host(outs[0]), *rotated64(r.q, r.qw, 1e-6, r.angles, r.pos, False))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            call(outs[i], i)
    rng = np.random.default_rng(4)
    for i in range(4):
        qn, kn = (rng.standard_normal(tuple(x.shape)).astype(np.float16) for x in (r.qd, r.kd))
        r.qd.copy_(dev(qn, cuda_dev))
        r.kd.copy_(dev(kn, cuda_dev))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert_within(host(outs[i % 2]), *rotated64(qn, r.qw, 1e-6, r.angles, r.pos, False))
        blk, at = r.slots()
        assert_within(host(r.c.k_dev)[i % 2, blk, at], *rotated64(kn, r.kw, 1e-6, r.angles, r.pos, False))


def test_far_blocks_and_wide_rows(pkv, cuda_dev):
    """Pages past 2^32 bytes of the pool, and tokens 2^31 values and more apart in the projection."""
    import torch
    n_blocks, stride = 8600, 2 ** 30 + 8
    k, v = (torch.empty((1, n_blocks, 256, 8, 128), dtype=torch.float16, device=cuda_dev) for _ in range(2))
    pool = pkv.pf_pool_create(k, v)
    flat = torch.empty(2 * stride + 24 * 128, dtype=torch.float16, device=cuda_dev)
    x = flat.as_strided((3, 24, 128), (stride, 128, 1))
    rng = np.random.default_rng(6)
    rows = rng.standard_normal((3, 24, 128)).astype(np.float16)
    x.copy_(dev(rows, cuda_dev))
    angles = pkv.make_rope_angles(600, 128, device=cuda_dev)
    table = np.array([[n_blocks - 1, 0, n_blocks - 2]], np.int32)
    pos = np.array([0, 255, 599], np.int32)
    out = torch.empty((3, 8, 128), dtype=torch.float16, device=cuda_dev)
    pkv.pf_device_status(reset=True)
    pkv.pf_norm_rope_write(pool, 0, x[:, :8], x[:, 8:16], x[:, 16:], dev(table, cuda_dev), dev(np.zeros(3, np.int32), cuda_dev),
                           dev(pos, cuda_dev), angles, out)
    assert pkv.pf_device_status(reset=True) == 0
    assert_within(host(out), *rotated64(rows[:, :8], None, 0, host(angles), pos, False))
    for i, (blk, at) in enumerate(((n_blocks - 1, 0), (n_blocks - 1, 255), (n_blocks - 2, 87))):
        assert_within(host(k[0, blk, at])[None], *rotated64(rows[i:i + 1, 8:16], None, 0, host(angles), pos[i:i + 1], False))
        assert np.array_equal(host(v[0, blk, at]), rows[i, 16:])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 48])
def test_values_outside_the_rotated_part_stay_as_they_are(pkv, cuda_dev, d, interleaved, rot):
    """Without a norm bit for bit: every fp16 number, zeros of either sign, infinities and NaNs; with one a
    zero keeps its sign."""
    import torch
    T = 65536 // (d - rot) + 1
    r = Rows(pkv, cuda_dev, [T], [T], 2, 1, d, 16, norm=True, rot=rot)
    every = np.resize(np.arange(65536, dtype=np.uint16), T * (d - rot)).reshape(T, 1, d - rot)
    bits, kbits = r.q.view(np.uint16).copy(), r.k.view(np.uint16).copy()
    bits[..., rot:], kbits[..., rot:] = every, every
    q, k = (dev(x.view(np.float16), cuda_dev) for x in (bits, kbits))
    pkv.pf_norm_rope_write(r.c.pool, 1, q, k, r.vd, r.c.bt_dev, *r.ids, r.angles_dev, r.out[:-1], interleaved=interleaved)
    assert np.array_equal(host(r.out)[:-1, :, rot:].view(np.uint16), bits[..., rot:])
    blk, at = r.slots()
    assert np.array_equal(host(r.c.k_dev)[1, blk, at][..., rot:].view(np.uint16), kbits[..., rot:])
    zeros = np.zeros((T, 2, d), np.float16)
    zeros[:, 1] = -0.0
    zeros[..., 0] = 1
    pkv.pf_norm_rope_write(r.c.pool, 1, dev(zeros, cuda_dev), None, None, None, None, r.ids[1], r.angles_dev, r.out[:-1],
                           interleaved=interleaved, q_weight=torch.ones(d, device=cuda_dev))
    out = host(r.out)[:-1, :, max(rot, 1):]
    assert not out.any() and not np.signbit(out[:, 0]).any() and np.signbit(out[:, 1]).all()
