"""Plain 64-bit forms of the 8-bit pool's operators, for its tests: the
quantising append on fp64 values, attention over dequantised rows, and the
error bound that follows from the formats alone."""
import numpy as np


def decode_table():
    """The 256 e4m3 values: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    out = np.zeros(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = (m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        out[c] = -v if s else v
        if e == 15 and m == 7:
            out[c] = np.nan
    return out


TABLE = decode_table()


def round_e4m3(y):
    """Nearest e4m3 value (ties to even) of fp64 y, |y| <= 448, on its grid."""
    _, e = np.frexp(np.abs(y))
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.rint(y / step) * step


def scale_for(amax):
    """2^k, k the smallest integer >= -24 with amax <= 448 * 2^k."""
    k = -24
    while amax > 448.0 * 2.0 ** k:
        k += 1
    return 2.0 ** k


class Model:
    """One layer of an 8-bit pool in fp64: values in units of the scale, and scales."""

    def __init__(self, n_blocks, block_size, heads, dim):
        self.B = block_size
        self.code = np.full((n_blocks, block_size, heads, dim), np.nan)   # NaN: never written
        self.scale = np.full((n_blocks, heads), np.nan)

    def append(self, rows, table, lens, cu):
        """rows fp16 [T, H, D]: sequence s's last cu[s+1]-cu[s] tokens."""
        B = self.B
        for s, L in enumerate(lens):
            n = int(cu[s + 1] - cu[s])
            start = int(L) - n
            for j in range(start // B, -(-int(L) // B)) if n else ():
                lo, hi = max(start - j * B, 0), min(int(L) - j * B, B)
                blk = table[s][j]
                x = rows[cu[s] + j * B + lo - start:cu[s] + j * B + hi - start].astype(np.float64)
                for h in range(x.shape[1]):
                    xh = x[:, h]
                    fin = np.abs(xh[np.isfinite(xh)])
                    new = scale_for(fin.max() if fin.size else 0.0)
                    if lo:
                        old = self.scale[blk, h]
                        new = max(new, old)
                        self.code[blk, :lo, h] = round_e4m3(self.code[blk, :lo, h] * (old / new))
                    lim = min(448.0, 61440.0 / new)
                    xh = np.where(np.isnan(xh), 0.0, xh)
                    self.code[blk, lo:hi, h] = round_e4m3(np.clip(xh / new, -lim, lim))
                    self.scale[blk, h] = new

    def rows(self, table_row, L):
        """Dequantised fp64 rows of a sequence, [L, H, D]."""
        t = np.arange(int(L))
        blk = np.asarray(table_row)[t // self.B]
        return self.code[blk, t % self.B] * self.scale[blk][:, :, None]


def attention64(q, k, v, scale, causal, weight_step, out_step):
    """fp64 attention of one sequence, and how far a computation may be off.

    q [n, Hq, D], k, v [L, Hkv, D].  The bound: with z the scores,
    * a score is a sum of D products in fp32 (each partial sum may lose
      2^-23 of its size, truncation included) times the scale: its error is at
      most e_z = scale * sum |q k| * (D + 4) * 2^-23, and 2^-22 |z| more for
      the log2 factor and exp2's argument, and 2^-22 for exp2 itself;
    * weights of that relative error e change the mean by at most 2 e times
      A = sum w |V|; each weight is rounded once more for the product, off by
      weight_step relative, and the product and row sums in fp32 add
      (L / 16 + 4) * 2^-23 of A;
    * the result is rounded once: out_step relative (half a step of its type),
      or half of fp16's smallest subnormal."""
    n, Hq, D = q.shape
    L, Hkv, _ = k.shape
    G = Hq // Hkv
    q, k, v = q.astype(np.float64), k.astype(np.float64), v.astype(np.float64)
    out, tol = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    if L == 0:
        return out, tol
    for hq in range(Hq):
        kh, vh = k[:, hq // G], v[:, hq // G]
        z = q[:, hq] @ kh.T * scale
        size = np.abs(q[:, hq]) @ np.abs(kh).T * scale
        if causal:
            seen = np.arange(L)[None, :] <= (L - n + np.arange(n))[:, None]
            z = np.where(seen, z, -np.inf)
            size = np.where(seen, size, 0.0)
        w = np.exp(z - z.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        out[:, hq] = w @ vh
        A = w @ np.abs(vh)
        zmax = np.where(np.isfinite(z), np.abs(z), 0.0).max(-1)
        e = size.max(-1) * (D + 4) * 2.0 ** -23 + (zmax + 16) * 2.0 ** -22
        tol[:, hq] = A * (2 * e[:, None] + weight_step + (L / 16 + 4) * 2.0 ** -23)
    return out, tol + np.abs(out) * out_step + 2.0 ** -25


def assert_within(got, want, tol, what=""):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == want.shape, (got.shape, want.shape)
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    if not want.size:
        return
    over = np.abs(got - want) - tol
    at = np.unravel_index(over.argmax(), over.shape)
    assert over.max() <= 0, f"{what}: off by {abs(got[at] - want[at]):.3e}, allowed {tol[at]:.3e}, at {at}"
