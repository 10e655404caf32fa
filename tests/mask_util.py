"""Plain 64-bit attention under a mask, with the error bound that follows from
the formats (attention64's, over what a query sees), and the masks of windows
and of trees of drafts."""
import numpy as np


def masked64(q, k, v, scale, seen, weight_step, out_step):
    """q [n, Hq, D], k, v [L, Hkv, D], seen [n, L]: fp64 outputs and tolerances.

    The bound is that of attention64 in e4m3_util (its derivation is there), and
    for weights that are stored as subnormal fp16, below 2^-14 of the largest:
    off by 2^-25 instead of 2^-11 relative, so 2^-25 |v| for each token seen."""
    n, Hq, D = q.shape
    L, Hkv, _ = k.shape
    G = Hq // Hkv
    q, k, v = q.astype(np.float64), k.astype(np.float64), v.astype(np.float64)
    out, tol = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    some = seen.any(1) if L else np.zeros(n, bool)
    if not some.any():
        return out, tol
    for hq in range(Hq):
        kh, vh = k[:, hq // G], np.where(seen.any(0)[:, None], v[:, hq // G], 0.0)
        z = np.where(seen, q[:, hq] @ np.where(seen.any(0)[:, None], kh, 0.0).T * scale, -np.inf)[some]
        size = np.where(seen, np.abs(q[:, hq]) @ np.abs(np.where(seen.any(0)[:, None], kh, 0.0)).T * scale, 0.0)[some]
        w = np.exp(z - z.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        out[some, hq] = w @ vh
        A = w @ np.abs(vh)
        zmax = np.where(np.isfinite(z), np.abs(z), 0.0).max(-1)
        e = size.max(-1) * (D + 4) * 2.0 ** -23 + (zmax + 16) * 2.0 ** -22
        tol[some, hq] = (A * (2 * e[:, None] + weight_step + (L / 16 + 4) * 2.0 ** -23) +
                         2.0 ** -25 * seen[some].astype(np.float64) @ np.abs(vh))
    return out, tol + np.where(some[:, None, None], np.abs(out) * out_step + 2.0 ** -25, 0.0)


def window_seen(L, n, window, sinks):
    """[n, L]: the last n of L tokens, each seeing `window` tokens up to its own and the first `sinks`."""
    p, t = np.arange(L - n, L)[:, None], np.arange(L)
    return (t <= p) & ((t > p - window) | (t < sinks))


def tree_seen(L, sees):
    """[n, L]: everything before the drafts, and of those what `sees` [n, n] says."""
    n = len(sees)
    return np.concatenate([np.ones((n, L - n), bool), sees], 1)


def random_tree(rng, n):
    """A draft's ancestors and itself; parents among the four drafts before, or none."""
    sees = np.zeros((n, n), bool)
    for i in range(n):
        parent = i - 1 - int(rng.integers(0, 4))
        if parent >= 0:
            sees[i] = sees[parent]
        sees[i, i] = True
    return sees


def pack(trees, words, rng=None):
    """int64 [sum of drafts, words]; with rng the bits past a sequence's drafts are random."""
    T = sum(len(x) for x in trees)
    bits = np.zeros((T, 64 * words), np.uint8)
    at = 0
    for x in trees:
        n = len(x)
        if rng is not None:
            bits[at:at + n, n:] = rng.integers(0, 2, (n, 64 * words - n))
        bits[at:at + n, :n] = x
        at += n
    return np.packbits(bits, axis=1, bitorder="little").view("<i8").reshape(T, words)
