"""Measured cases of the rotated cache write, sliding-window attention and tree
attention.

Three operators, each in its plain form (torch, 32 bits) and as the calls of
this package (``own``):

* ``rope``    norms of queries and keys for each head, the position rotation
              and the write of K and V into their pages in one pass: for a row
              x of a q- or k-head y = x / sqrt(mean(x^2) + eps) * w (without a
              norm y = x); of its first `rot` dims the pairs (a, b) -- dims i
              and i + rot / 2, or 2 i and 2 i + 1 -- become (a c - b s, b c +
              a s) with c, s the cosine and sine of the token's position at
              pair i, from a table; rounded once.  V rows are copied.
* ``window``  causal attention of a sequence's last tokens, where the query at
              position p sees the tokens t <= p with t > p - window or t <
              sinks.  Pages that no query sees are not the sequence's any more.
* ``tree``    attention of drafted tokens, a sequence's last n, that form a
              tree: each sees all tokens before them and those drafts that its
              row of bits names (its ancestors and itself).

Scores are scale * q . K, outputs sum_t softmax(z)_t V_t; a query that sees
nothing gives zeros.  Pools are [layers][pages][page tokens][kv heads][head
dim], fp16 or e4m3 with a scale per page and kv-head; token t of a sequence is
row t % B of page table[t // B].
"""
import math

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
EPS = 1e-6


# ------------------------------------------------------------------- cases

def _case(name, op, **kw):
    c = dict(name=name, op=op, seqs=1, q_heads=12, kv_heads=12, head_dim=64, page=16, len_lo=1, len_hi=100, new_lo=1,
             new_hi=1)
    if op == "rope":
        c.update(norm=True, rot=64, interleaved=False, packed=False)
    else:
        c.update(cache="f16", out32=False)
    if op == "window":
        c.update(window=64, sinks=0)
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of the smallest serving batch: latency
        _case("rope_step_tiny", "rope", seqs=4),
        # one decode step of many sequences, grouped heads, half of each row rotated in neighbouring pairs, no norm
        _case("rope_step_grouped", "rope", seqs=256, q_heads=14, kv_heads=2, page=64, len_lo=32, len_hi=4096,
              norm=False, rot=32, interleaved=True),
        # ragged chunks of prompts, rows as the projection leaves them (q, k and v of a token side by side)
        _case("rope_chunks_packed", "rope", seqs=16, q_heads=32, kv_heads=8, head_dim=128, len_lo=512, len_hi=2048,
              new_lo=1, new_hi=512, rot=128, packed=True),
        # four whole prompts of a 40-head model
        _case("rope_prompts_40x128", "rope", seqs=4, q_heads=40, kv_heads=40, head_dim=128, len_lo=2048, len_hi=2048,
              new_lo=2048, new_hi=2048, rot=128),
        # the smallest serving batch with a short window: latency
        _case("window_step_tiny", "window", seqs=4, len_lo=1, len_hi=200, window=64, sinks=4),
        # a decode step of many long conversations, grouped heads
        _case("window_step_long", "window", seqs=128, q_heads=14, kv_heads=2, page=64, len_lo=32, len_hi=16384,
              window=1024, sinks=4),
        # a decode step of a 40-head model over the 8-bit cache, fp32 results
        _case("window_step_40x128_f32", "window", seqs=16, q_heads=40, kv_heads=40, head_dim=128, len_lo=4096,
              len_hi=8192, window=2048, sinks=64, cache="e4m3", out32=True),
        # whole prompts through a layer with a window, 32 q-heads over 8 kv-heads
        _case("window_prompts_32q8kv", "window", seqs=4, q_heads=32, kv_heads=8, head_dim=128, len_lo=4000,
              len_hi=4096, new_lo=4000, new_hi=4096, window=512, sinks=4),
        # a few drafts for the smallest serving batch: latency
        _case("tree_tiny", "tree", seqs=2, len_lo=8, len_hi=200, new_lo=4, new_hi=8),
        # a serving batch checks trees of up to 32 drafts, 32 q-heads over 8 kv-heads, 8-bit cache
        _case("tree_batch_e4m3", "tree", seqs=32, q_heads=32, kv_heads=8, head_dim=128, len_lo=256, len_hi=2048,
              new_lo=12, new_hi=32, cache="e4m3"),
        # few long conversations, 64 drafts each, grouped heads
        _case("tree_long_page64", "tree", seqs=4, q_heads=14, kv_heads=2, page=64, len_lo=8192, len_hi=16384,
              new_lo=60, new_hi=64),
        # wide trees for a 40-head model
        _case("tree_wide_40x128", "tree", seqs=8, q_heads=40, kv_heads=40, head_dim=128, len_lo=1024, len_hi=2048,
              new_lo=100, new_hi=200),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "window", "tree"))
    page = rng.choice((1, 16, 16, 64, 256))
    head_dim = rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 3, 4, 5, 8, 12, 14, 32, 40))
    group = rng.choice((1, 1, 2, 3, 4, 7, 8, 16))
    while group * kv_heads > 64:
        group = max(1, group // 2)
    q_heads = kv_heads * group
    c = _case("", op, kv_heads=kv_heads, q_heads=q_heads, head_dim=head_dim, page=page)
    del c["name"]
    row = kv_heads * head_dim
    if op == "rope":
        new_hi = _log(rng, 1, 2048)
        seqs = _log(rng, 1, max(1, min(256, 8192 * 120 * 128 // ((q_heads + 2 * kv_heads) * head_dim * new_hi))))
        len_hi = new_hi + _log(rng, 1, 4096)
        len_hi = max(new_hi, min(len_hi, 2 ** 28 // (row * seqs)))
        rot = rng.choice((head_dim, head_dim, head_dim // 2, 16, 0))
        c.update(seqs=seqs, new_lo=rng.randint(0, new_hi), new_hi=new_hi, len_lo=rng.randint(new_hi, len_hi),
                 len_hi=len_hi, norm=rot == 0 or rng.random() < 0.6, rot=rot, interleaved=rng.random() < 0.4,
                 packed=rng.random() < 0.4)
        return c
    c.update(cache=rng.choice(("f16", "e4m3")))
    if op == "window":
        window, sinks = _log(rng, 1, 4096), rng.choice((0, 1, 4, 64, 100))
        if rng.random() < 0.5:            # a decode step
            len_hi, new_hi = _log(rng, 1, 16384), 1
        else:                             # prompts, and chunks of them
            len_hi = _log(rng, 2, 4096)
            new_hi = _log(rng, 2, len_hi)
        seen = min(len_hi, window + sinks + new_hi)
        most = min(128, 4096 * 4096 * 4 * 32 * 128 // 8 // (min(len_hi, window + sinks) * new_hi * q_heads * head_dim),
                   2 ** 31 // (q_heads * new_hi * len_hi), 16 * 2048 * 40 * 128 // (row * seen), 2 ** 28 // (row * len_hi),
                   2 ** 26 // (q_heads * head_dim * new_hi))
        c.update(window=window, sinks=sinks)
    else:
        new_hi = _log(rng, 1, 200)
        len_hi = new_hi + _log(rng, 1, 16384)
        most = min(32, 8 * 200 * 2048 * 40 * 128 // (len_hi * new_hi * q_heads * head_dim),
                   2 ** 31 // (q_heads * new_hi * len_hi), 8 * 2048 * 40 * 128 // (row * len_hi))
        while most < 1 and len_hi > new_hi + 1:
            len_hi = max(new_hi + 1, len_hi // 2)
            most = min(8 * 200 * 2048 * 40 * 128 // (len_hi * new_hi * q_heads * head_dim),
                       8 * 2048 * 40 * 128 // (row * len_hi))
    while most < 1:                       # one sequence of the largest heads: shorter
        len_hi = max(2, len_hi // 2)
        new_hi = min(new_hi, len_hi)
        if len_hi == 2:
            most = 1
        else:
            most = min(4096 * 4096 * 4 * 32 * 128 // 8 // (len_hi * new_hi * q_heads * head_dim),
                       8 * 2048 * 40 * 128 // (row * len_hi))
    c.update(seqs=_log(rng, 1, most), len_lo=rng.randint(new_hi if new_hi > 1 or op == "tree" else 0, len_hi),
             len_hi=len_hi, new_hi=new_hi, new_lo=rng.randint(1, new_hi),
             out32=rng.random() < 0.4 and new_hi * group <= 16)     # (more rows: fp16 is what a next layer takes)
    return c


def _lengths(case):
    """Context lengths (the new tokens included) and new-token counts: part of the case, not of the seed."""
    S = case["seqs"]
    rng = np.random.default_rng(42)
    lens = rng.integers(case["len_lo"], case["len_hi"] + 1, S)
    new = np.minimum(rng.integers(case["new_lo"], case["new_hi"] + 1, S), lens)
    new[0] = max(new[0], min(1, lens[0]))     # a batch has some token
    return lens.astype(np.int64), new.astype(np.int64)


def _step(case):
    """A call without row offsets: one query per sequence."""
    return case["op"] == "window" and case["new_hi"] == 1


def _trees(case):
    """Per sequence the matrix of what a draft sees among the drafts: itself
    and its ancestors.  Parents lie close by, so that chains and forks mix."""
    rng = np.random.default_rng(5)
    out = []
    for n in _lengths(case)[1]:
        sees = np.zeros((n, n), bool)
        for i in range(n):
            parent = i - 1 - int(rng.integers(0, 4))
            if parent >= 0:
                sees[i] = sees[parent]
            sees[i, i] = True
        out.append(sees)
    return out


def _live_pages(case, lens, new):
    """Which pages of each sequence some query sees, [S][pages]."""
    B = case["page"]
    out = []
    for L, n in zip(lens, new):
        live = np.ones(-(-L // B), bool)
        if case["op"] == "window":
            first = max(0, L - n - case["window"] + 1) // B
            live[-(-min(case["sinks"], L) // B):first] = False
        out.append(live)
    return out


def _pairs(case, lens, new):
    """(query, token) pairs, and tokens that some query sees."""
    if case["op"] == "tree":
        drafts = sum(int(x.sum()) for x in _trees(case))
        return int((new * (lens - new)).sum()) + drafts, int(lens[new > 0].sum())
    W, K = case["window"], case["sinks"]
    pairs = tokens = 0
    for L, n in zip(lens.tolist(), new.tolist()):
        p = np.arange(L - n, L, dtype=np.int64)
        lo = np.maximum(0, p - W + 1)
        pairs += int((p + 1 - lo + np.minimum(K, lo)).sum())
        if n:
            tokens += L - int(lo[0]) + min(K, int(lo[0]))
    return pairs, tokens


def work(case):
    lens, new = _lengths(case)
    H, Hq, D = case["kv_heads"], case["q_heads"], case["head_dim"]
    if case["op"] == "rope":
        T = int(new.sum())
        rotated = T * (Hq + H)
        angles = min(T, int(lens.max())) * 4.0 * case["rot"]
        return {"bytes": 4.0 * T * (Hq + 2 * H) * D + angles + T * 12.0,
                "flops": rotated * (3.0 * case["rot"] + (4.0 * D if case["norm"] else 0.0))}
    pairs, tokens = _pairs(case, lens, new)
    pages = sum(int(x.sum()) for x, n in zip(_live_pages(case, lens, new), new) if n)
    elem = 2 if case["cache"] == "f16" else 1
    rows = int(new.sum()) if not _step(case) else case["seqs"]
    bits = int((new * -(-new // 8)).sum()) if case["op"] == "tree" else 0
    return {"bytes": 2.0 * tokens * H * D * elem + pages * (4 + (0 if elem == 2 else 8 * H)) + bits +
            rows * Hq * D * (2 + (4 if case["out32"] else 2)), "flops": 4.0 * pairs * Hq * D}


# ------------------------------------------------------------------ inputs

def _tables(live, n_pages, gen):
    """Shuffled frames: every live page of a sequence is one of a permutation; entries of the others hold anything."""
    order = torch.randperm(n_pages, generator=gen, device="cuda", dtype=torch.int32).cpu().numpy()
    width = max(1, max(x.size for x in live))
    table = np.zeros((len(live), width), np.int32)
    at = 0
    for row, x in zip(table, live):
        n = int(x.sum())
        row[:x.size][x] = order[at:at + n]
        at += n
    return torch.from_numpy(table).cuda()


def _fill(shape, cache, gen):
    """A K or V pool's content: fp16 N(0, 1), or e4m3 codes and scales of such values."""
    if cache == "f16":
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16), None
    codes = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16)
    codes = codes.mul_(64).clamp_(-448, 448).to(E4M3)
    exp = torch.randint(-8, -4, (shape[0], shape[1], shape[3]), generator=gen, device="cuda")
    return codes, torch.exp2(exp.float())


def _angles(positions, rot):
    """[positions, rot] fp32: cosines, then sines, of p * 10000^(-2 i / rot); the angles in 64 bits."""
    p = torch.arange(positions, device="cuda", dtype=torch.float64)
    f = 10000.0 ** (-2.0 * torch.arange(rot // 2, device="cuda", dtype=torch.float64) / rot)
    a = p[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens, new = _lengths(case)
    B, H, Hq, D = case["page"], case["kv_heads"], case["q_heads"], case["head_dim"]
    live = _live_pages(case, lens, new)
    n_pages = max(1, sum(int(x.sum()) for x in live)) + 3
    shape = (1, n_pages, B, H, D)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1]) if not _step(case) else case["seqs"]
    randn = lambda *size: torch.randn(size, generator=gen, device="cuda", dtype=torch.float16)   # noqa: E731
    s = {"case": case, "tables": _tables(live, n_pages, gen), "most": max(1, int(new.max()))}
    if case["op"] == "rope":
        if case["packed"]:
            qkv = randn(T, Hq + 2 * H, D)
            s["q"], s["k_new"], s["v_new"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        else:
            s["q"], s["k_new"], s["v_new"] = randn(T, Hq, D), randn(T, H, D), randn(T, H, D)
        for name in ("q_weight", "k_weight"):
            s[name] = 1.0 + 0.1 * torch.randn(D, generator=gen, device="cuda") if case["norm"] else None
        s["angles"] = _angles(int(lens.max()), case["rot"]) if case["rot"] else None
        s["seq"] = torch.from_numpy(np.repeat(np.arange(case["seqs"]), new).astype(np.int32)).cuda()
        pos = [np.arange(L - n, L) for L, n in zip(lens, new)]
        s["pos"] = torch.from_numpy(np.concatenate(pos).astype(np.int32)).cuda()
        s["q_out"] = torch.empty((T, Hq, D), device="cuda", dtype=torch.float16)
        s["k"] = torch.zeros(shape, device="cuda", dtype=torch.float16)
        s["v"] = torch.zeros(shape, device="cuda", dtype=torch.float16)
    else:
        s["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
        s["cu"] = None if _step(case) else torch.from_numpy(cu).cuda()
        s["q"] = randn(T, Hq, D)
        s["scale"] = 1.0 / math.sqrt(D)
        s["out"] = torch.empty((T, Hq, D), device="cuda", dtype=torch.float32 if case["out32"] else torch.float16)
        s["k"], s["ks"] = _fill(shape, case["cache"], gen)
        s["v"], s["vs"] = _fill(shape, case["cache"], gen)
        if case["op"] == "tree":
            # a row of 64-bit words per draft: bit j for draft j of its sequence
            words = -(-s["most"] // 64)
            bits = np.zeros((T, words * 64), np.uint8)
            for first, sees in zip(cu, _trees(case)):
                bits[first:first + len(sees), :len(sees)] = sees
            packed = np.packbits(bits, axis=1, bitorder="little").view("<i8")
            s["mask"] = torch.from_numpy(np.ascontiguousarray(packed)).cuda()
    if own:   # the handle and the workspace that a serving program keeps for its pool
        import paged_kv_cache_37_gb300 as pkv
        s["pkv"] = pkv
        s["pool"] = pkv.pf_pool_create(s["k"], s["v"], s.get("ks"), s.get("vs"))
        width = s["tables"].shape[1]
        if case["op"] == "window":
            s["ws"] = pkv.make_window_workspace(s["pool"], case["seqs"], Hq, width, s["most"], case["window"],
                                                case["sinks"])
        elif case["op"] == "tree":
            s["ws"] = pkv.make_tree_workspace(s["pool"], case["seqs"], Hq, width, s["most"])
    return s


# ------------------------------------------------------------- plain forms

def _rope_plain(s):
    case = s["case"]
    rot, B = case["rot"], case["page"]

    def turned(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
        if rot:
            cos, sin = s["angles"][s["pos"].long()][:, None].chunk(2, -1)
            if case["interleaved"]:
                a, b = x[..., 0:rot:2], x[..., 1:rot:2]
                turn = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
            else:
                a, b = x[..., :rot // 2], x[..., rot // 2:rot]
                turn = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
            x = torch.cat([turn, x[..., rot:]], -1)
        return x.half()

    pos = s["pos"].long()
    blk = s["tables"].long()[s["seq"].long(), pos // B]
    s["k"][0, blk, pos % B] = turned(s["k_new"], s["k_weight"])
    s["v"][0, blk, pos % B] = s["v_new"]
    return {"q": turned(s["q"], s["q_weight"]), "k": s["k"], "v": s["v"]}


def _values(s, name):
    """[S, T, H, D] fp32: every sequence's rows, padded to the table's width."""
    x = s[name][0][s["tables"].long()].float()                                         # [S, P, B, H, D]
    if s[name + "s"] is not None:
        x = x * s[name + "s"][0][s["tables"].long()][:, :, None, :, None]
    return x.flatten(1, 2)


def _seen(s, first, n, T):
    """[S, Q, T]: what each query sees."""
    case = s["case"]
    L = s["lens"].long()
    i = torch.arange(s["most"], device="cuda")
    t = torch.arange(T, device="cuda")
    if case["op"] == "window":
        p = ((L - n)[:, None] + i)[:, :, None]
        return (t <= p) & (t < L[:, None, None]) & ((t > p - case["window"]) | (t < case["sinks"]))
    row = (first[:, None] + i).clamp(max=max(0, s["q"].shape[0] - 1))
    bits = (s["mask"][row][..., None] >> torch.arange(64, device="cuda")) & 1          # [S, Q, words, 64]
    bits = bits.flatten(2).bool()
    draft = t - (L - n)[:, None]                                                       # [S, T]
    at = draft.clamp(0, bits.shape[2] - 1)[:, None].expand(-1, s["most"], -1)
    among = bits.gather(2, at) & ((draft >= 0) & (draft < n[:, None]))[:, None]
    return (draft < 0)[:, None] | among


def _attend_plain(s):
    case = s["case"]
    H, G, D = case["kv_heads"], case["q_heads"] // case["kv_heads"], case["head_dim"]
    S, Q = case["seqs"], s["most"]
    k, v = _values(s, "k"), _values(s, "v")
    T = k.shape[1]
    if s["cu"] is None:
        n = torch.ones_like(s["lens"]).long()
        first = torch.arange(S, device="cuda")
    else:
        n = (s["cu"][1:] - s["cu"][:-1]).long()
        first = s["cu"][:-1].long()
    i = torch.arange(Q, device="cuda")
    row = (first[:, None] + i).clamp(max=max(0, s["q"].shape[0] - 1))
    q = s["q"].float()[row].view(S, Q, H, G, D).permute(0, 2, 3, 1, 4).reshape(S, H, G * Q, D)
    z = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]                            # [S, H, G Q, T]
    seen = _seen(s, first, n, T)[:, None, None].expand(S, 1, G, Q, T).reshape(S, 1, G * Q, T)
    z = torch.where(seen, z, -math.inf)
    m = z.amax(-1, keepdim=True)
    w = torch.exp(z - torch.where(torch.isfinite(m), m, 0.0))
    del z
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1.0)
    o = o.view(S, H, G, Q, D).permute(0, 3, 1, 2, 4).reshape(S, Q, H * G, D)
    return o[i[None, :] < n[:, None]].to(s["out"].dtype)


# --------------------------------------------------------------------- run

def run(s):
    case = s["case"]
    if not own:
        return _rope_plain(s) if case["op"] == "rope" else _attend_plain(s)
    pkv = s["pkv"]
    if case["op"] == "rope":
        pkv.pf_norm_rope_write(s["pool"], 0, s["q"], s["k_new"], s["v_new"], s["tables"], s["seq"], s["pos"],
                               s["angles"], s["q_out"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                               interleaved=case["interleaved"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    if case["op"] == "window":
        pkv.pf_paged_window_attention(s["pool"], 0, s["q"], s["tables"], s["lens"], s["cu"], s["most"], s["scale"],
                                      case["window"], case["sinks"], s["out"], s["ws"])
    else:
        pkv.pf_paged_tree_attention(s["pool"], 0, s["q"], s["tables"], s["lens"], s["cu"], s["most"], s["scale"],
                                    s["mask"], s["out"], s["ws"])
    return s["out"]


# ------------------------------------------------------------------- exact

def _exact_rope(s):
    """Each pair of dims as a complex number, turned by the table's."""
    case, rot, B = s["case"], s["case"]["rot"], s["case"]["page"]

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()
        if not rot:
            return x
        table = s["angles"].double()[s["pos"].long()]
        unit = torch.complex(table[:, :rot // 2], table[:, rot // 2:])[:, None]
        head = x[..., :rot].reshape(*x.shape[:-1], *((rot // 2, 2) if case["interleaved"] else (2, rot // 2)))
        if not case["interleaved"]:
            head = head.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(head.contiguous()) * unit)
        if not case["interleaved"]:
            z = z.transpose(-1, -2)
        return torch.cat([z.reshape(*x.shape[:-1], rot), x[..., rot:]], -1)

    out = {"q": turned(s["q"], s["q_weight"]), "k": s["k"].double(), "v": s["v"].double()}
    k, v = turned(s["k_new"], s["k_weight"]), s["v_new"].double()
    where = s["tables"].flatten().long()[s["seq"].long() * s["tables"].shape[1] + s["pos"].long().div(B, rounding_mode="floor")]
    slot = where * B + s["pos"].long().remainder(B)
    out["k"].view(-1, *k.shape[1:]).index_copy_(0, slot, k)
    out["v"].view(-1, *v.shape[1:]).index_copy_(0, slot, v)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    lens, new = _lengths(case)
    if 4.0 * _pairs(case, lens, new)[0] * case["q_heads"] * case["head_dim"] > 4e11:
        return None
    B, G = case["page"], case["q_heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    trees = _trees(case) if case["op"] == "tree" else None
    row = 0
    for i, (L, n) in enumerate(zip(lens.tolist(), [1] * len(lens) if _step(case) else new.tolist())):
        for a in range(0, n, 512):                                                     # queries a .. b - 1
            b = min(n, a + 512)
            t = torch.arange(L, device="cuda")
            p = torch.arange(L - n + a, L - n + b, device="cuda")[:, None]
            if trees is None:
                t = t[(t < case["sinks"]) | (t > L - n + a - case["window"])]
                sees = (p >= t) & ((p - t < case["window"]) | (t < case["sinks"]))
            else:
                sees = torch.cat([torch.ones((b - a, L - n), dtype=torch.bool, device="cuda"),
                                  torch.from_numpy(trees[i][a:b]).cuda()], 1)
            if L == 0 or not t.numel():
                continue
            blk = s["tables"][i].long()[t // B]
            k, v = s["k"][0][blk, t % B].double(), s["v"][0][blk, t % B].double()      # [tokens, H, D]
            if s["ks"] is not None:
                k, v = k * s["ks"][0][blk].double()[..., None], v * s["vs"][0][blk].double()[..., None]
            for h in range(case["kv_heads"]):
                q = s["q"][row + a:row + b, h * G:(h + 1) * G].double()                # [b - a, G, D]
                z = ((q @ k[:, h].T) * s["scale"]).masked_fill(~sees[:, None], -math.inf)
                w = torch.softmax(z, -1).nan_to_num(0.0)                               # a row that sees nothing
                out[row + a:row + b, h * G:(h + 1) * G] = w @ v[:, h]
        row += n
    return out
