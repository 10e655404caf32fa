"""Measured cases of the 8-bit cache, cross attention and page compaction.

Four operators, each in its plain form (torch, 32 bits) and as the calls of
this package (``own``):

* ``append``   new K/V rows quantised into e4m3 pages, one power-of-two scale
               per page and kv-head: for a page with the rows x,
               scale = max(old scale, 2^k), k the smallest integer >= -24 with
               max |x| <= 448 * 2^k, rows stored as e4m3(x / scale) (nearest
               even, magnitudes at most min(448, 61440 / scale)); when the
               scale grows, the page's earlier rows are rounded again to it.
* ``decode``   single-query attention over an e4m3 cache,
               z_t = scale * q . K_t, out = sum_t softmax(z)_t V_t, with
               K_t, V_t = code * scale of the page and kv-head.
* ``attend``   several query tokens per sequence: causal over an e4m3 cache
               (the sequence's last tokens), or cross attention (every query
               sees all of the context, whose length is its own) over an fp16
               or e4m3 cache.  An empty context gives zeros.
* ``compact``  live pages above the live count move into the holes below it,
               in every layer, and the block tables follow.

Pools are [layers][pages][page tokens][kv heads][head dim]; token t of a
sequence is row t % B of page table[t // B].
"""
import math

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases

def _attention(name, op, **kw):
    c = dict(name=name, op=op, seqs=1, q_heads=12, kv_heads=12, head_dim=64, page=16, lens="uniform", len_lo=1,
             len_hi=100, new_lo=1, new_hi=1, cache="e4m3", causal=False, out32=False)
    c.update(kw)
    return c


def listed():
    return [
        # one decode step's new tokens of a mixed batch, into partly filled pages
        _attention("append_step_mixed", "append", seqs=128, lens="mixed", len_hi=2048),
        # chunks of prompts of many sequences on 64-token pages, few kv-heads
        _attention("append_chunks_page64", "append", seqs=256, q_heads=14, kv_heads=2, page=64, len_lo=32,
                   len_hi=4096, new_lo=1, new_hi=64),
        # four whole prompts of a 40-head model
        _attention("append_prompts_40x128", "append", seqs=4, q_heads=40, kv_heads=40, head_dim=128, len_lo=2048,
                   len_hi=2048, new_lo=2048, new_hi=2048),
        # the smallest serving batch: latency
        _attention("decode_tiny", "decode", seqs=4, len_lo=1, len_hi=100),
        # the mixed serving batch: 50 % short, 30 % middle, 20 % long contexts
        _attention("decode_mixed", "decode", seqs=128, lens="mixed", len_hi=2048),
        # grouped heads (7 q-heads per kv-head), long ragged contexts, 64-token pages
        _attention("decode_grouped_page64", "decode", seqs=256, q_heads=14, kv_heads=2, page=64, len_lo=32,
                   len_hi=4096),
        # a 40-head model, 16 sequences of 2048 tokens, fp32 results
        _attention("decode_40x128_f32", "decode", seqs=16, q_heads=40, kv_heads=40, head_dim=128, len_lo=2048,
                   len_hi=2048, out32=True),
        # a decoder's few tokens per step against encoder states
        _attention("cross_few_tokens", "attend", seqs=32, len_lo=16, len_hi=512, new_lo=1, new_hi=4, cache="f16"),
        # whole decoder prompts against encoder states of another length
        _attention("cross_prompts", "attend", seqs=4, len_lo=1024, len_hi=2048, new_lo=1500, new_hi=2048,
                   cache="f16"),
        # causal prompts over the 8-bit cache, 32 q-heads over 8 kv-heads
        _attention("prompts_e4m3_32q8kv", "attend", seqs=4, q_heads=32, kv_heads=8, head_dim=128, len_lo=2048,
                   len_hi=2048, new_lo=2048, new_hi=2048, causal=True),
        # one small pool after churn: latency
        dict(name="compact_tiny", op="compact", layers=1, pages=64, page=16, kv_heads=12, head_dim=64, live=24,
             seqs=4, cache="e4m3"),
        # a 12-layer fp16 pool, a quarter of its pages live
        dict(name="compact_12_layers", op="compact", layers=12, pages=1024, page=16, kv_heads=12, head_dim=64,
             live=256, seqs=32, cache="f16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "decode", "attend", "compact"))
    page = rng.choice((1, 16, 16, 64, 256))
    head_dim = rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 3, 4, 5, 8, 12, 14, 32, 40))
    if op == "compact":
        layers = _log(rng, 1, 12)
        most = 150_000_000 // (layers * page * kv_heads * head_dim)
        if most < 16:
            layers, most = 1, 150_000_000 // (page * kv_heads * head_dim)
        pages = _log(rng, 16, min(2048, most))
        return dict(op=op, layers=layers, pages=pages, page=page, kv_heads=kv_heads, head_dim=head_dim,
                    live=max(1, int(pages * rng.uniform(0.1, 0.6))), seqs=_log(rng, 1, 64),
                    cache=rng.choice(("f16", "e4m3")))
    group = rng.choice((1, 1, 2, 3, 4, 7, 8, 16))
    while group * kv_heads > 64:
        group = max(1, group // 2)
    row = kv_heads * head_dim
    c = _attention("", op, kv_heads=kv_heads, q_heads=kv_heads * group, head_dim=head_dim, page=page)
    del c["name"]
    if op == "append":
        new_hi = _log(rng, 1, 2048)
        seqs = _log(rng, 1, max(1, min(256, 8192 * 40 * 128 // (row * new_hi))))
        len_hi = new_hi + _log(rng, 1, 2048)
        c.update(seqs=seqs, new_lo=rng.randint(0, new_hi), new_hi=new_hi, len_lo=rng.randint(new_hi, len_hi),
                 len_hi=len_hi)
        most = 268435456 // row     # tokens the pool holds
        c["len_hi"] = min(len_hi, max(new_hi, most // seqs))
        c["len_lo"] = min(c["len_lo"], c["len_hi"])
    elif op == "decode":
        len_hi = _log(rng, 1, 4096)
        seqs = _log(rng, 1, max(1, min(256, 16 * 2048 * 40 * 128 // (row * len_hi))))
        c.update(seqs=seqs, len_lo=rng.randint(0, len_hi), len_hi=len_hi, out32=rng.random() < 0.25)
    else:
        causal = rng.random() < 0.4
        len_hi = _log(rng, 1, 2048)
        new_hi = min(_log(rng, 1, 2048), len_hi) if causal else _log(rng, 1, 2048)
        cost = len_hi * new_hi * c["q_heads"] * head_dim
        seqs = _log(rng, 1, max(1, min(64, 2048 * 2048 * 32 * 128 * 2 // cost, 2 ** 26 // (row * len_hi),
                                       2 ** 26 // (c["q_heads"] * head_dim * new_hi))))
        c.update(seqs=seqs, causal=causal, cache="e4m3" if causal else rng.choice(("f16", "e4m3")), len_hi=len_hi,
                 len_lo=rng.randint(new_hi if causal else 0, len_hi), new_hi=new_hi,
                 new_lo=rng.randint(1, new_hi))
    return c


def _lengths(case):
    """Context lengths and new-token counts: part of the case, not of the seed."""
    S = case["seqs"]
    rng = np.random.default_rng(42)
    if case["lens"] == "mixed":
        bands = ((S // 2, 32, 128), (S * 3 // 10, 256, 512), (S - S // 2 - S * 3 // 10, 1024, 2048))
        lens = np.concatenate([rng.integers(lo, hi + 1, n) for n, lo, hi in bands])
        rng.shuffle(lens)
    else:
        lens = rng.integers(case["len_lo"], case["len_hi"] + 1, S)
    new = rng.integers(case["new_lo"], case["new_hi"] + 1, S)
    if case["op"] == "append" or case["causal"]:
        new = np.minimum(new, lens)
    return lens.astype(np.int64), new.astype(np.int64)


def work(case):
    if case["op"] == "compact":
        elem = 2 if case["cache"] == "f16" else 1
        block = 2 * case["layers"] * (case["page"] * case["kv_heads"] * case["head_dim"] * elem +
                                      (0 if elem == 2 else 4 * case["kv_heads"]))
        moves = _moves(case)[0].size
        return {"bytes": 2.0 * moves * block + 8.0 * moves, "flops": 0.0}
    lens, new = _lengths(case)
    H, Hq, D, B = case["kv_heads"], case["q_heads"], case["head_dim"], case["page"]
    elem = 2 if case["cache"] == "f16" else 1
    pages = int((-(-lens // B)).sum())
    if case["op"] == "append":
        T = int(new.sum())
        touched = int(np.where(new > 0, (lens - 1) // B - (lens - new) // B + 1, 0).sum())
        return {"bytes": 2.0 * T * H * D * 3 + touched * (2 * H * 4 + 4), "flops": 4.0 * T * H * D}
    # of a sequence without queries nothing has to be read
    seen = lens if case["op"] == "decode" else np.where(new > 0, lens, 0)
    cache = 2.0 * int(seen.sum()) * H * D * elem + pages * (4 + (0 if elem == 2 else 8 * H))
    if case["op"] == "decode":
        rows, pairs = case["seqs"], int(lens.sum())
    elif case["causal"]:
        rows, pairs = int(new.sum()), int((new * (lens - new) + new * (new + 1) // 2).sum())
    else:
        rows, pairs = int(new.sum()), int((new * lens).sum())
    return {"bytes": cache + rows * Hq * D * (2 + (4 if case["out32"] else 2)), "flops": 4.0 * pairs * Hq * D}


# ------------------------------------------------------------------ inputs

def _tables(lens, B, n_pages, gen):
    """Shuffled frames: every sequence owns pages(L) pages of a permutation."""
    need = -(-lens // B)
    width = max(1, int(need.max()))
    order = torch.randperm(n_pages, generator=gen, device="cuda", dtype=torch.int32)
    first = torch.from_numpy(np.concatenate([[0], np.cumsum(need)[:-1]])).cuda()
    j = torch.arange(width, device="cuda")
    used = j[None, :] < torch.from_numpy(need).cuda()[:, None]
    at = (first[:, None] + j[None, :]).clamp(max=n_pages - 1)
    return torch.where(used, order[at], torch.zeros_like(order[at])).contiguous()


def _fill(shape, cache, gen):
    """A K or V pool's content: fp16 N(0, 1), or e4m3 codes and scales of such values."""
    if cache == "f16":
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16), None
    codes = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16)
    codes = codes.mul_(64).clamp_(-448, 448).to(E4M3)
    exp = torch.randint(-8, -4, (shape[0], shape[1], shape[3]), generator=gen, device="cuda")
    return codes, torch.exp2(exp.float())


def _moves(case):
    """Which pages of a churned pool are live, and the moves that pack them."""
    rng = np.random.default_rng(7)
    live = np.sort(rng.permutation(case["pages"])[: case["live"]])
    n = live.size
    src = live[live >= n]
    dst = np.setdiff1d(np.arange(n), live)
    return src.astype(np.int32), dst.astype(np.int32), rng.permutation(live).astype(np.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "compact":
        src, dst, order = _moves(case)
        N, B = case["pages"], case["page"]
        shape = (case["layers"], N, B, case["kv_heads"], case["head_dim"])
        counts = np.full(case["seqs"], order.size // case["seqs"], np.int64)
        counts[: order.size % case["seqs"]] += 1
        lens = np.maximum(counts * B - (np.arange(case["seqs"]) % B), 0)
        width = max(1, int(counts.max()))
        table = np.zeros((case["seqs"], width), np.int32)
        for i, (at, n) in enumerate(zip(np.concatenate([[0], np.cumsum(counts)[:-1]]), counts)):
            table[i, :n] = order[at:at + n]
        block_map = np.arange(N, dtype=np.int32)
        block_map[src] = dst
        s.update(src=src, dst=dst, map=block_map, tables=table, lens=lens.astype(np.int32))
        s = {k: torch.from_numpy(v).cuda() if isinstance(v, np.ndarray) else v for k, v in s.items()}
    else:
        lens, new = _lengths(case)
        B, H, D = case["page"], case["kv_heads"], case["head_dim"]
        n_pages = max(1, int((-(-lens // B)).sum())) + 3
        shape = (1, n_pages, B, H, D)
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        s["tables"] = _tables(lens, B, n_pages, gen)
        s["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
        s["cu"] = torch.from_numpy(cu).cuda()
        s["most"] = max(1, int(new.max()))
        rows = case["seqs"] if case["op"] == "decode" else int(cu[-1])
        if case["op"] == "append":
            s["k_new"] = torch.randn((rows, H, D), generator=gen, device="cuda", dtype=torch.float16)
            s["v_new"] = torch.randn((rows, H, D), generator=gen, device="cuda", dtype=torch.float16)
        else:
            s["q"] = torch.randn((rows, case["q_heads"], D), generator=gen, device="cuda", dtype=torch.float16)
            s["scale"] = 1.0 / math.sqrt(D)
            s["out"] = torch.empty(s["q"].shape, device="cuda",
                                   dtype=torch.float32 if case["out32"] else torch.float16)
    s["k"], s["ks"] = _fill(shape, case["cache"], gen)
    s["v"], s["vs"] = _fill(shape, case["cache"], gen)
    if own:   # the handle and the workspace that a serving program keeps for its pool
        import paged_kv_cache_37_gb300 as pkv
        s["pkv"] = pkv
        s["pool"] = pkv.pf_pool_create(s["k"], s["v"], s["ks"], s["vs"])
        width = s["tables"].shape[1]
        if case["op"] == "decode":
            s["ws"] = pkv.make_workspace(s["pool"], case["seqs"], case["q_heads"], width, 0)
        elif case["op"] == "attend" and case["causal"]:
            s["ws"] = pkv.make_prefill_workspace(s["pool"], case["seqs"], case["q_heads"], width, s["most"])
        elif case["op"] == "attend":
            s["ws"] = pkv.make_cross_workspace(s["pool"], case["seqs"], case["q_heads"], width, s["most"])
    return s


# ------------------------------------------------------------- plain forms

def _pow2_scale(amax):
    """2^k, k the smallest integer >= -24 with amax <= 448 * 2^k."""
    _, e = torch.frexp(amax)
    k = e - 9                                     # 448 * 2^(e - 9) < 2^e
    k = k + (torch.ldexp(torch.full_like(amax, 448.0), k) < amax).to(k.dtype)
    return torch.exp2(k.clamp(min=-24).float())


def _append_plain(s, pool, scales, rows):
    case = s["case"]
    B, n_new = case["page"], s["most"]
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    L = s["lens"].long()
    start = L - n
    P = (n_new - 1) // B + 2                       # pages a sequence's new tokens touch, at most
    page = (start // B)[:, None] + torch.arange(P, device="cuda")
    live = (page * B < L[:, None]) & (n > 0)[:, None]
    at = s["tables"].long().gather(1, page.clamp(max=s["tables"].shape[1] - 1))[live]   # [M] physical pages
    t = page[:, :, None] * B + torch.arange(B, device="cuda")
    is_new = ((t >= start[:, None, None]) & (t < L[:, None, None]))[live][..., None, None]
    is_old = (t < start[:, None, None])[live][..., None, None]
    row = (s["cu"][:-1].long()[:, None, None] + t - start[:, None, None])[live].clamp(0, rows.shape[0] - 1)
    x = torch.where(is_new, rows[row].float(), 0.0)                                    # [M, B, H, D]
    old_scale = scales[0, at]                                                          # [M, H]
    has_old = (page * B < start[:, None])[live][:, None]
    scale = _pow2_scale(x.abs().amax(dim=(1, 3)))
    scale = torch.where(has_old, torch.maximum(scale, old_scale), scale)
    old = pool[0, at].float()
    lim = (61440.0 / scale).clamp(max=448.0)[:, None, :, None]
    again = old * (old_scale / scale)[:, None, :, None]
    value = torch.where(is_new, torch.clamp(x / scale[:, None, :, None], -lim, lim), torch.where(is_old, again, old))
    pool[0, at] = value.to(E4M3)
    scales[0, at] = scale


def _values(s, name):
    """[S, T, H, D] fp32: every sequence's rows, padded to the table's width."""
    x = s[name][0][s["tables"].long()].float()                                         # [S, P, B, H, D]
    if s[name + "s"] is not None:
        x = x * s[name + "s"][0][s["tables"].long()][:, :, None, :, None]
    return x.flatten(1, 2)


def _attend_plain(s):
    case = s["case"]
    H, G, D = case["kv_heads"], case["q_heads"] // case["kv_heads"], case["head_dim"]
    S, Q = case["seqs"], s["most"]
    k, v = _values(s, "k"), _values(s, "v")
    L = s["lens"].long()
    if case["op"] == "decode":
        n = torch.ones_like(L)
        first = torch.arange(S, device="cuda")
    else:
        n = (s["cu"][1:] - s["cu"][:-1]).long()
        first = s["cu"][:-1].long()
    i = torch.arange(Q, device="cuda")
    row = (first[:, None] + i).clamp(max=max(0, s["q"].shape[0] - 1))
    q = s["q"].float()[row].view(S, Q, H, G, D).permute(0, 2, 3, 1, 4).reshape(S, H, G * Q, D)
    z = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]                            # [S, H, G Q, T]
    t = torch.arange(k.shape[1], device="cuda")
    last = (L - n)[:, None] + i if case["causal"] else (L - 1)[:, None].expand(S, Q)
    seen = (t <= last[:, :, None]) & (t < L[:, None, None])                            # [S, Q, T]
    seen = seen[:, None, None].expand(S, 1, G, Q, -1).reshape(S, 1, G * Q, -1)
    z = torch.where(seen, z, -math.inf)
    m = z.amax(-1, keepdim=True)
    w = torch.exp(z - torch.where(torch.isfinite(m), m, 0.0))
    del z
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1.0)
    o = o.view(S, H, G, Q, D).permute(0, 3, 1, 2, 4).reshape(S, Q, H * G, D)
    return o[i[None, :] < n[:, None]].to(s["out"].dtype)


def _compact_plain(s):
    src, dst = s["src"].long(), s["dst"].long()
    for name in ("k", "ks", "v", "vs"):
        x = s[name]
        if x is not None:
            x = x.view(torch.uint8) if x.dtype == E4M3 else x
            x[:, dst] = x[:, src]
    B, width = s["case"]["page"], s["tables"].shape[1]
    used = torch.arange(width, device="cuda") * B < s["lens"][:, None]
    s["tables"].copy_(torch.where(used, s["map"][s["tables"].long()], s["tables"]))


# --------------------------------------------------------------------- run

def run(s):
    case = s["case"]
    if case["op"] == "append":
        if own:
            s["pkv"].pf_append_kv(s["pool"], 0, s["k_new"], s["v_new"], s["tables"], s["lens"], s["cu"], s["most"])
        else:
            _append_plain(s, s["k"], s["ks"], s["k_new"])
            _append_plain(s, s["v"], s["vs"], s["v_new"])
    elif case["op"] == "compact":
        if own:
            s["pkv"].pf_compact_blocks(s["pool"], s["src"], s["dst"], s["map"], s["tables"], s["lens"])
        else:
            _compact_plain(s)
        return {"k": s["k"], "v": s["v"], "tables": s["tables"]} if s["ks"] is None else {
            "k": s["k"], "v": s["v"], "ks": s["ks"], "vs": s["vs"], "tables": s["tables"]}
    elif own and case["op"] == "decode":
        s["pkv"].pf_paged_decode_attention(s["pool"], 0, s["q"], s["tables"], s["lens"], s["scale"], s["out"], 0,
                                           s["ws"])
    elif own:
        call = s["pkv"].pf_paged_prefill_attention if case["causal"] else s["pkv"].pf_paged_cross_attention
        call(s["pool"], 0, s["q"], s["tables"], s["lens"], s["cu"], s["most"], s["scale"], s["out"], s["ws"])
    else:
        return _attend_plain(s)
    if case["op"] == "append":   # the pools' values, in units of their scales
        return {"k": s["k"], "v": s["v"], "ks": s["ks"], "vs": s["vs"]}
    return s["out"]


# ------------------------------------------------------------------- exact

def _round_e4m3(y):
    """Nearest e4m3 value of each fp64 entry (ties to even), by its grid."""
    _, e = np.frexp(np.abs(y))
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.rint(y / step) * step


def _exact_append(s, pool, scales, rows):
    case = s["case"]
    B = case["page"]
    x64 = rows.cpu().numpy().astype(np.float64)
    pool64 = pool[0].float().cpu().numpy().astype(np.float64)
    sc = scales[0].cpu().numpy().astype(np.float64)
    cu, lens, tables = s["cu"].tolist(), s["lens"].tolist(), s["tables"].tolist()
    for i, L in enumerate(lens):
        start = L - (cu[i + 1] - cu[i])
        for j in range(start // B, -(-L // B) if L > start else 0):
            blk, lo, hi = tables[i][j], max(start, j * B), min(L, (j + 1) * B)
            x = x64[cu[i] + lo - start: cu[i] + hi - start]                            # [n, H, D]
            amax = np.abs(x).max(axis=(0, 2))
            with np.errstate(divide="ignore"):
                k = np.ceil(np.log2(amax / 448.0))
            new = np.exp2(np.maximum(k, -24.0))
            if lo > j * B:
                new = np.maximum(new, sc[blk])
                pool64[blk, : lo - j * B] = _round_e4m3(pool64[blk, : lo - j * B] * (sc[blk] / new)[None, :, None])
            lim = np.minimum(448.0, 61440.0 / new)[None, :, None]
            pool64[blk, lo - j * B: hi - j * B] = _round_e4m3(np.clip(x / new[None, :, None], -lim, lim))
            sc[blk] = new
    return pool64[None], sc[None]


def exact(case, seed):
    if work(case)["flops"] > 4e11 or case["op"] == "compact":
        return None
    if case["op"] == "append" and _lengths(case)[0].sum() * case["kv_heads"] * case["head_dim"] > 1e8:
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        k, ks = _exact_append(s, s["k"], s["ks"], s["k_new"])
        v, vs = _exact_append(s, s["v"], s["vs"], s["v_new"])
        return {"k": k, "v": v, "ks": ks, "vs": vs}
    B, G = case["page"], case["q_heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    cu = s["cu"].tolist()
    for i, L in enumerate(s["lens"].tolist()):
        first, n = (i, 1) if case["op"] == "decode" else (cu[i], cu[i + 1] - cu[i])
        if L == 0 or n == 0:
            continue
        t = torch.arange(L, device="cuda")
        blk = s["tables"][i].long()[t // B]
        k, v = s["k"][0][blk, t % B].double(), s["v"][0][blk, t % B].double()          # [L, H, D]
        if s["ks"] is not None:
            k, v = k * s["ks"][0][blk].double()[..., None], v * s["vs"][0][blk].double()[..., None]
        for h in range(case["kv_heads"]):
            q = s["q"][first:first + n, h * G:(h + 1) * G].double()                    # [n, G, D]
            z = (q @ k[:, h].T) * s["scale"]
            if case["causal"]:
                z = z.masked_fill(t > (L - n + torch.arange(n, device="cuda"))[:, None, None], -math.inf)
            out[first:first + n, h * G:(h + 1) * G] = torch.softmax(z, -1) @ v[:, h]
    return out
