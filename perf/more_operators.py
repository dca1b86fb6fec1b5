"""The operators around a paged cache of keys and values, as cases to measure:
rotary positions with several axes (and their gradient), the append that rotates
new tokens straight into the cache, attention of new tokens over the cache, and
the copies that fork sequences and compact the cache.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, angles in 64, rounded once at the end) or, where ``own`` is true, through
this framework's entry points. ``exact`` computes the same outputs in 64 bits
from the definitions.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---- cases -----------------------------------------------------------------
#
# axes / axes_bwd: q [tokens, q_heads, dim] and k [tokens, kv_heads, dim], thirds of
#   one projection where kv_heads is q_heads and fused is true. Pair j of a head
#   turns by positions[axis(j)][token] * freqs[j]; sections says how many pairs
#   each axis has. pairs: "interleaved" (2j, 2j + 1) or "halves" (j, j + pairs).
#   frac: positions with fractions (float32), else whole numbers (int64).
# append: q, k, v of new tokens; q rotated, k rotated into its cache, v copied into its.
# attention: new tokens of several sequences over their pages.
#   A batch is described by seqs and the ranges of new tokens and lengths
#   (the length includes the new tokens); every third sequence has one new token
#   where mixed is true. pad: rows behind the last sequence.
# fork: children that share their parents' full pages and copy the last one.
# compact: used pages move to the front; moved is how many have to.


def _axes(name, op, tokens, q_heads, kv_heads, dim, sections, dtype, pairs, frac=False, fused=False, far=1024):
    c = {"op": op, "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
         "s0": sections[0], "s1": sections[1], "s2": sections[2], "dtype": dtype, "pairs": pairs,
         "frac": frac, "fused": fused, "far": far}
    return dict(c, name=name) if name else c


def _batch(name, op, seqs, new, lens, q_heads, kv_heads, dim, page, dtype, mixed=False, window=0, causal=True,
           pad=0, sections=(0, 0, 0), pairs="halves"):
    c = {"op": op, "seqs": seqs, "new_lo": new[0], "new_hi": new[1], "len_lo": lens[0], "len_hi": lens[1],
         "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "mixed": mixed,
         "window": window, "causal": causal, "pad": pad, "s0": sections[0], "s1": sections[1], "s2": sections[2],
         "pairs": pairs}
    return dict(c, name=name) if name else c


def _pages(name, op, seqs, lens, planes, kv_heads, dim, page, dtype, forks=0, spare=0.5):
    c = {"op": op, "seqs": seqs, "len_lo": lens[0], "len_hi": lens[1], "planes": planes, "kv_heads": kv_heads,
         "dim": dim, "page": page, "dtype": dtype, "forks": forks, "spare": spare}
    return dict(c, name=name) if name else c


def listed():
    return [
        # video tokens of 16 x 64 x 64, q and k as they lie in the fused projection, one call per block
        _axes("axes_video", "axes", 65536, 16, 16, 128, (16, 24, 24), "bf16", "interleaved", fused=True),
        # training on a packed batch of pictures and text of odd length: the gradient
        _axes("axes_packed_bwd", "axes_bwd", 1531, 8, 4, 256, (32, 48, 48), "f16", "halves", frac=True),
        # a long prompt enters the cache
        _batch("append_prompt", "append", 3, (1200, 3001), (2000, 9000), 8, 4, 256, 16, "bf16", sections=(128, 0, 0)),
        # a decoding step of a text and picture model: one token of each sequence enters the cache
        _batch("append_tokens", "append", 48, (1, 1), (20, 6000), 16, 2, 128, 64, "f16", pad=16, sections=(16, 24, 24)),
        # one sequence decoding: latency
        _batch("attention_token", "attention", 1, (1, 1), (8191, 8191), 8, 4, 256, 16, "bf16"),
        # many sequences decoding
        _batch("attention_tokens", "attention", 64, (1, 1), (100, 16000), 32, 8, 128, 16, "f16"),
        # a whole prompt of a text encoder
        _batch("attention_prompt", "attention", 1, (8192, 8192), (8192, 8192), 8, 4, 256, 64, "bf16"),
        # a serving step: ragged chunks of new prompts beside decoding sequences
        _batch("attention_chunks", "attention", 13, (130, 1999), (700, 24000), 16, 2, 128, 32, "f16", mixed=True, pad=5),
        # a few samples branch off one prompt
        _pages("fork_few", "fork", 9, (33, 700), 4, 4, 128, 16, "bf16", forks=4),
        # a beam search step over many layers
        _pages("fork_beams", "fork", 64, (100, 900), 52, 4, 256, 16, "bf16", forks=64, spare=0.1),
        # a small cache tidied up
        _pages("compact_small", "compact", 12, (10, 900), 4, 4, 128, 16, "f16"),
        # a large one, after many sequences have ended
        _pages("compact_large", "compact", 96, (300, 2400), 8, 4, 128, 16, "bf16", spare=0.6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _sections(rng, pairs):
    a = rng.choice((pairs // 4, rng.randint(1, max(1, pairs - 2)), pairs))
    b = rng.choice(((pairs - a) // 2, rng.randint(0, pairs - a)))
    return (a, b, pairs - a - b)


def draw(rng):
    kind = rng.choice(("axes", "append", "attention", "attention", "attention", "fork", "compact"))
    dtype = rng.choice(("bf16", "f16"))
    if kind == "axes":
        heads = rng.choice((4, 8, 16, 24))
        dim = rng.choice((48, 64, 80, 128, 128, 256))
        kv = rng.choice((heads, heads // 2, heads // 4, 1))
        tokens = max(1, min(_log(rng, 1, 65536), 65536 * 32 * 128 // ((heads + kv) * dim)))
        pairs = dim // 2 if rng.random() < 0.7 else dim // 4
        return _axes(None, rng.choice(("axes", "axes_bwd")), tokens, heads, kv, dim, _sections(rng, pairs),
                     rng.choice(("bf16", "f16", "f32")), rng.choice(("interleaved", "halves")),
                     rng.random() < 0.4, heads == kv and rng.random() < 0.6, rng.choice((64, 1024, 1 << 20)))
    if kind in ("fork", "compact"):
        seqs, planes = _log(rng, 2, 128), rng.choice((2, 4, 8, 52))
        longest = max(20, min(_log(rng, 20, 2000), 2000000 // (seqs * planes)))
        return _pages(None, kind, seqs, (rng.randint(1, longest), longest), planes, rng.choice((1, 2, 4)),
                      rng.choice((64, 80, 128)), rng.choice((8, 16, 16, 24, 64)), dtype,
                      rng.randint(1, max(1, seqs // 2)) if kind == "fork" else 0, rng.choice((0.1, 0.5, 1.0)))
    group = rng.choice((1, 2, 4, 6, 8, 16))
    kv = rng.choice((1, 2, 4, 8))
    dim = rng.choice((64, 80, 128, 128, 128, 256))
    page = rng.choice((5, 8, 16, 16, 24, 32, 64, 128))
    seqs = _log(rng, 1, 64)
    mixed = rng.random() < 0.3
    new_hi = 1 if rng.random() < 0.4 else _log(rng, 2, 4096)
    longest = max(new_hi, _log(rng, 16, 32768))
    if kind == "append":
        new_hi = max(1, min(new_hi, 9000 // seqs))
        longest = max(new_hi, min(longest, 200000 // seqs))
    else:   # no more work than the largest listed case
        budget = 1 << 38
        while 4 * seqs * new_hi * longest * group * kv * dim > budget or seqs * longest * kv * dim > 1 << 29:
            if seqs > 1:
                seqs = max(1, seqs // 2)
            else:
                longest = max(longest // 2, new_hi // 2, 1)
                new_hi = min(new_hi, longest)
    pairs = dim // 2
    return _batch(None, kind, seqs, (rng.randint(1, new_hi), new_hi), (rng.randint(new_hi, longest), longest),
                  group * kv, kv, dim, page, dtype, mixed, rng.choice((0, 0, rng.randint(1, 2048))),
                  rng.random() < 0.85, rng.choice((0, 0, rng.randint(1, 40))),
                  _sections(rng, pairs) if rng.random() < 0.5 else (pairs, 0, 0), rng.choice(("halves", "interleaved")))


def _spread(i, lo, hi):
    """The i-th of a row of sizes spread over lo .. hi."""
    return lo + (i * 2654435761 + 12345) % (1 << 32) * (hi - lo + 1) // (1 << 32)


def _sizes(case):
    """(new tokens, length) of every sequence."""
    out = []
    for i in range(case["seqs"]):
        n = _spread(i, case["new_lo"], case["new_hi"])
        if case["mixed"] and i % 3 == 2:
            n = 1
        out.append((n, max(n, _spread(i + 7, case["len_lo"], case["len_hi"]))))
    return out


def _lengths(case):
    return [_spread(i, case["len_lo"], case["len_hi"]) for i in range(case["seqs"])]


def _up(a, b):
    return -(-a // b)


# ---- inputs ----------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(DTYPES[dtype])


def _int(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _freqs(case):
    """A frequency for every pair: each axis starts anew at 1."""
    per = [case["s0"], case["s1"], case["s2"]]
    return torch.tensor([10000.0 ** (-j / n) for n in per for j in range(n)], dtype=torch.float32, device="cuda")


def _prepare_axes(case, g):
    T, H, K, D, t = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"], case["dtype"]
    if case["fused"]:
        qkv = _normal(g, (T, 3, H, D), t)
        q, k = qkv[:, 0], qkv[:, 1]
    else:
        q, k = _normal(g, (T, H, D), t), _normal(g, (T, K, D), t)
    far = case["far"]
    if case["frac"]:
        pos = torch.rand((3, T), generator=g, device="cuda") * far
    else:
        pos = torch.randint(0, far, (3, T), generator=g, device="cuda", dtype=torch.int64)
    return {"q": q, "k": k, "positions": pos, "freqs": _freqs(case),
            "sections": [case["s0"], case["s1"], case["s2"]]}


def _prepare_batch(case, g):
    sizes = _sizes(case)
    P, K, D, H, t = case["page"], case["kv_heads"], case["dim"], case["q_heads"], case["dtype"]
    held = [_up(n, P) for _, n in sizes]
    pages = sum(held) + sum(held) // 10 + 1
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(sizes), max(held) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(held):
        table[i, :n] = order[at:at + n]
        at += n
    cache = _normal(g, (2, pages, P, K, D), t)
    starts = [0]
    for n, _ in sizes:
        starts.append(starts[-1] + n)
    tokens = starts[-1] + case["pad"]
    qkv = _normal(g, (tokens, H + 2 * K, D), t)   # one fused projection
    s = {"sizes": sizes, "starts": starts, "tokens": tokens, "table": table, "k_cache": cache[0], "v_cache": cache[1],
         "lens": _int([n for _, n in sizes]), "q_starts": _int(starts), "q": qkv[:, :H],
         "most_new": max(n for n, _ in sizes)}
    if case["op"] == "append":
        s["k"], s["v"] = qkv[:, H:H + K], qkv[:, H + K:]
        s["freqs"], s["sections"] = _freqs(case), [case["s0"], case["s1"], case["s2"]]
        s["positions"] = None
        if case["s1"] or case["s2"]:   # pictures among the text: each axis has positions of its own
            s["positions"] = torch.randint(0, 8192, (3, tokens), generator=g, device="cuda", dtype=torch.int64)
        s["q_out"] = torch.zeros((tokens, H, D), dtype=DTYPES[t], device="cuda")
    else:
        s["out"] = torch.zeros((tokens, H, D), dtype=DTYPES[t], device="cuda")
    return s


def _moves(case):
    """(used pages, all pages, pages that have to move) of a compaction."""
    used = sum(_up(n, case["page"]) for n in _lengths(case))
    pages = used + int(used * case["spare"]) + 1
    return used, pages, min(used, pages - used, used * (pages - used) // pages)


def _prepare_pages(case, g):
    lens, P, t = _lengths(case), case["page"], case["dtype"]
    held = [_up(n, P) for n in lens]
    used, pages, moved = _moves(case)
    if case["op"] == "fork":
        pages += case["forks"]
        order = torch.randperm(pages, generator=g, device="cuda")
    else:   # `moved` holes among the first `used` pages, as many used ones behind them
        low = torch.randperm(used, generator=g, device="cuda")
        high = used + torch.randperm(pages - used, generator=g, device="cuda")
        order = torch.cat((low[moved:], high[:moved]))
        order = order[torch.randperm(used, generator=g, device="cuda")]
    order = order.to(torch.int32)
    rows = len(lens) + case["forks"]
    table = torch.full((rows, max(held) + 2), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(held):
        table[i, :n] = order[at:at + n]
        at += n
    s = {"cache": _normal(g, (case["planes"], pages, P, case["kv_heads"], case["dim"]), t), "table": table,
         "lengths": lens, "lens": _int(lens + [0] * case["forks"])}
    if case["op"] == "fork":
        s["parents_list"] = [i * 7 % len(lens) for i in range(case["forks"])]
        s["parents"] = _int(s["parents_list"])
        s["children"] = _int([len(lens) + i for i in range(case["forks"])])
        s["new_pages"] = order[used:used + case["forks"]].clone()
    return s


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] in ("axes", "axes_bwd"):
        s = _prepare_axes(case, g)
    elif case["op"] in ("append", "attention"):
        s = _prepare_batch(case, g)
    else:
        s = _prepare_pages(case, g)
    return dict(s, case=case)


# ---- plain forms -----------------------------------------------------------


def _plain_angles(positions, freqs, sections):
    """cos and sin [tokens, 1, pairs] in 32 bits, from angles in 64."""
    axis = torch.repeat_interleave(torch.arange(3), torch.tensor(sections)).to(freqs.device)
    angle = positions.double()[axis].T * freqs.double()
    return torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)


def _plain_rotate(x, cos, sin, pairs):
    n = 2 * cos.shape[-1]
    y = x.float()
    turned, rest = y[..., :n], y[..., n:]
    if pairs == "interleaved":
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = turned[..., :n // 2], turned[..., n // 2:]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, rest), -1).to(x.dtype)


def _plain_axes(s):
    cos, sin = _plain_angles(s["positions"], s["freqs"], s["sections"])
    if s["case"]["op"] == "axes_bwd":
        sin = -sin
    p = s["case"]["pairs"]
    return {"q": _plain_rotate(s["q"], cos, sin, p), "k": _plain_rotate(s["k"], cos, sin, p)}


def _token_places(s):
    """(sequence, place in it) of every token of the sequences."""
    lens, starts = s["lens"].long(), s["q_starts"].long()
    i = torch.arange(s["starts"][-1], device=starts.device)
    seq = torch.searchsorted(starts, i, right=True) - 1
    return seq, lens[seq] - (starts[seq + 1] - starts[seq]) + i - starts[seq]


def _plain_append(s):
    P, n = s["case"]["page"], s["starts"][-1]
    seq, place = _token_places(s)
    page = s["table"].long()[seq, place // P]
    pos = place.expand(3, -1) if s["positions"] is None else s["positions"][:, :n]
    cos, sin = _plain_angles(pos, s["freqs"], s["sections"])
    s["q_out"][:n] = _plain_rotate(s["q"][:n], cos, sin, s["case"]["pairs"])
    s["k_cache"][page, place % P] = _plain_rotate(s["k"][:n], cos, sin, s["case"]["pairs"])
    s["v_cache"][page, place % P] = s["v"][:n]
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attention(s):
    c = s["case"]
    P, K, D = c["page"], c["kv_heads"], c["dim"]
    G = c["q_heads"] // K
    out = s["out"]
    for i, (n, L) in enumerate(s["sizes"]):
        lo = s["starts"][i]
        first = max(0, L - n - c["window"] + 1) if c["window"] else 0   # the first key that anyone sees
        pages = s["table"][i, first // P:_up(L, P)].long()
        skip = first // P * P
        keys = s["k_cache"][pages].flatten(0, 1)[:L - skip].float()
        vals = s["v_cache"][pages].flatten(0, 1)[:L - skip].float()
        mask = None
        if n > 1 or c["window"]:
            at = torch.arange(L - n, L, device=out.device).unsqueeze(1)
            key = torch.arange(skip, L, device=out.device).unsqueeze(0)
            mask = key > at if c["causal"] else torch.zeros_like(key > at)
            if c["window"]:
                mask = mask | (key <= at - c["window"])
        q = s["q"][lo:lo + n].float() * D ** -0.5
        for h in range(K):
            w = torch.einsum("ngd,ld->gnl", q[:, h * G:(h + 1) * G], keys[:, h])
            if mask is not None:
                w = w.masked_fill(mask, float("-inf"))
            w = torch.exp(w - w.amax(-1, keepdim=True))
            o = torch.einsum("gnl,ld->ngd", w, vals[:, h]) / w.sum(-1).T.unsqueeze(-1)
            out[lo:lo + n, h * G:(h + 1) * G] = o.to(out.dtype)
    return {"out": out}


def _plain_fork(s):
    P = s["case"]["page"]
    table, lens, parents, children = s["table"], s["lens"], s["parents"].long(), s["children"].long()
    width = table.shape[1]
    n = lens[parents].long()
    whole = n // P
    slot = torch.arange(width, device=table.device)
    row = torch.where(slot < whole.unsqueeze(1), table[parents], table[children])
    row = torch.where(slot == whole.unsqueeze(1), s["new_pages"].unsqueeze(1), row)
    last = table[parents, whole.clamp(max=width - 1)].long()
    part = (n % P > 0).nonzero().squeeze(1)
    s["cache"][:, s["new_pages"].long()[part]] = s["cache"][:, last[part]]
    table[children] = row
    lens[children] = lens[parents]
    return {"table": table, "lens": lens, "cache": s["cache"]}


def _plain_compact(s):
    P = s["case"]["page"]
    table, cache = s["table"], s["cache"]
    pages = cache.shape[1]
    held = torch.arange(table.shape[1], device=table.device) < ((s["lens"] + P - 1) // P).unsqueeze(1)
    used = torch.zeros(pages, dtype=torch.bool, device=table.device)
    used[table[held].long()] = True
    count = used.sum()
    front = torch.arange(pages, device=table.device) < count
    src, dst = (used & ~front).nonzero().squeeze(1), (~used & front).nonzero().squeeze(1)
    remap = torch.arange(pages, device=table.device)
    remap[src] = dst
    cache[:, dst] = cache[:, src]
    out = torch.where(held, remap[table.clamp(min=0).long()].int(), -1)
    return {"table": out, "used": count.int().reshape(1), "cache": cache}


# ---- one pass --------------------------------------------------------------


def _own_axes(s):
    import rope_rope3d_apply_gb300 as rope3d

    pairing = {"interleaved": rope3d.PAIRS_INTERLEAVED, "halves": rope3d.PAIRS_HALVES}[s["case"]["pairs"]]
    call = rope3d.rope3d_apply_axes_backward if s["case"]["op"] == "axes_bwd" else rope3d.rope3d_apply_axes
    q, k = call(s["q"], s["k"], s["positions"], s["freqs"], s["sections"], pairing=pairing)
    return {"q": q, "k": k}


def _own_append(s):
    import rope_rope3d_apply_gb300 as rope3d

    pairing = {"interleaved": rope3d.PAIRS_INTERLEAVED, "halves": rope3d.PAIRS_HALVES}[s["case"]["pairs"]]
    rope3d.rope3d_cache_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["q_starts"],
                               freqs=s["freqs"], positions=s["positions"], sections=s["sections"], pairing=pairing,
                               q_out=s["q_out"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attention(s):
    import rope_rope3d_apply_gb300 as rope3d

    c = s["case"]
    rope3d.rope3d_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["q_starts"],
                                  scale=c["dim"] ** -0.5, causal=c["causal"], window=c["window"],
                                  max_new=s["most_new"], out=s["out"])
    return {"out": s["out"]}


def _own_fork(s):
    import rope_rope3d_apply_gb300 as rope3d

    rope3d.rope3d_cache_fork(s["cache"], s["table"], s["lens"], s["parents"], s["children"], s["new_pages"],
                             page_size=s["case"]["page"])
    return {"table": s["table"], "lens": s["lens"], "cache": s["cache"]}


def _own_compact(s):
    import rope_rope3d_apply_gb300 as rope3d

    table, used = rope3d.rope3d_cache_compact(s["cache"], s["table"], s["lens"], page_size=s["case"]["page"])
    return {"table": table, "used": used, "cache": s["cache"]}


def run(state):
    op = state["case"]["op"]
    op = "axes" if op == "axes_bwd" else op
    return globals()[("_own_" if own else "_plain_") + op](state)


# ---- what a pass cannot do without -----------------------------------------


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] in ("axes", "axes_bwd"):
        T, D, heads = case["tokens"], case["dim"], case["q_heads"] + case["kv_heads"]
        pairs = case["s0"] + case["s1"] + case["s2"]
        return {"bytes": T * (2 * e * heads * D + 3 * (4 if case["frac"] else 8)) + 4 * pairs,
                "flops": 6 * T * heads * pairs}
    if case["op"] == "append":
        n, D = sum(n for n, _ in _sizes(case)), case["dim"]
        return {"bytes": 2 * e * n * (case["q_heads"] + 2 * case["kv_heads"]) * D,
                "flops": 6 * n * (case["q_heads"] + case["kv_heads"]) * D // 2}
    if case["op"] == "attention":
        H, K, D, W = case["q_heads"], case["kv_heads"], case["dim"], case["window"]
        rows, keys, seen = 0, 0, 0
        for n, L in _sizes(case):
            rows += n
            first = max(0, L - n - W + 1) if W else 0
            keys += L - first
            for i in range(n):
                end = L - n + i + 1 if case["causal"] else L
                seen += end - (max(0, L - n + i - W + 1) if W else 0)
        return {"bytes": 2 * e * (rows * H + keys * K) * D, "flops": 4 * seen * H * D}
    page = e * case["page"] * case["kv_heads"] * case["dim"] * case["planes"]
    if case["op"] == "fork":
        lens = _lengths(case)
        of = [lens[i * 7 % len(lens)] for i in range(case["forks"])]
        return {"bytes": 2 * page * sum(n % case["page"] > 0 for n in of) + sum(8 * (n // case["page"] + 1) for n in of),
                "flops": 0}
    used, _, moved = _moves(case)
    return {"bytes": 2 * page * moved + 8 * used, "flops": 0}


# ---- in 64 bits ------------------------------------------------------------


def _exact_turn(x, positions, freqs, sections, pairs, sign):
    """x [tokens, heads, dim] with each pair as a complex number, turned."""
    x = x.double()
    n = sum(sections)
    of = torch.cat([positions[a].double().unsqueeze(1).expand(-1, m) for a, m in enumerate(sections)], 1)
    turn = torch.polar(torch.ones_like(of), sign * of * freqs.double()).unsqueeze(1)
    z = x[..., :2 * n]
    z = z.reshape(*z.shape[:-1], n, 2) if pairs == "interleaved" else z.reshape(*z.shape[:-1], 2, n).transpose(-1, -2)
    w = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
    w = w if pairs == "interleaved" else w.transpose(-1, -2)
    return torch.cat((w.flatten(-2), x[..., 2 * n:]), -1)


def _exact_append(s, case):
    P = case["page"]
    table = s["table"].cpu()
    k_cache, v_cache, q_out = s["k_cache"].double(), s["v_cache"].double(), s["q_out"].double()
    for i, (n, L) in enumerate(s["sizes"]):
        rows = slice(s["starts"][i], s["starts"][i] + n)
        where = torch.arange(L - n, L)
        pos = where.cuda().repeat(3, 1) if s["positions"] is None else s["positions"][:, rows]
        turn = lambda x: _exact_turn(x[rows], pos, s["freqs"], s["sections"], case["pairs"], 1.0)  # noqa: E731
        page, slot = table[i, where // P].long().cuda(), (where % P).cuda()
        q_out[rows], k_cache[page, slot], v_cache[page, slot] = turn(s["q"]), turn(s["k"]), s["v"][rows].double()
    return {"q": q_out, "k_cache": k_cache, "v_cache": v_cache}


def _exact_attention(s, case):
    P, H, K, W = case["page"], case["q_heads"], case["kv_heads"], case["window"]
    out = s["out"].double()
    for i, (n, L) in enumerate(s["sizes"]):
        rows = slice(s["starts"][i], s["starts"][i] + n)
        of = s["table"][i, :_up(L, P)].long()
        for h in range(H):
            keys = s["k_cache"][of, :, h // (H // K)].reshape(-1, case["dim"])[:L].double()
            vals = s["v_cache"][of, :, h // (H // K)].reshape(-1, case["dim"])[:L].double()
            score = s["q"][rows, h].double() @ keys.T / math.sqrt(case["dim"])
            behind = torch.arange(L - n, L, device="cuda")[:, None] - torch.arange(L, device="cuda")
            seen = (behind >= 0) if case["causal"] else torch.ones_like(behind, dtype=torch.bool)
            if W:
                seen &= behind < W
            score[~seen] = -math.inf
            out[rows, h] = torch.softmax(score, 1) @ vals
    return {"out": out}


def _exact_fork(s, case):
    P = case["page"]
    table, lens, cache = s["table"].cpu(), s["lens"].cpu(), s["cache"].double()
    for parent, child, new in zip(s["parents"].tolist(), s["children"].tolist(), s["new_pages"].tolist()):
        n = int(lens[parent])
        lens[child] = n
        table[child, :n // P] = table[parent, :n // P]
        table[child, n // P] = new
        if n % P:
            cache[:, new] = s["cache"][:, int(table[parent, n // P])].double()
    return {"table": table.cuda(), "lens": lens.cuda(), "cache": cache}


def _exact_compact(s, case):
    table, cache = s["table"].tolist(), s["cache"].double()
    held = [row[:_up(n, case["page"])] for row, n in zip(table, s["lengths"])]
    used = sorted(set(sum(held, [])))
    count = len(used)
    to = dict(zip([p for p in used if p >= count], sorted(set(range(count)) - set(used))))
    for a, b in to.items():
        cache[:, b] = s["cache"][:, a].double()
    out = torch.full_like(s["table"], -1, device="cpu")
    for i, row in enumerate(held):
        out[i, :len(row)] = torch.tensor([to.get(p, p) for p in row], dtype=torch.int32)
    return {"table": out.cuda(), "used": _int([count]), "cache": cache}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("axes", "axes_bwd"):
        sign = -1.0 if case["op"] == "axes_bwd" else 1.0
        return {x: _exact_turn(s[x], s["positions"], s["freqs"], s["sections"], case["pairs"], sign) for x in ("q", "k")}
    return {"append": _exact_append, "attention": _exact_attention, "fork": _exact_fork,
            "compact": _exact_compact}[case["op"]](s, case)
