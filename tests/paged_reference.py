"""The operators around a paged cache in 64 bits, from their definitions, with bounds
on what a sound computation in 32 bits may differ by (test infrastructure; plain
torch, no code of the library).

Roundings counted: half a step of the type, finfo(t).eps / 2 relative, for an output
and for a softmax weight as an operand; 2^-24 for a product or sum in fp32; 2^-22 for a sum
inside a matrix instruction (which may cut instead of round) and for exp2.
"""
from __future__ import annotations

import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}   # half a step of subnormal results


def close(got, want, bound, what=""):
    """got within `bound` of want everywhere; NaN nowhere."""
    got = got.double()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= bound)
    if bad.any():
        i = bad.nonzero()[0].tolist()
        at = tuple(i)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {got[at].item()} for "
                             f"{want[at].item()}, bound {bound.expand_as(want)[at].item()}")


# ---- rotations ---------------------------------------------------------------


def rotate64(x, angle, pairing, pairs):
    """(result, bound) of x [tokens, heads, dim] turned by angle [tokens, pairs] (64
    bits). Bound: cos and sin within 2^-22 (sincospi to a unit in the last place of 1, 2^-23,
    the reduced angle and the correction 2^-23 together), two products and a sum."""
    y = x.double()
    c, s = torch.cos(angle).unsqueeze(1), torch.sin(angle).unsqueeze(1)
    if pairing == "interleaved":
        a, b = y[..., 0:2 * pairs:2], y[..., 1:2 * pairs:2]
    else:
        a, b = y[..., :pairs], y[..., pairs:2 * pairs]
    first, second, size = a * c - b * s, a * s + b * c, a.abs() + b.abs()
    out, bound = y.clone(), torch.zeros_like(y)
    half, tiny = HALF[x.dtype], TINY[x.dtype]
    if pairing == "interleaved":
        out[..., 0:2 * pairs:2], out[..., 1:2 * pairs:2] = first, second
        bound[..., 0:2 * pairs:2] = bound[..., 1:2 * pairs:2] = size * (2.0 ** -22 + 2 * 2.0 ** -24)
    else:
        out[..., :pairs], out[..., pairs:2 * pairs] = first, second
        bound[..., :pairs] = bound[..., pairs:2 * pairs] = size * (2.0 ** -22 + 2 * 2.0 ** -24)
    turned = bound > 0
    return out, bound + turned * ((out.abs() + bound) * half + tiny)


def angles(positions, freqs, sections):
    """[tokens, pairs] from positions [axes, tokens]."""
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    return positions.double()[axis].T * freqs.double()


# ---- attention -----------------------------------------------------------------


def gather(cache, table_row, length, absent):
    """Rows 0 .. length - 1 of a sequence [length, heads, dim], and which of them lie on
    pages that are there."""
    pages, size = cache.shape[:2]
    place = torch.arange(length, device=cache.device)
    page = table_row.long()[place // size] if length else place
    there = (page >= 0) & (page < pages)
    rows = cache[page.clamp(0, pages - 1), place % size]
    assert absent or bool(there.all())
    return rows, there


def attention64(q, k_cache, v_cache, table, lens, starts, scale, causal, window, absent=False):
    """(out, bound, lse, lse bound) for the tokens of the sequences; rows behind the last
    are NaN in `out` (not compared). All lists on the host: lens, starts.

    Bound: a score is a sum of dim products (2^-22 each, of the sum of their sizes),
    scaled (2^-23 of it with the subtraction of the maximum, both up to the largest score);
    its weight is off by that relative, by 2^-22 for exp2, and as an operand by half a
    step (or, fp16, by 2^-25 of the largest weight, which is 1). Weighted sums and the
    sum of weights add up to length / 16 + 40 sums of 2^-22 each."""
    T, H, D = q.shape
    K, group, half = k_cache.shape[2], H // k_cache.shape[2], HALF[q.dtype]
    out = torch.full((T, H, D), math.nan, dtype=torch.float64, device=q.device)
    bound, lse = out.clone(), torch.full((T, H), math.nan, dtype=torch.float64, device=q.device)
    lse_bound = lse.clone()
    for s, L in enumerate(lens):
        lo, n = starts[s], starts[s + 1] - starts[s]
        if n == 0:
            continue
        keys, there = gather(k_cache, table[s], L, absent)
        vals, _ = gather(v_cache, table[s], L, absent)
        at = torch.arange(L - n, L, device=q.device).unsqueeze(1)
        key = torch.arange(L, device=q.device).unsqueeze(0)
        seen = there.unsqueeze(0).expand(n, L)
        if causal:
            seen = seen & (key <= at)
        if window:
            seen = seen & (key > at - window)
        for h in range(H):
            x, kk, vv = q[lo:lo + n, h].double(), keys[:, h // group].double(), vals[:, h // group].double()
            kk = torch.where(there.unsqueeze(1), kk, 0.0)
            vv = torch.where(seen.any(0).unsqueeze(1), vv, 0.0)
            score = x @ kk.T * scale
            size = x.abs() @ kk.abs().T * scale
            score = torch.where(seen, score, -math.inf)
            top = score.amax(1, keepdim=True) if L else torch.full((n, 1), -math.inf, dtype=torch.float64, device=q.device)
            top = torch.where(top == -math.inf, 0.0, top)
            w = torch.exp(score - top)
            total = w.sum(1, keepdim=True)
            safe = torch.where(total > 0, total, 1.0)
            p = w / safe
            off = torch.where(seen, size * (D + 2) * 2.0 ** -22, 0.0)
            off = off + torch.where(seen, (score.abs().masked_fill(~seen, 0.0).amax(1, keepdim=True) if L else 0.0) * 2.0 ** -22, 0.0)
            each = off + 2.0 ** -22          # a weight's relative error before it is an operand
            sums = (L / 16 + 40) * 2.0 ** -22
            rel = torch.expm1(each)
            o = p @ vv
            mag = p @ vv.abs()
            err = (p * (rel + half)) @ vv.abs() + mag * ((p * rel).sum(1, keepdim=True) + 2 * sums)
            if q.dtype == torch.float16:
                err = err + (seen.double() @ vv.abs()) * 2.0 ** -25 / safe
            out[lo:lo + n, h] = o
            bound[lo:lo + n, h] = err + (o.abs() + err) * half + TINY[q.dtype]
            lse[lo:lo + n, h] = torch.where(total > 0, top + torch.log(safe), -math.inf)[:, 0]
            lse_bound[lo:lo + n, h] = ((p * rel).sum(1) + sums + (top.abs()[:, 0] + torch.log(safe).abs()[:, 0] + 1) * 2.0 ** -22)
    return out, bound, lse, lse_bound


def check_attention(r, q, k_cache, v_cache, table, lens, starts, scale=None, causal=True, window=0, absent=False, **kw):
    """One call of the library against the 64-bit formulas, log sum exp included; what
    lies behind the last sequence stays as it was."""
    dev = q.device
    T, H, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    out = kw.pop("out", None)
    out = torch.full((T, H, D), 7.0, dtype=q.dtype, device=dev) if out is None else out.fill_(7.0)
    lse = torch.full((T, H), 7.0, device=dev)
    got, got_lse = r.rope3d_paged_attention(q, k_cache, v_cache, table, ints(lens), ints(starts), scale=scale, causal=causal,
                                            window=window, out=out, lse=lse, **kw)
    want, bound, want_lse, lse_bound = attention64(q, k_cache, v_cache, table, lens, starts, scale, causal, window, absent)
    end = starts[-1]
    close(got[:end], want[:end], bound[:end], "out")
    empty = want_lse[:end] == -math.inf
    assert torch.equal(got_lse[:end] == -math.inf, empty)
    close(got_lse[:end].masked_fill(empty, 0.0), want_lse[:end].masked_fill(empty, 0.0), lse_bound[:end], "lse")
    assert bool((got[end:] == 7.0).all()) and bool((got_lse[end:] == 7.0).all())
    return got


def make_cache(g, lens, page, heads, dim, dtype, width=None, layout="places", spare=3, fill=math.nan):
    """(k_cache, v_cache, table) whose sequences hold normal values; everything else,
    behind the lengths and on unused pages, is `fill`. layout: "places" ([pages, page,
    heads, dim]), "heads" (heads before places in memory), "joint" (K and V of a place
    side by side)."""
    dev = g.device
    held = [-(-n // page) for n in lens]
    pages = sum(held) + spare
    if layout == "heads":
        make = lambda: torch.full((pages, heads, page, dim), fill, dtype=dtype, device=dev).transpose(1, 2)  # noqa: E731
        k, v = make(), make()
    elif layout == "joint":
        both = torch.full((pages, page, 2, heads, dim), fill, dtype=dtype, device=dev)
        k, v = both[:, :, 0], both[:, :, 1]
    else:
        k, v = (torch.full((pages, page, heads, dim), fill, dtype=dtype, device=dev) for _ in range(2))
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(lens), max(1, width or max(held) + 1)), -1, dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(lens):
        table[s, :held[s]] = order[at:at + held[s]]
        at += held[s]
        place = torch.arange(n, device=dev)
        if n:
            page_of = table[s].long()[place // page]
            for c in (k, v):
                c[page_of, place % page] = torch.randn((n, heads, dim), generator=g, device=dev).to(dtype)
    return k, v, table
