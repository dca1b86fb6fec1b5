"""rope3d_apply_axes, its gradient and rope3d_cache_append against 64-bit formulas."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import rope_rope3d_apply_gb300 as r  # noqa: E402
from tests.paged_reference import angles, close, rotate64  # noqa: E402

DEV = torch.device("cuda:0")
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
PAIRING = {"interleaved": r.PAIRS_INTERLEAVED, "halves": r.PAIRS_HALVES}


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def freqs_of(sections):
    return torch.tensor([10000.0 ** (-j / n) for n in sections for j in range(n)], dtype=torch.float32, device=DEV)


def positions_of(g, kind, axes, tokens, far):
    if kind == "f32":
        return (torch.rand((axes, tokens), generator=g, device=DEV) - 0.3) * far
    p = torch.randint(-far // 3, far, (axes, tokens), generator=g, device=DEV)
    return p.to({"i64": torch.int64, "i32": torch.int32}[kind])


SHAPES = [
    # tokens, heads, kv, dim, sections, kernel that takes it in 16 bits
    (1, 1, 1, 16, (8, 0, 0), 1),
    (77, 4, 2, 64, (8, 12, 12), None),
    (300, 8, 4, 256, (32, 48, 48), 1),
    (33, 20, 20, 128, (16, 24, 24), 1),
    (1000, 3, 1, 80, (40,), None),
    (50, 2, 2, 48, (3, 5, 7), 2),
    (9, 5, 1, 6, (1, 1, 1), 2),
    (130, 2, 1, 130, (0, 17, 31), 2),
    (3000, 16, 2, 128, (10, 11, 11), None),
]


@pytest.mark.parametrize("pairing", list(PAIRING))
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_rotation_and_gradient(case, dtype, pairing):
    tokens, heads, kv, dim, sections, kernel = SHAPES[case]
    g, t = gen(case), TYPES[dtype]
    q, k = (torch.randn((tokens, n, dim), generator=g, device=DEV).to(t) for n in (heads, kv))
    freqs, pairs = freqs_of(sections), sum(sections)
    for kind, far in (("i64", 2000), ("i32", 1 << 24), ("f32", 1000), ("i64", 1 << 30)):
        pos = positions_of(g, kind, len(sections), tokens, far)
        a = angles(pos, freqs, sections)
        got = r.rope3d_apply_axes(q, k, pos, freqs, sections, pairing=PAIRING[pairing])
        back = r.rope3d_apply_axes_backward(q, k, pos, freqs, sections, pairing=PAIRING[pairing])
        if kernel and dtype != "f32":
            assert r.rope3d_apply_axes_last_kernel() == kernel
        for x, y, z in zip((q, k), got, back):
            close(y, *rotate64(x, a, pairing, pairs), f"{kind} forward")
            close(z, *rotate64(x, -a, pairing, pairs), f"{kind} backward")
            assert torch.equal(y[..., 2 * pairs:], x[..., 2 * pairs:])


@pytest.mark.parametrize("kind,far,top", [("f32", 1, 2e4), ("f32", 1 << 26, 1.0), ("i64", 1 << 20, 2e4), ("i64", 1 << 33, 1.0),
                                          ("i32", (1 << 31) - 1, 1.0), ("i64", 1 << 12, 1e7), ("f32", 3000, 1e5)])
def test_far_positions_and_high_frequencies(kind, far, top):
    """Frequencies far above 1 (a vector that grows with the pair) and positions that no fp32 has:
    against angles reduced with whole numbers."""
    from fractions import Fraction

    g, pairs, tokens = gen(40), 16, 12
    freqs = torch.tensor([top ** (j / (pairs - 1)) if top > 1 else 10000.0 ** (-j / pairs) for j in range(pairs)], device=DEV)
    pos = positions_of(g, kind, 1, tokens, far)
    # 40 digits of 1 / 2 pi: the reduced angle is right to 2^-53 or so
    inv = Fraction(1591549430918953357688837633725143620345, 10 ** 40)
    turns = [[Fraction(p) * Fraction(f) * inv for f in freqs.tolist()] for p in pos[0].tolist()]
    a = torch.tensor([[float(t - round(t)) for t in row] for row in turns], dtype=torch.float64, device=DEV) * (2 * math.pi)
    q = torch.randn((tokens, 2, 2 * pairs), generator=g, device=DEV)
    for pairing in PAIRING:
        got, _ = r.rope3d_apply_axes(q, None, pos, freqs, pairing=PAIRING[pairing])
        close(got, *rotate64(q, a, pairing, pairs))


def test_agrees_with_whole_grids():
    """Positions that are a grid's coordinates, frequencies as the tables have them: the
    operator for grids within the error of the tables' rounding and the cosine's."""
    T, H, W, split = 3, 5, 7, (16, 24, 24)
    g = gen(1)
    n = T * H * W
    q, k = (torch.randn((1, n, 4, 64), generator=g, device=DEV) for _ in range(2))
    with r.rope3d_build_tables(T, H, W, split, 10000.0) as tables:
        want = r.rope3d_apply_pair(q, k, tables)
    at = torch.arange(n, device=DEV)
    pos = torch.stack((at // (H * W), at // W % H, at % W))
    got = r.rope3d_apply_axes(q[0], k[0], pos, freqs_of([d // 2 for d in split]), [d // 2 for d in split])
    for a, b, x in zip(got, want, (q, k)):
        size = x[0].abs().unfold(-1, 2, 2).sum(-1).repeat_interleave(2, -1).double()
        # cos and sin: 2^-22 here, half a step there; frequencies in fp32 here: positions to 6, 6 * 2^-24
        close(a, b[0].double(), size * (2.0 ** -22 + 2.0 ** -24 + 6 * 2.0 ** -24 + 4 * 2.0 ** -24))


def test_turning_back_and_differences():
    """The gradient is the transpose: <R x, y> = <x, R' y>, and differences of the operator
    give the same (it is linear)."""
    g = gen(2)
    q, y = (torch.randn((40, 2, 32), generator=g, device=DEV) for _ in range(2))
    freqs, sections = freqs_of((5, 5, 4)), (5, 5, 4)
    pos = positions_of(g, "f32", 3, 40, 300)
    turn = lambda x: r.rope3d_apply_axes(x, None, pos, freqs, sections)[0]  # noqa: E731
    grad = r.rope3d_apply_axes_backward(y, None, pos, freqs, sections)[0]
    left, right = (turn(q).double() * y.double()).sum(), (q.double() * grad.double()).sum()
    size = float(q.double().norm() * y.double().norm())
    assert abs(float(left - right)) <= size * 2.0 ** -20
    d = torch.randn(q.shape, generator=g, device=DEV)
    step = ((turn(q + 0.5 * d).double() - turn(q - 0.5 * d).double()) * y.double()).sum()
    assert abs(float(step - (d.double() * grad.double()).sum())) <= 2.0 ** -19 * float((q.norm() + d.norm()) * y.norm())


@pytest.mark.parametrize("pairing", list(PAIRING))
@pytest.mark.parametrize("dim,sections", [(128, (16, 24, 24)), (20, (2, 3, 4))])
def test_views_in_place_and_neighbours(pairing, dim, sections):
    """q and k in place inside one projection; heads first in memory; odd addresses; the
    rest of the buffers keeps its values."""
    g, t = gen(3), torch.bfloat16
    tokens, pairs = 37, sum(sections)
    pos, freqs = positions_of(g, "i64", 3, tokens, 900), freqs_of(sections)
    a = angles(pos, freqs, sections)
    qkv = torch.randn((tokens, 3, 4, dim), generator=g, device=DEV).to(t)
    was = qkv.clone()
    q, k = qkv[:, 0], qkv[:, 1]
    out = r.rope3d_apply_axes(q, k, pos, freqs, sections, pairing=PAIRING[pairing], q_out=q, k_out=k)
    assert out[0] is q and out[1] is k
    for i in (0, 1):
        close(qkv[:, i], *rotate64(was[:, i], a, pairing, pairs))
    assert torch.equal(qkv[:, 2], was[:, 2])
    flat = torch.full((tokens * 4 * dim + 3,), 5.0, dtype=t, device=DEV)   # two bytes past a boundary
    odd = flat[1:-2].view(4, tokens, dim).transpose(0, 1)
    r.rope3d_apply_axes(was[:, 0], None, pos, freqs, sections, pairing=PAIRING[pairing], q_out=odd)
    close(odd, *rotate64(was[:, 0], a, pairing, pairs))
    assert flat[0] == 5 and bool((flat[-2:] == 5).all())
    one = was[:1, 0].expand(tokens, 4, dim)   # a broadcast input
    got, _ = r.rope3d_apply_axes(one, None, pos, freqs, sections, pairing=PAIRING[pairing], q_out=torch.empty_like(was[:, 0]))
    close(got, *rotate64(one, a, pairing, pairs))


def test_special_values():
    """Infinities and NaN stay in their pairs."""
    x = torch.ones((3, 1, 8), device=DEV)
    x[0, 0, 2], x[1, 0, 5] = math.inf, math.nan
    pos, freqs = torch.tensor([[1, 2, 0]], device=DEV), torch.tensor([1.0, 0.5, 0.25, 0.1], device=DEV)
    got, _ = r.rope3d_apply_axes(x, None, pos, freqs)
    ok = torch.ones_like(x, dtype=torch.bool)
    ok[0, 0, 2:4], ok[1, 0, 4:6] = False, False
    assert bool(got[ok].isfinite().all()) and not bool(got[~ok].isfinite().any())
    assert torch.equal(got[2], x[2])   # position 0 turns nothing


# ---- append --------------------------------------------------------------------


def place_of(seq_len, new, i):
    return seq_len - new + i


APPENDS = [
    # new, lens, heads, kv, dim, page, sections, positions
    ([1], [1], 1, 1, 64, 16, (32,), None),
    ([1] * 9, [5, 64, 65, 1, 300, 16, 17, 31, 33], 8, 4, 128, 16, (64, 0, 0), None),
    ([40, 0, 7], [40, 9, 130], 4, 2, 256, 8, (32, 48, 48), "i64"),
    ([33, 61], [70, 61], 3, 1, 80, 5, (10, 10, 20), "f32"),
    ([20], [20], 2, 2, 48, 128, (3, 5, 7), "i32"),
    ([300, 11], [900, 11], 6, 2, 96, 24, (24, 0, 0), None),
]


@pytest.mark.parametrize("layout", ["places", "heads", "joint"])
@pytest.mark.parametrize("pairing", list(PAIRING))
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append(case, dtype, pairing, layout):
    new, lens, heads, kv, dim, page, sections, kind = APPENDS[case]
    g, t = gen(10 + case), TYPES[dtype]
    from tests.paged_reference import make_cache

    k_cache, v_cache, table = make_cache(g, lens, page, kv, dim, t, layout=layout, fill=9.0)
    was = k_cache.clone(), v_cache.clone()
    n, pad = sum(new), 3
    qkv = torch.randn((n + pad, heads + 2 * kv, dim), generator=g, device=DEV).to(t)
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    starts = [sum(new[:i]) for i in range(len(new) + 1)]
    places = torch.cat([torch.arange(L - m, L, device=DEV) for L, m in zip(lens, new)])
    pos = positions_of(g, kind, len(sections), n + pad, 1000) if kind else None
    freqs, pairs = freqs_of(sections), sum(sections)
    a = angles(pos[:, :n] if kind else places.expand(3, n), freqs, sections)
    out, bad = torch.full((n + pad, heads, dim), 5.0, dtype=t, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    got = r.rope3d_cache_append(q, k, v, k_cache, v_cache, table, ints(lens), ints(starts), freqs=freqs, positions=pos,
                                sections=sections, pairing=PAIRING[pairing], q_out=out, invalid_count=bad)
    assert got is out and int(bad) == 0
    close(out[:n], *rotate64(q[:n], a, pairing, pairs), "q")
    assert bool((out[n:] == 5).all())
    seq = torch.cat([torch.full((m,), s, device=DEV) for s, m in enumerate(new)])
    page_of = table.long()[seq, places // page]
    close(k_cache[page_of, places % page], *rotate64(k[:n], a, pairing, pairs), "k")
    assert torch.equal(v_cache[page_of, places % page], v[:n])
    for now, before, x in ((k_cache, was[0], k), (v_cache, was[1], v)):   # and nothing else changed
        before[page_of, places % page] = now[page_of, places % page]
        assert torch.equal(now, before)


def test_append_without_rotation_and_bad_pages():
    """No frequencies: a copy. Tokens without a page leave the cache alone and are counted."""
    g, t = gen(30), torch.float16
    k_cache, v_cache = (torch.full((6, 4, 2, 24), 9.0, dtype=t, device=DEV) for _ in range(2))
    k, v = (torch.randn((8, 2, 24), generator=g, device=DEV).to(t) for _ in range(2))
    table = torch.tensor([[2, -1, 5], [6, 0, 1]], dtype=torch.int32, device=DEV)
    lens, bad = torch.tensor([10, 3], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    assert r.rope3d_cache_append(None, k, v, k_cache, v_cache, table, lens, invalid_count=bad) is None
    # sequence 0: places 6 and 7 on page -1, 8 and 9 on page 5; sequence 1: place -1 and the rest on page 6 of 6
    assert int(bad) == 2 + 4
    for c, x in ((k_cache, k), (v_cache, v)):
        want = torch.full_like(c, 9.0)
        want[5, :2] = x[2:4]
        assert torch.equal(c, want)


def test_append_offsets_past_32_bits():
    pages, page, kv, dim = 66000, 16, 16, 128
    cache = torch.zeros((2, pages, page, kv, dim), dtype=torch.bfloat16, device=DEV)
    g = gen(31)
    k, v = (torch.randn((5, kv, dim), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device=DEV)
    r.rope3d_cache_append(None, k, v, cache[0], cache[1], table, torch.tensor([5], dtype=torch.int32, device=DEV))
    assert torch.equal(cache[0, -1, :5], k) and torch.equal(cache[1, -1, :5], v)
    assert int((cache[0] != 0).sum()) == int((k != 0).sum())
