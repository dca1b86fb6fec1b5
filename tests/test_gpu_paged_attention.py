"""rope3d_paged_attention against 64-bit formulas: types, head layouts, lengths, page
sizes, masks, absent pages, views, and what lies behind lengths and sequences."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import rope_rope3d_apply_gb300 as r  # noqa: E402
from tests.paged_reference import attention64, check_attention, close, make_cache  # noqa: E402

DEV = torch.device("cuda:0")
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    assert r.rope3d_testing_paged_wait_timeouts() == 0


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def starts_of(new):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return out


def run(seed, new, lens, heads, kv, dim, page, dtype=BF, pad=0, layout="places", width=None, **kw):
    g = gen(seed)
    k, v, table = make_cache(g, lens, page, kv, dim, dtype, layout=layout, width=width)
    starts = starts_of(new)
    q = torch.randn((starts[-1] + pad, heads, dim), generator=g, device=DEV).to(dtype)
    return check_attention(r, q, k, v, table, lens, starts, **kw)


# one new token of every sequence
ONE = [
    # lens, heads, kv, dim, page
    ([1], 1, 1, 64, 16),
    ([2, 1, 63, 64, 65], 4, 4, 64, 16),
    ([200, 1000, 17], 8, 4, 128, 16),
    ([1500], 8, 4, 256, 16),
    ([130, 129, 128, 127], 16, 1, 128, 64),
    ([700, 5], 12, 2, 80, 24),
    ([333, 90, 1], 5, 5, 72, 7),
    ([257, 3], 6, 2, 192, 1),
    ([400, 12], 3, 1, 8, 5),
    ([5000] + [40] * 70, 8, 2, 64, 32),
    ([999, 1024, 1025], 7, 1, 96, 128),
    ([640, 40], 20, 1, 128, 16),
    ([300, 41], 64, 1, 64, 16),
    ([90], 130, 1, 128, 8),
    ([1 + 7 * (i % 11) for i in range(3000)], 2, 1, 64, 8),
]


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("case", range(len(ONE)))
def test_single_tokens(case, dtype):
    lens, heads, kv, dim, page = ONE[case]
    run(case, [1] * len(lens), lens, heads, kv, dim, page, dtype, max_new=1)


# chunks of new tokens
CHUNKS = [
    # new, lens, heads, kv, dim, page
    ([2], [2], 1, 1, 64, 16),
    ([17, 1, 40], [17, 100, 300], 4, 2, 128, 16),
    ([128], [128], 2, 2, 128, 64),
    ([129, 127], [129, 500], 8, 4, 256, 16),
    ([300, 5], [1000, 5], 6, 2, 64, 8),
    ([77, 0, 33], [150, 90, 33], 3, 1, 96, 128),
    ([65, 64, 63], [65, 200, 333], 5, 5, 72, 24),
    ([50], [700], 16, 2, 80, 256),
    ([90, 31], [400, 31], 4, 1, 192, 3),
    ([512], [1024], 8, 1, 128, 32),
    ([700], [700], 2, 1, 256, 64),
    ([40, 9], [200, 9], 66, 1, 128, 16),
    ([33, 5], [100, 700], 4, 2, 8, 8),
    ([150], [333], 3, 1, 136, 40),
    ([20, 3], [40000, 70000], 8, 1, 200, 128),
    ([1, 0, 2] * 400, [3, 0, 2] * 400, 2, 1, 64, 8),
]


# a hint that makes a kernel of the call's rows: few, one block's, a pair's (or the next below)
HINTS = {"few": 1, "tile": 128, "pair": 0}


@pytest.mark.parametrize("kernel", list(HINTS))
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("case", range(len(CHUNKS)))
def test_chunks(case, dtype, kernel):
    new, lens, heads, kv, dim, page = CHUNKS[case]
    group, pad = heads // kv, case % 3
    hint = max(HINTS[kernel] // group, 1) if HINTS[kernel] else 0
    run(100 + case, new, lens, heads, kv, dim, page, dtype, pad=pad, max_new=hint)
    tokens = sum(new) + pad
    rows = min(tokens, hint or tokens) * group
    assert r.rope3d_paged_attention_last_kernel() == (1 if rows <= 16 or page % 8 else 3 if rows > 128 and dim > 64 else 2)


@pytest.mark.parametrize("window", [1, 5, 64, 100, 129, 300, 1000])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hint", [0, 64])
@pytest.mark.parametrize("new,lens,page,dim", [([1, 1, 1], [90, 700, 3], 16, 128), ([150, 40, 1], [400, 40, 600], 16, 64),
                                               ([140], [300], 8, 256), ([310, 1, 500], [900, 40, 800], 32, 128)])
def test_windows(window, causal, hint, new, lens, page, dim):
    run(7, new, lens, 4, 2, dim, page, HF, window=window, causal=causal, max_new=hint)


@pytest.mark.parametrize("new,lens", [([40, 7], [300, 90]), ([1, 1], [300, 64]), ([200], [200])])
def test_every_place_seen(new, lens):
    run(8, new, lens, 4, 2, 128, 16, BF, causal=False)


@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("kernel_rows", [1, 64])
def test_rows_that_see_nothing(page, kernel_rows):
    """Lengths of zero, and shorter than the new tokens: the first of those see no key."""
    new = [kernel_rows, kernel_rows, kernel_rows, 2]
    run(9, new, [0, kernel_rows // 2, kernel_rows, 0], 4, 2, 64, page, BF, pad=2, width=48)
    run(10, new, [0, kernel_rows // 2, 200, 0], 4, 2, 64, page, HF, window=3, width=48)


@pytest.mark.parametrize("layout", ["heads", "joint"])
@pytest.mark.parametrize("new,lens,dim", [([1, 1], [300, 41], 128), ([70, 9], [300, 41], 128), ([70, 9], [300, 41], 256)])
def test_cache_layouts(layout, new, lens, dim):
    run(11, new, lens, 4, 2, dim, 16, BF, layout=layout)


@pytest.mark.parametrize("new", [[1, 1, 1], [60, 1, 100]])
def test_absent_pages(new):
    """Numbers outside the cache name pages that are not there: their keys are left out,
    and a sequence without any page gives zeros."""
    g = gen(12)
    lens = [300, 90, 200]
    k, v, table = make_cache(g, lens, 16, 2, 64, BF)
    table[0, 3], table[0, 7], table[0, 18] = -1, k.shape[0], 1 << 30
    table[1, :] = -(1 << 31)
    starts = starts_of(new)
    q = torch.randn((starts[-1], 4, 64), generator=g, device=DEV).to(BF)
    check_attention(r, q, k, v, table, lens, starts, absent=True)


@pytest.mark.parametrize("new", [1, 50])
def test_views_of_one_projection(new):
    """q from a fused projection, out into a wider buffer, heads first in memory; the
    elements beside out keep their values."""
    g = gen(13)
    lens = [130, 77]
    k, v, table = make_cache(g, lens, 16, 2, 128, HF)
    starts = starts_of([new, new])
    qkv = torch.randn((2 * new, 8, 128), generator=g, device=DEV).to(HF)
    wide = torch.full((2 * new, 6, 136), 3.0, dtype=HF, device=DEV)
    check_attention(r, qkv[:, :4], k, v, table, lens, starts, out=wide[:, 1:5, :128])
    assert bool((wide[:, 0] == 3).all()) and bool((wide[:, 5] == 3).all()) and bool((wide[:, :, 128:] == 3).all())
    across = torch.full((4, 2 * new, 128), 3.0, dtype=HF, device=DEV).transpose(0, 1)
    flipped = qkv[:, :4].transpose(0, 1).contiguous().transpose(0, 1)
    check_attention(r, flipped, k, v, table, lens, starts, out=across)


def test_equal_tokens_without_starts():
    g = gen(14)
    for n in (1, 3, 40):
        lens = [50, 200, 333]
        k, v, table = make_cache(g, lens, 16, 2, 64, BF)
        q = torch.randn((3 * n, 4, 64), generator=g, device=DEV).to(BF)
        got = r.rope3d_paged_attention(q, k, v, table, torch.tensor(lens, dtype=torch.int32, device=DEV))
        want, bound, _, _ = attention64(q, k, v, table, lens, [0, n, 2 * n, 3 * n], 64 ** -0.5, True, 0)
        close(got, want, bound)


@pytest.mark.parametrize("new,hint", [(1, 0), (200, 64), (200, 0)])
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_large_scores(new, hint, dtype, dim):
    """Scores of hundreds, rising along the keys, so that the maximum moves in every block."""
    g = gen(15)
    lens = [900]
    k, v, table = make_cache(g, lens, 16, 1, dim, dtype)
    k[table[0, :57].long()] *= torch.linspace(0.1, 12, 57, device=DEV).reshape(57, 1, 1, 1).to(dtype)
    q = (torch.randn((new, 2, dim), generator=g, device=DEV) * 4).to(dtype)
    check_attention(r, q, k, v, table, lens, [0, new], max_new=hint)


@pytest.mark.parametrize("new", [1, 150])
def test_offsets_past_32_bits(new):
    """A cache of 2^31 elements and more, the sequence on its last pages."""
    pages, page, kv, dim = 66000, 16, 16, 128
    k = torch.zeros((pages, page, kv, dim), dtype=BF, device=DEV)
    assert k.numel() > 1 << 31
    v = torch.zeros_like(k)
    g = gen(16)
    lens = [300]
    table = torch.arange(pages - 19, pages, dtype=torch.int32, device=DEV).flip(0).reshape(1, 19).contiguous()
    for c in (k, v):
        c[-19:] = torch.randn((19, page, kv, dim), generator=g, device=DEV).to(BF)
    q = torch.randn((new, kv, dim), generator=g, device=DEV).to(BF)
    check_attention(r, q, k, v, table, lens, [0, new])


@pytest.mark.parametrize("new,lens", [([1] * 6, [4000, 3, 77, 900, 20000, 1]), ([300, 1, 700], [2000, 9000, 700])])
def test_results_do_not_depend_on_the_hint_or_the_call(new, lens):
    """The same call twice gives the same bits; max_new changes the kernel, and results
    only within the bounds."""
    g = gen(17)
    k, v, table = make_cache(g, lens, 16, 2, 128, BF)
    starts = starts_of(new)
    q = torch.randn((starts[-1], 8, 128), generator=g, device=DEV).to(BF)
    a = check_attention(r, q, k, v, table, lens, starts)
    b = check_attention(r, q, k, v, table, lens, starts)
    assert torch.equal(a, b)
    check_attention(r, q, k, v, table, lens, starts, max_new=max(new))
    check_attention(r, q, k, v, table, lens, starts, max_new=1)   # a wrong one: slower at most


def test_special_values():
    """An infinite score gives NaN as the formula does, and only in rows that see it; a NaN
    key behind the mask of single tokens is not seen."""
    g = gen(18)
    lens = [40, 40]
    k, v, table = make_cache(g, lens, 16, 1, 64, BF)
    k[table[0, 0].long(), 3, 0, 0] = math.inf
    q = torch.randn((2, 1, 64), generator=g, device=DEV).to(BF).abs()
    got = r.rope3d_paged_attention(q, k, v, table, torch.tensor(lens, dtype=torch.int32, device=DEV))
    assert bool(got[0].isnan().all()) and bool(got[1].isfinite().all())


@pytest.mark.parametrize("new,length", [(1, 40), (1, 5000), (200, 300), (200, 5000)])
def test_rows_of_nan(new, length):
    """A query row of NaN gives NaN in its own row, whole or joined from parts, and nowhere else."""
    g = gen(20)
    k, v, table = make_cache(g, [length], 16, 2, 64, BF)
    q = torch.randn((new, 4, 64), generator=g, device=DEV).to(BF)
    q[new // 2, 1] = math.nan
    got, lse = r.rope3d_paged_attention(q, k, v, table, torch.tensor([length], dtype=torch.int32, device=DEV), lse=True)
    bad = torch.zeros((new, 4), dtype=torch.bool, device=DEV)
    bad[new // 2, 1] = True
    assert torch.equal(got.isnan().all(-1), bad) and torch.equal(got.isnan().any(-1), bad) and torch.equal(lse.isnan(), bad)


def test_damaged_lengths_and_starts_stay_inside():
    """Lengths past the table, falling and wild starts: nothing outside is read or written."""
    g = gen(19)
    k, v, table = make_cache(g, [64, 64, 64], 16, 2, 64, BF, fill=0.0)
    q = torch.randn((30, 4, 64), generator=g, device=DEV).to(BF)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    for lens, starts in (([1 << 30, -5, 64], [0, 10, 20, 30]), ([64, 64, 64], [-9, 1 << 30, 5, 30]),
                         ([64, 64, 64], [20, 10, 5, 0])):
        beside = torch.full((32, 4, 64), 7.0, dtype=BF, device=DEV)
        r.rope3d_paged_attention(q, k, v, table, ints(lens), ints(starts), out=beside[1:31])
        torch.cuda.synchronize()
        assert bool((beside[0] == 7).all()) and bool((beside[31] == 7).all()) and bool(beside.isfinite().all())
