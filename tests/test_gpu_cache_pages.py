"""rope3d_cache_fork and rope3d_cache_compact against plain loops on the host."""
from __future__ import annotations

import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import rope_rope3d_apply_gb300 as r  # noqa: E402

DEV = torch.device("cuda:0")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def make(seed, planes, pages, page, row, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn((planes, pages, page, *row), generator=g, device=DEV).to(dtype)


FORKS = [
    # lens, (parent, child) pairs, page, planes, row
    ([5], [(0, 1)], 16, 1, (1, 8)),
    ([33, 64, 7, 0, 16], [(0, 5), (1, 6), (1, 7), (2, 8), (3, 9), (4, 10), (0, 11)], 16, 3, (2, 64)),
    ([100, 900], [(1, i) for i in range(2, 40)], 24, 5, (4, 40)),
    ([3000], [(0, 1), (0, 2)], 256, 2, (8, 128)),
]


@pytest.mark.parametrize("case", range(len(FORKS)))
def test_fork(case):
    lens, forks, page, planes, row = FORKS[case]
    rnd = random.Random(case)
    held = [n // page + 1 for n in lens]
    pages = sum(held) + len(forks) + 5
    order = rnd.sample(range(pages), pages)
    width, seqs = max(held) + 1, len(lens) + len(forks) + 1
    table = [[rnd.randint(-3, pages) for _ in range(width)] for _ in range(seqs)]
    for s, n in enumerate(held):
        table[s][:n] = [order.pop() for _ in range(n)]
    new = [order.pop() for _ in forks]
    lens = lens + [rnd.randint(0, 50) for _ in range(seqs - len(lens))]
    cache = make(case, planes, pages, page, row)
    want = cache.clone()
    t, n, bad = ints(table), ints(lens), ints([0])
    r.rope3d_cache_fork(cache, t, n, ints([p for p, _ in forks]), ints([c for _, c in forks]), ints(new), invalid_count=bad)
    for (p, c), fresh in zip(forks, new):
        whole = lens[p] // page
        if lens[p] % page:
            want[:, fresh] = want[:, table[p][whole]]
        table[c][:whole] = table[p][:whole]
        table[c][whole] = fresh
        lens[c] = lens[p]
    assert t.tolist() == table and n.tolist() == lens and torch.equal(cache, want) and int(bad) == 0


def test_forks_that_cannot_be():
    """Numbers out of range, a parent that is its child, a last page that is not there, a full
    row: nothing changes, and each is counted; the good one among them is made."""
    cache = make(9, 2, 10, 4, (1, 16))
    table = [[0, 1, 2], [3, -1, 4], [5, 6, 7], [8, 8, 8]]
    lens = [6, 5, 12, 2]
    forks = [(-1, 3, 9), (4, 3, 9), (0, -1, 9), (0, 4, 9), (0, 3, -1), (0, 3, 10), (0, 0, 9), (1, 3, 9), (2, 3, 9)]
    t, n, bad, was = ints(table), ints(lens), ints([0]), cache.clone()
    r.rope3d_cache_fork(cache, t, n, *(ints(list(x)) for x in zip(*forks)), invalid_count=bad)
    assert t.tolist() == table and n.tolist() == lens and torch.equal(cache, was) and int(bad) == len(forks)
    r.rope3d_cache_fork(cache, t, n, *(ints(list(x)) for x in zip(*forks, (0, 3, 9))), invalid_count=None)
    assert t.tolist()[3] == [0, 9, 8] and n.tolist()[3] == 6
    assert torch.equal(cache[:, 9], was[:, 1])
    was[:, 9] = was[:, 1]
    assert torch.equal(cache, was)


def plain_compact(cache, table, lens, page, reserve):
    planes, pages = cache.shape[:2]
    held = [row[:min(len(row), -(-(n + reserve) // page))] if n > 0 else [] for row, n in zip(table, lens)]
    used = sorted({p for row in held for p in row if 0 <= p < pages})
    count, there = len(used), set(used)
    to = dict(zip([p for p in used if p >= count], [p for p in range(count) if p not in there]))
    want = cache.clone()
    for a, b in to.items():
        want[:, b] = cache[:, a]
    out = [[(to.get(p, p) if 0 <= p < pages else -1) for p in row] + [-1] * (len(full) - len(row)) for row, full in zip(held, table)]
    return want, out, count


COMPACTS = [
    # seqs, pages, longest, page, planes, row, reserve
    (1, 1, 3, 4, 1, (1, 8), 0),
    (3, 31, 40, 4, 2, (1, 24), 0),
    (7, 64, 60, 8, 3, (2, 64), 1),
    (40, 700, 200, 16, 2, (1, 40), 0),
    (300, 5000, 500, 64, 1, (1, 8), 0),
    (33, 33000, 900, 1, 1, (1, 8), 0),
    (64, 400000, 900, 1, 1, (1, 8), 5),
    (5, 1 << 20, 4000, 1, 1, (1, 8), 0),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("case", range(len(COMPACTS)))
def test_compact(case, full, in_place):
    seqs, pages, longest, page, planes, row, reserve = COMPACTS[case]
    rnd = random.Random(case)
    lens = [rnd.choice((0, 1, page, rnd.randint(0, longest), longest)) for _ in range(seqs)]
    width = -(-longest // page) + 2
    table = [[rnd.randint(-2, pages + 2) for _ in range(width)] for _ in range(seqs)]   # shared and absent pages among them
    if full:   # every page in use
        lens, width = lens + [pages * page], max(width, pages)
        if width > 40000:
            pytest.skip("no table of that width on the host")
        table = [row_ + [-1] * (width - len(row_)) for row_ in table] + [rnd.sample(range(pages), pages) + [-1] * (width - pages)]
    cache = make(case, planes, pages, page, row, torch.float16)
    want, out, count = plain_compact(cache, table, lens, page, reserve)
    t = ints(table)
    got, used = r.rope3d_cache_compact(cache, t, ints(lens), reserve=reserve, table_out=t if in_place else None)
    assert int(used) == count and got.tolist() == out
    assert torch.equal(cache.view(torch.int16), want.view(torch.int16))
    assert in_place or t.tolist() == table


def test_planes_of_a_strided_cache():
    """Pages beside others' in one buffer: what lies between them keeps its values."""
    base = make(20, 3, 40, 8, (2, 16))
    cache = base[::2, 1::3]
    pages = cache.shape[1]
    was = base.clone()
    table, lens = [[12, 3, 7], [9, 3, 0]], [20, 9]
    want, out, count = plain_compact(cache, table, lens, 8, 0)
    got, used = r.rope3d_cache_compact(cache, ints(table), ints(lens))
    assert pages == 13 and int(used) == count and got.tolist() == out and torch.equal(cache, want)
    was[::2, 1::3] = want
    assert torch.equal(base, was)
    r.rope3d_cache_fork(cache, t := ints([[4, 5], [0, 0]]), n := ints([9, 0]), ints([0]), ints([1]), ints([11]))
    assert t.tolist() == [[4, 5], [4, 11]] and n.tolist() == [9, 9]
    was[::2, 1::3][:, 11] = was[::2, 1::3][:, 5]
    assert torch.equal(base, was)


def test_offsets_past_32_bits():
    cache = torch.zeros((2, 40000, 64, 4, 128), dtype=torch.float16, device=DEV)   # 5.2 GB
    cache[:, -1], cache[1, -2] = 3.0, 5.0
    got, used = r.rope3d_cache_compact(cache, ints([[39999, 39998]]), ints([100]))
    assert got.tolist() == [[1, 0]] and int(used) == 2
    assert bool((cache[:, 1] == 3).all()) and bool((cache[1, 0] == 5).all()) and bool((cache[0, 0] == 0).all())
