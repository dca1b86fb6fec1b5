"""The operators around a paged cache as they are used together: a serving loop with
prompts, single tokens, forks and a compaction; captured graphs; other streams; calls side
by side; seeded random calls of the attention."""
from __future__ import annotations

import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import rope_rope3d_apply_gb300 as r  # noqa: E402
from tests.paged_reference import angles, attention64, check_attention, close, make_cache, rotate64  # noqa: E402

DEV = torch.device("cuda:0")
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    assert r.rope3d_testing_paged_wait_timeouts() == 0


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Serving:
    """A model's attention of a few layers over one cache, with a plain copy of what every
    sequence has been given."""

    def __init__(self, layers=2, heads=8, kv=2, dim=64, page=16, pages=80, seqs=6, width=12):
        self.layers, self.heads, self.kv, self.dim, self.page = layers, heads, kv, dim, page
        self.cache = torch.full((2 * layers, pages, page, kv, dim), float("nan"), dtype=BF, device=DEV)
        self.table = torch.full((seqs, width), -1, dtype=torch.int32, device=DEV)
        self.lens = [0] * seqs
        self.free = list(range(pages))
        random.Random(3).shuffle(self.free)
        self.freqs = torch.tensor([10000.0 ** (-j / (dim // 2)) for j in range(dim // 2)], device=DEV)
        self.given = [[[], []] for _ in range(seqs)]   # (k, v) [tokens, kv, dim] of each layer, a sequence
        self.k64 = [[[None, None] for _ in range(layers)] for _ in range(seqs)]
        self.g = gen(77)

    def room(self, s, new):
        for i in range(-(-self.lens[s] // self.page), -(-(self.lens[s] + new) // self.page)):
            self.table[s, i] = self.free.pop()

    def step(self, news):
        """Appends and attends news[s] tokens of every sequence, in every layer, and checks both."""
        for s, n in enumerate(news):
            self.room(s, n)
            self.lens[s] += n
        starts = [sum(news[:s]) for s in range(len(news) + 1)]
        lens, q_starts, total = ints(self.lens), ints(starts), starts[-1]
        for layer in range(self.layers):
            qkv = torch.randn((total, self.heads + 2 * self.kv, self.dim), generator=self.g, device=DEV).to(BF)
            q, k, v = qkv.split((self.heads, self.kv, self.kv), 1)
            kc, vc = self.cache[2 * layer], self.cache[2 * layer + 1]
            turned = r.rope3d_cache_append(q, k, v, kc, vc, self.table, lens, q_starts, freqs=self.freqs, pairing=r.PAIRS_HALVES)
            out = r.rope3d_paged_attention(turned, kc, vc, self.table, lens, q_starts, max_new=max(news))
            # what the cache should hold: rotations rounded as the cache is, so that the attention is
            # judged by itself; and the rotations themselves
            place = torch.cat([torch.arange(self.lens[s] - n, self.lens[s], device=DEV) for s, n in enumerate(news)])
            a = angles(place.expand(1, -1), self.freqs, (self.dim // 2,))
            close(turned, *rotate64(q, a, "halves", self.dim // 2))
            seq = torch.cat([torch.full((n,), s, device=DEV) for s, n in enumerate(news)])
            page = self.table.long()[seq, place // self.page]
            close(kc[page, place % self.page], *rotate64(k, a, "halves", self.dim // 2))
            for s, n in enumerate(news):
                kept = self.k64[s][layer]
                rows = slice(starts[s], starts[s + 1])
                new = kc[page[rows], place[rows] % self.page].clone(), v[rows].clone()
                self.k64[s][layer] = [x if old is None else torch.cat((old, x)) for old, x in zip(kept, new)]
                if n:
                    self.check(turned[rows], out[rows], s, layer)

    def check(self, q, out, s, layer):
        """One sequence against its keys and values as they were given, in a cache of one page."""
        k, v = self.k64[s][layer]
        want, bound, _, _ = attention64(q, k.unsqueeze(0), v.unsqueeze(0), ints([[0]]), [self.lens[s]], [0, q.shape[0]],
                                        self.dim ** -0.5, True, 0)
        close(out, want, bound)

    def fork(self, parent, child):
        fresh = self.free.pop()
        lens = ints(self.lens)
        r.rope3d_cache_fork(self.cache, self.table, lens, ints([parent]), ints([child]), ints([fresh]))
        self.lens[child] = self.lens[parent]
        assert lens.tolist() == self.lens
        self.k64[child] = [list(pair) for pair in self.k64[parent]]

    def end(self, s):
        self.lens[s] = 0
        self.k64[s] = [[None, None] for _ in range(self.layers)]

    def compact(self):
        self.table, used = r.rope3d_cache_compact(self.cache, self.table, ints(self.lens))
        self.free = list(range(int(used), self.cache.shape[1]))


def test_a_serving_loop():
    m = Serving()
    m.step([40, 0, 7, 0, 0, 0])            # two prompts
    m.step([1, 90, 1, 0, 0, 0])            # single tokens beside a third
    m.fork(1, 3)                           # 90 places: five full pages and a part of one
    m.fork(0, 4)
    m.step([1, 1, 1, 1, 30, 0])            # they part ways
    m.step([1] * 5 + [0])
    m.end(1)                               # its full pages live on in 3
    m.end(2)
    m.compact()
    assert len(m.free) > 60 and int((m.table >= 0).sum()) == sum(-(-n // 16) for n in m.lens)
    m.step([1, 0, 100, 1, 1, 3])           # into the pages that were freed
    m.compact()
    m.step([1] * 6)


def test_a_captured_step_follows_lengths():
    """One graph of append and attention; replays with other inputs, lengths and tables do
    what calls would."""
    g = gen(1)
    seqs, page, kv, dim, heads = 5, 16, 2, 128, 8
    cache = torch.zeros((2, 100, page, kv, dim), dtype=HF, device=DEV)
    for new in (1, 50):
        n = seqs * new
        table = torch.zeros((seqs, 20), dtype=torch.int32, device=DEV)
        lens = torch.zeros(seqs, dtype=torch.int32, device=DEV)
        qkv = torch.zeros((n, heads + 2 * kv, dim), dtype=HF, device=DEV)
        freqs = torch.rand(dim // 2, generator=g, device=DEV)

        def step():
            q, k, v = qkv.split((heads, kv, kv), 1)
            turned = r.rope3d_cache_append(q, k, v, cache[0], cache[1], table, lens, freqs=freqs)
            return turned, *r.rope3d_paged_attention(turned, cache[0], cache[1], table, lens, lse=True)

        lens.fill_(new)
        table.copy_(torch.arange(100, device=DEV).reshape(seqs, 20))
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        for most in (new, 100, 300):
            lens.copy_(torch.randint(new, most + 1, (seqs,), generator=g, device=DEV))
            table.copy_(torch.randperm(100, generator=g, device=DEV).reshape(seqs, 20))
            cache.copy_(torch.randn(cache.shape, generator=g, device=DEV))
            qkv.copy_(torch.randn(qkv.shape, generator=g, device=DEV))
            before = cache.clone()
            graph.replay()
            torch.cuda.synchronize()
            first, after = [x.clone() for x in got], cache.clone()
            cache.copy_(before)
            again = step()
            assert all(torch.equal(a, b) for a, b in zip(first, again)) and torch.equal(cache, after)


@pytest.mark.parametrize("new", [1, 200])
def test_two_graphs_and_their_workspaces(new):
    """Graphs captured one after the other and replayed side by side on two streams."""
    g = gen(2)
    graphs, results, wants = [], [], []
    for seed in range(2):
        k, v, table = make_cache(g, [3000, 900], 16, 2, 128, BF, fill=0.0)
        q = torch.randn((2 * new, 8, 128), generator=g, device=DEV).to(BF)
        lens = ints([3000, 900])
        call = lambda: r.rope3d_paged_attention(q, k, v, table, lens)  # noqa: E731
        wants.append(call())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(call())
        graphs.append((graph, q, k, v, table, lens))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (graph, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(results, wants))


def test_streams_by_argument_and_dropped_inputs():
    """Calls behind a delay on another stream, whose inputs the caller drops at once."""
    g = gen(3)
    normal = lambda *s: torch.randn(s, generator=g, device=DEV).to(BF)  # noqa: E731
    k, v, table = make_cache(g, [400, 77], 16, 2, 64, BF, fill=0.0)
    both = torch.stack((k, v))
    lens, freqs = ints([400, 77]), torch.rand(32, generator=g, device=DEV)
    q, pos = normal(60, 4, 64), torch.arange(60, device=DEV)
    new_k, new_v, starts = normal(60, 2, 64), normal(60, 2, 64), ints([0, 50, 60])
    zero, one, page = ints([0]), ints([1]), ints([int(k.shape[0]) - 1])

    def appended(q, **kw):
        c = both.clone()
        torch.cuda.synchronize()
        out = r.rope3d_cache_append(q, new_k.clone(), new_v.clone(), c[0], c[1], table.clone(), lens.clone(), starts.clone(), freqs=freqs.clone(), **kw)
        return out, c

    def forked(q, **kw):
        c, t, n = both.clone(), table.clone(), lens.clone()
        torch.cuda.synchronize()
        r.rope3d_cache_fork(c, t, n, zero.clone(), one.clone(), page.clone(), **kw)
        return c, t, n

    calls = {
        "axes": lambda q, **kw: r.rope3d_apply_axes(q, None, pos.clone(), freqs.clone(), **kw)[:1],
        "append": appended,
        "attention": lambda q, **kw: r.rope3d_paged_attention(q, k.clone(), v.clone(), table.clone(), lens.clone(), starts.clone(), lse=True, **kw),
        "fork": forked,
        "compact": lambda q, **kw: r.rope3d_cache_compact(both.clone(), table.clone(), lens.clone(), **kw),
    }
    side = torch.cuda.Stream()
    for name, call in calls.items():
        want = call(q)
        x = q.clone()
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(50_000_000)
        out = call(x, stream=side)
        del x
        trash = [torch.full((1 << n,), -1.0, dtype=BF, device=DEV) for n in range(4, 20) for _ in range(4)]
        torch.cuda.synchronize()
        del trash
        assert all(torch.equal(a, b) for a, b in zip(out, want)), name


def test_calls_on_two_streams_at_once():
    g = gen(4)
    work = []
    for i in range(4):
        lens = [1000 + 500 * i, 90]
        k, v, table = make_cache(g, lens, 16, 2, 128, HF, fill=0.0)
        q = torch.randn((2 * (1 + 90 * (i % 2)), 8, 128), generator=g, device=DEV).to(HF)
        work.append((q, k, v, table, ints(lens)))
    want = [r.rope3d_paged_attention(*w) for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(10):
        got = []
        for w, s in zip(work, streams):
            with torch.cuda.stream(s):
                got.append(r.rope3d_paged_attention(*w))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_given_outputs_and_workspace():
    g = gen(5)
    k, v, table = make_cache(g, [3000], 16, 4, 64, BF, fill=0.0)
    q, lens = torch.randn((1, 8, 64), generator=g, device=DEV).to(BF), ints([3000])
    want, want_lse = r.rope3d_paged_attention(q, k, v, table, lens, lse=True)
    out, lse, ws = torch.empty_like(q), torch.empty((1, 8), device=DEV), torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    got = r.rope3d_paged_attention(q, k, v, table, lens, out=out, lse=lse, workspace=ws)
    assert got[0] is out and got[1] is lse and torch.equal(out, want) and torch.equal(lse, want_lse)
    with pytest.raises(r.Rope3dError, match="ERR_SCRATCH"):
        r.rope3d_paged_attention(q, k, v, table, lens, workspace=ws[:256])
    with pytest.raises(r.Rope3dError, match="ERR_DEVICE"):
        r.rope3d_paged_attention(q, k, v, table, lens.cpu())
    with pytest.raises(r.Rope3dError, match="ERR_ALIAS"):
        r.rope3d_paged_attention(q, k, v, table, lens, out=q)


@pytest.mark.parametrize("seed", range(40))
def test_random_attention(seed):
    """Sizes, layouts, masks and hints by chance."""
    rnd, g = random.Random(seed), gen(1000 + seed)
    kv, group = rnd.choice((1, 2, 3, 4)), rnd.choice((1, 1, 2, 3, 4, 5, 7, 8, 16, 20))
    dim = rnd.choice((8, 16, 24, 40, 64, 64, 72, 104, 128, 128, 136, 192, 256))
    page = rnd.choice((1, 2, 3, 8, 8, 16, 16, 24, 32, 40, 64, 128, 256))
    seqs = rnd.randint(1, 9)
    most = rnd.choice((1, 1, 3, 60, 200))
    new = [rnd.choice((0, 1, rnd.randint(0, most), most)) for _ in range(seqs)]
    new[0] = max(new[0], 1)
    lens = [max(0, n + rnd.choice((0, 0, rnd.randint(0, 40), rnd.randint(0, 900), -rnd.randint(0, n)))) for n in new]
    dtype, layout = rnd.choice((BF, HF)), rnd.choice(("places", "heads", "joint"))
    k, v, table = make_cache(g, lens, page, kv, dim, dtype, layout=layout)
    starts = [sum(new[:i]) for i in range(seqs + 1)]
    q = torch.randn((starts[-1] + rnd.choice((0, 0, 5)), kv * group, dim), generator=g, device=DEV).to(dtype)
    absent = rnd.random() < 0.3
    if absent:
        for _ in range(4):
            table[rnd.randrange(seqs), rnd.randrange(table.shape[1])] = rnd.choice((-1, 1 << 29))
    check_attention(r, q, k, v, table, lens, starts, scale=rnd.choice((None, 0.05, 1.0)), causal=rnd.random() < 0.7,
                    window=rnd.choice((0, 0, rnd.randint(1, 300))), absent=absent, max_new=rnd.choice((0, 0, 1, 30, most)))
