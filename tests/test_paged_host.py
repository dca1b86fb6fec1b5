"""Host-side checks of the operators around a paged cache (no GPU): what they refuse, their
workspaces, the binding's own checks, and the arithmetic that divides the attention."""
from __future__ import annotations

import ctypes
import random

import pytest

import rope_rope3d_apply_gb300 as r


@pytest.fixture(scope="module", autouse=True)
def lib():
    from rope_rope3d_apply_gb300 import build

    build.build()
    return r.load_library()


MB = 1 << 20
BATCH = dict(page_table=100 * MB, seq_lens=101 * MB, q_starts=102 * MB, seqs=3, table_width=5, table_stride=5, pages=12, page_size=16)


def cases(check, base, good, bad):
    for change in good:
        assert check(**{**base, **change}) == "OK", change
    for change, status in bad:
        assert check(**{**base, **change}) == status, change


def test_axes():
    base = dict(q=1 * MB, k=2 * MB, q_out=3 * MB, k_out=4 * MB, positions=5 * MB, freqs=6 * MB, tokens=10, q_heads=4, k_heads=2,
                head_dim=64, q_token_stride=256, q_head_stride=64, k_token_stride=128, k_head_stride=64, q_out_token_stride=256,
                q_out_head_stride=64, k_out_token_stride=128, k_out_head_stride=64, positions_stride=10, section0=8, section1=12,
                section2=12, dtype=r.BF16, position_type=r.POSITIONS_I64, pairing=r.PAIRS_HALVES, inverse=0)
    third = dict(q=1 * MB, k=1 * MB + 512, k_heads=4, q_token_stride=768, k_token_stride=768)   # thirds of [tokens, 3, 4, 64]
    cases(r.rope3d_apply_axes_check, base, [
        {}, dict(k=0, k_out=0), dict(dtype=r.F32), dict(dtype=r.F16, position_type=r.POSITIONS_F32), dict(section1=0, section2=0),
        dict(section0=0), dict(q_token_stride=0, q_head_stride=0), dict(q_token_stride=64, q_head_stride=640), dict(q_out=1 * MB),
        dict(q=1 * MB + 2, q_out=3 * MB + 2), dict(k_out_token_stride=64, k_out_head_stride=640), dict(k=1 * MB),
        dict(third, q_out=1 * MB, k_out=1 * MB + 512, q_out_token_stride=768, k_out_token_stride=768), dict(tokens=1, positions_stride=0),
        dict(head_dim=4096, q_head_stride=4096, q_token_stride=16384, k_head_stride=4096, k_token_stride=8192, q_out=30 * MB,
             k_out=40 * MB, q_out_head_stride=4096, q_out_token_stride=16384, k_out_head_stride=4096, k_out_token_stride=8192),
    ], [
        (dict(q=0), "ERR_NULL"), (dict(q_out=0), "ERR_NULL"), (dict(k=0), "ERR_NULL"), (dict(k_out=0), "ERR_NULL"),
        (dict(positions=0), "ERR_NULL"), (dict(freqs=0), "ERR_NULL"), (dict(tokens=0), "ERR_SHAPE"), (dict(tokens=-1), "ERR_SHAPE"),
        (dict(q_heads=0), "ERR_SHAPE"), (dict(k_heads=0), "ERR_SHAPE"), (dict(head_dim=0), "ERR_SHAPE"), (dict(head_dim=62), "ERR_SHAPE"),
        (dict(head_dim=4098), "ERR_SHAPE"), (dict(section0=0, section1=0, section2=0), "ERR_SHAPE"), (dict(section0=-1), "ERR_SHAPE"),
        (dict(section0=9), "ERR_SHAPE"), (dict(head_dim=4096, section0=1025), "ERR_SHAPE"), (dict(dtype=7), "ERR_DTYPE"),
        (dict(position_type=3), "ERR_DTYPE"), (dict(pairing=2), "ERR_ARG"), (dict(q_token_stride=-1), "ERR_SHAPE"),
        (dict(q_out_head_stride=32), "ERR_SHAPE"), (dict(q_out_token_stride=0), "ERR_SHAPE"), (dict(q_out_token_stride=255), "ERR_SHAPE"),
        (dict(positions_stride=-1), "ERR_SHAPE"), (dict(q=1 * MB + 1), "ERR_ALIGN"), (dict(positions=5 * MB + 4), "ERR_ALIGN"),
        (dict(freqs=6 * MB + 2), "ERR_ALIGN"), (dict(q_out=1 * MB + 64), "ERR_ALIAS"), (dict(q_out=2 * MB), "ERR_ALIAS"),
        (dict(k_out=3 * MB + 128), "ERR_ALIAS"), (dict(q_out=5 * MB), "ERR_ALIAS"), (dict(k_out=6 * MB), "ERR_ALIAS"),
        (dict(q_out=1 * MB, q_token_stride=320), "ERR_ALIAS"), (dict(third, q_out=1 * MB, q_out_token_stride=768, k_out=1 * MB + 448,
                                                                 k_out_token_stride=768), "ERR_ALIAS"),
    ])


def append_base():
    return dict(BATCH, q=1 * MB, q_out=2 * MB, k=3 * MB, v=4 * MB, k_cache=20 * MB, v_cache=40 * MB, positions=5 * MB, freqs=6 * MB,
                invalid_count=7 * MB, tokens=9, q_heads=4, kv_heads=2, head_dim=64, q_token_stride=256, q_head_stride=64,
                q_out_token_stride=256, q_out_head_stride=64, k_token_stride=128, k_head_stride=64, v_token_stride=128,
                v_head_stride=64, k_page_stride=2048, k_slot_stride=128, k_cache_head_stride=64, v_page_stride=2048,
                v_slot_stride=128, v_cache_head_stride=64, positions_stride=9, section0=32, section1=0, section2=0, dtype=r.F16,
                position_type=r.POSITIONS_I32, pairing=r.PAIRS_INTERLEAVED)


def test_append():
    joint = dict(v_cache=20 * MB + 256, k_page_stride=4096, k_slot_stride=256, v_page_stride=4096, v_slot_stride=256)
    cases(r.rope3d_cache_append_check, append_base(), [
        {}, dict(q=0, q_out=0), dict(positions=0), dict(invalid_count=0), dict(q_starts=0), dict(freqs=0, q=0, q_out=0, positions=0),
        dict(q_out=1 * MB), joint, dict(k_slot_stride=64, k_cache_head_stride=1024), dict(page_size=1, k_page_stride=128),
        dict(k=4 * MB), dict(table_stride=1000), dict(dtype=r.F32),
    ], [
        (dict(k=0), "ERR_NULL"), (dict(v=0), "ERR_NULL"), (dict(k_cache=0), "ERR_NULL"), (dict(v_cache=0), "ERR_NULL"),
        (dict(q=0), "ERR_NULL"), (dict(q_out=0), "ERR_NULL"), (dict(page_table=0), "ERR_NULL"), (dict(seq_lens=0), "ERR_NULL"),
        (dict(freqs=0), "ERR_ARG"), (dict(freqs=0, q=0, q_out=0), "ERR_ARG"), (dict(seqs=0), "ERR_SHAPE"), (dict(pages=0), "ERR_SHAPE"),
        (dict(page_size=0), "ERR_SHAPE"), (dict(table_width=0), "ERR_SHAPE"), (dict(table_stride=4), "ERR_SHAPE"),
        (dict(table_width=1 << 27, table_stride=1 << 27), "ERR_SHAPE"), (dict(q_starts=0, tokens=10), "ERR_SHAPE"),
        (dict(tokens=0), "ERR_SHAPE"), (dict(kv_heads=0), "ERR_SHAPE"), (dict(section0=33), "ERR_SHAPE"), (dict(dtype=9), "ERR_DTYPE"),
        (dict(position_type=-1), "ERR_DTYPE"), (dict(pairing=5), "ERR_ARG"), (dict(k_slot_stride=64), "ERR_SHAPE"),
        (dict(v_page_stride=2047), "ERR_SHAPE"), (dict(v_cache=20 * MB), "ERR_ALIAS"), (dict(joint, v_cache=20 * MB + 128), "ERR_ALIAS"),
        (dict(k=20 * MB), "ERR_ALIAS"), (dict(q_out=3 * MB), "ERR_ALIAS"), (dict(q_out=1 * MB + 64), "ERR_ALIAS"),
        (dict(invalid_count=101 * MB), "ERR_ALIAS"), (dict(k_cache=100 * MB), "ERR_ALIAS"), (dict(seq_lens=101 * MB + 1), "ERR_ALIGN"),
        (dict(v_cache=40 * MB + 1), "ERR_ALIGN"), (dict(invalid_count=7 * MB + 2), "ERR_ALIGN"),
    ])


def attention_base(**kw):
    a = dict(BATCH, q=1 * MB, k_cache=20 * MB, v_cache=40 * MB, out=2 * MB, lse=3 * MB, tokens=9, q_heads=4, kv_heads=2, head_dim=64,
             q_token_stride=256, q_head_stride=64, out_token_stride=256, out_head_stride=64, lse_stride=4, k_page_stride=2048,
             k_slot_stride=128, k_cache_head_stride=64, v_page_stride=2048, v_slot_stride=128, v_cache_head_stride=64, window=0,
             max_new=0, workspace=200 * MB, workspace_bytes=100 * MB, scale=0.125, dtype=r.BF16, causal=1)
    a.update(kw)
    return a


def need(**kw):
    n = ctypes.c_int64()
    args = r._AttentionArgs(**attention_base(**kw))
    return r.STATUS[r.load_library().rope3d_paged_attention_workspace(ctypes.byref(args), ctypes.byref(n))], n.value


def test_attention():
    cases(r.rope3d_paged_attention_check, attention_base(), [
        {}, dict(lse=0), dict(causal=0), dict(window=1 << 40), dict(max_new=1), dict(max_new=1 << 40), dict(q_starts=0),
        dict(k_cache=40 * MB), dict(k_cache_head_stride=0, v_cache_head_stride=0), dict(page_size=5), dict(scale=1e-30),
        dict(head_dim=256, q_heads=2, kv_heads=1, q_head_stride=256, q_token_stride=512, out_head_stride=256, out_token_stride=512),
        dict(out_token_stride=64, out_head_stride=640), dict(workspace_bytes=need()[1]), dict(head_dim=8),
    ], [
        (dict(q=0), "ERR_NULL"), (dict(k_cache=0), "ERR_NULL"), (dict(v_cache=0), "ERR_NULL"), (dict(out=0), "ERR_NULL"),
        (dict(page_table=0), "ERR_NULL"), (dict(seq_lens=0), "ERR_NULL"), (dict(workspace=0), "ERR_NULL"), (dict(tokens=0), "ERR_SHAPE"),
        (dict(q_heads=5), "ERR_SHAPE"), (dict(q_heads=1), "ERR_SHAPE"), (dict(kv_heads=0), "ERR_SHAPE"), (dict(head_dim=0), "ERR_SHAPE"),
        (dict(head_dim=60), "ERR_SHAPE"), (dict(head_dim=264), "ERR_SHAPE"), (dict(tokens=1 << 28, q_heads=1 << 12), "ERR_SHAPE"),
        (dict(dtype=r.F32), "ERR_DTYPE"), (dict(scale=0.0), "ERR_ARG"), (dict(scale=-1.0), "ERR_ARG"), (dict(scale=float("inf")), "ERR_ARG"),
        (dict(scale=float("nan")), "ERR_ARG"), (dict(scale=1e-60), "ERR_ARG"), (dict(causal=2), "ERR_ARG"), (dict(window=-1), "ERR_ARG"),
        (dict(max_new=-1), "ERR_ARG"), (dict(q=1 * MB + 2), "ERR_ALIGN"), (dict(out=2 * MB + 8), "ERR_ALIGN"),
        (dict(k_slot_stride=132), "ERR_ALIGN"), (dict(v_cache=40 * MB + 4), "ERR_ALIGN"), (dict(lse=3 * MB + 2), "ERR_ALIGN"),
        (dict(workspace=200 * MB + 128), "ERR_ALIGN"), (dict(out_head_stride=56), "ERR_SHAPE"), (dict(lse_stride=3), "ERR_SHAPE"),
        (dict(out=1 * MB), "ERR_ALIAS"), (dict(out=20 * MB), "ERR_ALIAS"), (dict(lse=2 * MB), "ERR_ALIAS"), (dict(out=200 * MB), "ERR_ALIAS"),
        (dict(workspace=20 * MB), "ERR_ALIAS"), (dict(workspace_bytes=need()[1] - 1), "ERR_SCRATCH"), (dict(q_starts=0, tokens=10), "ERR_SHAPE"),
    ])


def test_workspaces():
    """No device is needed for the sizes; they do not shrink with more tokens, and are
    bounded whatever the lengths are."""
    assert need()[0] == "OK" and need(workspace=0, workspace_bytes=0)[0] == "OK" and need(q=0)[0] == "ERR_NULL"
    sizes = [need(tokens=n, max_new=n, table_width=1 << 16, table_stride=1 << 16)[1] for n in (3, 9, 30, 300, 30000)]
    assert all(n % 256 == 0 for n in sizes) and max(sizes) < 64 * MB
    big = [need(tokens=1 << 20, head_dim=d, q_head_stride=256, q_token_stride=1024, out_head_stride=256, out_token_stride=1024, lse=0,
                out=1 << 40, workspace=0, k_page_stride=1 << 14, k_slot_stride=512, k_cache_head_stride=256, v_page_stride=1 << 14,
                v_slot_stride=512, v_cache_head_stride=256)[1] for d in (64, 128, 256)]
    assert big[0] <= big[1] <= big[2] < 64 * MB


def cache_base(**kw):
    return dict(dict(cache=10 * MB, page_table=100 * MB, seq_lens=101 * MB, planes=4, pages=12, page_bytes=4096, plane_stride=12 * 4096,
                     page_stride=4096, seqs=6, table_width=5, table_stride=5, page_size=16), **kw)


BAD_CACHE = [
    (dict(cache=0), "ERR_NULL"), (dict(page_table=0), "ERR_NULL"), (dict(seq_lens=0), "ERR_NULL"), (dict(planes=0), "ERR_SHAPE"),
    (dict(pages=0), "ERR_SHAPE"), (dict(pages=(1 << 20) + 1), "ERR_SHAPE"), (dict(page_bytes=0), "ERR_SHAPE"), (dict(seqs=0), "ERR_SHAPE"),
    (dict(table_width=0), "ERR_SHAPE"), (dict(table_stride=4), "ERR_SHAPE"), (dict(page_size=0), "ERR_SHAPE"),
    (dict(page_stride=4080), "ERR_SHAPE"), (dict(plane_stride=4096), "ERR_SHAPE"), (dict(cache=10 * MB + 8), "ERR_ALIGN"),
    (dict(page_bytes=4088), "ERR_ALIGN"), (dict(page_stride=4104), "ERR_SHAPE"), (dict(seq_lens=101 * MB + 2), "ERR_ALIGN"),
    (dict(cache=100 * MB), "ERR_ALIAS"),
]


def test_fork():
    base = cache_base(parents=102 * MB, children=103 * MB, new_pages=104 * MB, invalid_count=105 * MB, forks=3)
    cases(r.rope3d_cache_fork_check, base, [
        {}, dict(invalid_count=0), dict(planes=1, plane_stride=0), dict(pages=1, planes=1, page_stride=0), dict(parents=103 * MB),
        dict(plane_stride=4096, page_stride=4 * 4096),
    ], BAD_CACHE + [
        (dict(parents=0), "ERR_NULL"), (dict(children=0), "ERR_NULL"), (dict(new_pages=0), "ERR_NULL"), (dict(forks=0), "ERR_SHAPE"),
        (dict(parents=100 * MB), "ERR_ALIAS"), (dict(invalid_count=102 * MB), "ERR_ALIAS"), (dict(children=10 * MB), "ERR_ALIAS"),
        (dict(seq_lens=100 * MB + 4), "ERR_ALIAS"),   # (both are written)
    ])


def test_compact():
    base = cache_base(table_out=102 * MB, used=103 * MB, table_out_stride=5, reserve=0, workspace=200 * MB, workspace_bytes=MB)
    cases(r.rope3d_cache_compact_check, base, [
        {}, dict(table_out=100 * MB), dict(reserve=1), dict(table_out_stride=9),
    ], BAD_CACHE + [
        (dict(table_out=0), "ERR_NULL"), (dict(used=0), "ERR_NULL"), (dict(workspace=0), "ERR_NULL"), (dict(reserve=-1), "ERR_SHAPE"),
        (dict(table_out_stride=4), "ERR_SHAPE"), (dict(table_out=100 * MB, table_out_stride=6), "ERR_ALIAS"),
        (dict(table_out=100 * MB + 4), "ERR_ALIAS"), (dict(used=101 * MB), "ERR_ALIAS"), (dict(workspace=200 * MB + 16), "ERR_ALIGN"),
        (dict(workspace_bytes=255), "ERR_SCRATCH"), (dict(workspace=10 * MB), "ERR_ALIAS"), (dict(used=102 * MB + 8), "ERR_ALIAS"),
    ])


def test_null_arguments():
    lib = r.load_library()
    n = ctypes.c_int64()
    for name in ("rope3d_apply_axes", "rope3d_cache_append", "rope3d_paged_attention", "rope3d_cache_fork", "rope3d_cache_compact"):
        assert r.STATUS[getattr(lib, name)(None, None)] == "ERR_NULL"
        assert r.STATUS[getattr(lib, name + "_check")(None, 0)] == "ERR_NULL"
    for name in ("rope3d_paged_attention_workspace", "rope3d_cache_compact_workspace"):
        assert r.STATUS[getattr(lib, name)(None, ctypes.byref(n))] == "ERR_NULL"
        assert r.STATUS[getattr(lib, name)(None, None)] == "ERR_NULL"
    assert r.STATUS[lib.rope3d_testing_paged_wait_timeouts(None, 0)] == "ERR_NULL"


def test_what_the_binding_refuses():
    torch = pytest.importorskip("torch")
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q, k, c, t, n, f = z(4, 4, 32), z(4, 2, 32), z(5, 8, 2, 32), i(2, 3), i(2), z(16, dt=torch.float32)
    pos = torch.zeros((3, 4), dtype=torch.int64)
    refused = (ValueError, TypeError, r.Rope3dError)
    axes, append, attend = r.rope3d_apply_axes, r.rope3d_cache_append, r.rope3d_paged_attention
    for call in (
        lambda: axes(q, k, pos, f.double()), lambda: axes(q, k, pos[:, :3], f), lambda: axes(q, k, pos.half(), f),
        lambda: axes(q, k, pos[:2], f, (4, 4, 8)), lambda: axes(q, k, pos, f, (4, 4, 4)), lambda: axes(q, k, pos, f, (4, 4, 4, 4)),
        lambda: axes(q, k.float(), pos, f), lambda: axes(q, k[:3], pos, f), lambda: axes(q[0], k, pos, f),
        lambda: axes(q, k, pos, f, q_out=z(4, 4, 30)), lambda: axes(q, z(4, 32, 2).transpose(1, 2), pos, f), lambda: axes(q, k, pos, f[::2]),
        lambda: axes(q, k, pos, f),   # host memory
        lambda: append(q, k, k, c, c, t.long(), n, freqs=f), lambda: append(q, k, k, c, c, t, n.long(), freqs=f),
        lambda: append(q, k, k, c, z(5, 8, 2, 16), t, n, freqs=f), lambda: append(q, k, z(4, 1, 32), c, c, t, n, freqs=f),
        lambda: append(q, k, k, c, c, t[0], n, freqs=f), lambda: append(q, k, k, c, c, t, n, i(2), freqs=f),
        lambda: append(q, k, k, c, c, t, n), lambda: append(None, k, k, c, c, t, n, positions=pos),
        lambda: append(None, k, k, c, c, t, n, sections=(16,)), lambda: append(q, k, k, c, c, t, n, freqs=f, invalid_count=n),
        lambda: append(q, k, k, c, c.clone(), t, n, freqs=f),   # host memory
        lambda: attend(q, c, c.half(), t, n), lambda: attend(q, c, z(5, 8, 2, 16), t, n), lambda: attend(q, c[0], c[0], t, n),
        lambda: attend(q, c, c, t, n, out=z(4, 4, 16)), lambda: attend(q, c, c, t, n, lse=z(4, 4)), lambda: attend(q, c, c, t, i(3)),
        lambda: attend(q, c, c, t, n, i(2)), lambda: attend(q.float(), c.float(), c.float(), t, n), lambda: attend(q, c, c, t, n, scale=-1.0),
        lambda: attend(q, c, c, t, n),   # host memory
        lambda: r.rope3d_cache_fork(c, t, n, n, n, n, page_size=8), lambda: r.rope3d_cache_fork(z(2, 5, 8, 4)[:, :, ::2], t, n, n, n, n),
        lambda: r.rope3d_cache_fork(z(2, 5, 8, 32), t, n, n, i(3), n), lambda: r.rope3d_cache_compact(z(2, 5, 8, 32), t, i(3)),
        lambda: r.rope3d_cache_compact(z(2, 5, 8, 32), t, n, table_out=i(2, 2)), lambda: r.rope3d_cache_compact(z(2, 5, 8, 32), t, n, used=n),
    ):
        with pytest.raises(refused):
            call()


# ---- how the attention divides its work: the line's arithmetic, as the kernels have it -------


def tile(rows, keys, group, n, length, window, causal, t):
    """Blocks of tile t, from its rows."""
    last, past = min(n * group, (t + 1) * rows) - 1, length - n
    k1 = min(max(past + last // group + 1, 0), length) if causal else length
    k0 = min(max(past + t * rows // group - window + 1, 0), k1) if window else 0
    return max(-(-k1 // keys) - k0 // keys, 1) if k1 > k0 else 1


def floors(n, d):
    q = n // d
    return q * (q - 1) // 2 * d + q * (n - q * d)


def cost_before(rows, keys, group, n, length, window, causal, t):
    """The kernels' closed form of the blocks of tiles 0 .. t - 1 (without the constant a tile)."""
    d, past = keys * group // rows, length - n
    total = max(-(-length // keys), 1) * t
    if causal:
        a = (group * (past + keys) + rows - 1) // rows
        ones = min(max(d - a, 0), t)
        total = ones + (floors(a + t, d) - floors(a + ones, d) if t > ones else 0)
    c = group * (past - window + 1) // rows
    if window and c + t > 0:
        total -= floors(c + t, d) - floors(max(c, 0), d)
    return total


@pytest.mark.parametrize("rows,keys", [(16, 64), (128, 128), (256, 256)])
def test_the_cost_of_tiles_in_closed_form(rows, keys):
    rnd = random.Random(rows)
    for _ in range(3000):
        group, n = rnd.choice((1, 2, 3, 5, 6, 7, 8, 12, 16, 40, 200)), rnd.choice((1, 2, 5, rnd.randint(1, 700)))
        length = rnd.choice((0, n, max(0, n - rnd.randint(0, 50)), n + rnd.randint(0, 3000), rnd.randint(0, n)))
        window, causal, sum_ = rnd.choice((0, 0, 1, 5, 64, rnd.randint(1, 2000))), rnd.random() < 0.6, 0
        for t in range(-(-n * group // rows)):
            assert cost_before(rows, keys, group, n, length, window, causal, t) == sum_
            sum_ += tile(rows, keys, group, n, length, window, causal, t)


def test_every_block_belongs_to_one_part():
    """A line of items cut into parts: each item's blocks once, in order, and its parts as the
    joining kernel finds them."""
    rnd = random.Random(1)
    for _ in range(400):
        constant, parts = rnd.randint(0, 4), rnd.choice((1, 2, 7, 76, 152))
        items = [rnd.choice((1, 2, rnd.randint(1, 90))) for _ in range(rnd.randint(1, 40))]
        begins, total = [], 0
        for blocks in items:
            begins.append(total)
            total += blocks + constant
        cuts = [total * p // parts for p in range(parts + 1)]
        done = [[] for _ in items]
        for p in range(parts):
            at, left = cuts[p], cuts[p + 1] - cuts[p]
            i = max((j for j, b in enumerate(begins) if b <= at), default=0)
            while left > 0 and i < len(items):
                off, cost = at - begins[i], items[i] + constant
                take = min(left, cost - off)
                first, last = max(off - constant, 0), max(off + take - constant, 0)
                if last > first:
                    done[i].append((p, first, last, first > 0))
                at, left, i = at + take, left - take, i + 1
        for i, blocks in enumerate(items):
            assert [b for _, a, z, _ in done[i] for b in range(a, z)] == list(range(blocks))
            if len(done[i]) > 1:   # as the joining kernel lists them
                first = begins[i] + constant
                heads = [p for p in range(parts) if first < cuts[p] < begins[i] + blocks + constant and cuts[p] < cuts[p + 1]]
                lead = max(p for p in range(parts) if cuts[p] <= first and cuts[p] < cuts[p + 1])
                assert [p for p, *_ in done[i]] == [lead] + heads
                assert [h for *_, h in done[i]] == [False] + [True] * len(heads)
