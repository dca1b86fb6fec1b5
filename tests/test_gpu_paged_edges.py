"""The operators around a paged cache at the ends of their ranges: places far below zero and far
up, long lines of key blocks, windows over long sequences, rows whose scores are all -infinity."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import rope_rope3d_apply_gb300 as r  # noqa: E402
from tests.paged_reference import attention64, check_attention, close, make_cache, rotate64  # noqa: E402

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


@pytest.mark.parametrize("length", [0, 9, 1 << 25])
def test_append_at_places_that_no_float_has(length):
    """A sequence shorter than its many new tokens has places below -2^24, a long one above 2^24; q is
    rotated by them although they have no page (a table of absent pages: the cache stays as it is)."""
    tokens = (1 << 24) + 67
    g = gen(1)
    q = torch.randn((tokens, 1, 2), generator=g, device=DEV)
    k = torch.zeros((1, 1, 2), device=DEV).expand(tokens, 1, 2)
    k_cache, v_cache = torch.full((2, 1, 1 << 15, 1, 2), 9.0, device=DEV)
    table = torch.full((1, 1 << 10), -1, dtype=torch.int32, device=DEV)
    bad = ints([0])
    out = r.rope3d_cache_append(q, k, k, k_cache, v_cache, table, ints([length]), freqs=torch.full((1,), 0.5, device=DEV), invalid_count=bad)
    assert int(bad) == tokens and bool((k_cache == 9).all()) and bool((v_cache == 9).all())
    at = torch.cat((torch.arange(200, device=DEV), torch.arange(tokens // 2, tokens // 2 + 200, device=DEV),
                    torch.arange(tokens - 200, tokens, device=DEV)))
    place = length - tokens + at
    close(out[at], *rotate64(q[at], 0.5 * place.double().unsqueeze(1), "interleaved", 1), f"length {length}")


# ---- attention --------------------------------------------------------------------


# kernels by a hint: few rows, tiles of one block, tiles of pairs
HINTS = {"few": 1, "tile": 16, "pair": 0}


@pytest.mark.parametrize("kernel", list(HINTS))
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,lens,window", [([700, 33], [40000, 17000], 1000), ([40], [150000], (1 << 17) + 5), ([300], [20000], 19990)])
def test_windows_over_long_sequences(kernel, causal, new, lens, window):
    """Heads of a group times places past 2^17: the line's costs are taken in 64 bits, with a window."""
    g = gen(2)
    k, v, table = make_cache(g, lens, 16, 1, 72, HF)
    starts = [0, *(sum(new[:i + 1]) for i in range(len(new)))]
    q = torch.randn((starts[-1], 8, 72), generator=g, device=DEV).to(HF)
    check_attention(r, q, k, v, table, lens, starts, causal=causal, window=window, max_new=HINTS[kernel])
    assert r.rope3d_paged_attention_last_kernel() == {"few": 1, "tile": 2, "pair": 3}[kernel]


@pytest.mark.parametrize("new,kernel", [(1, 1), (17, 2), (140, 3)])
def test_long_lines(new, kernel):
    """More than 2^21 blocks of keys in one call: 64 sequences of 1,100,000 places that share a few pages."""
    g = gen(3)
    seqs, kv, dim, page, length = 64, 8, 72, 64, 1100003
    k, v = (torch.randn((600, page, kv, dim), generator=g, device=DEV).to(BF) for _ in range(2))
    table = torch.randint(0, 600, (seqs, -(-length // page)), generator=g, device=DEV, dtype=torch.int32)
    q = torch.randn((seqs * new, kv, dim), generator=g, device=DEV).to(BF)
    out, lse = r.rope3d_paged_attention(q, k, v, table, ints([length] * seqs), ints([new * s for s in range(seqs + 1)]), max_new=new, lse=True)
    assert r.rope3d_paged_attention_last_kernel() == kernel
    for s in (0, 31, 63):
        rows = slice(s * new, (s + 1) * new)
        want = attention64(q[rows], k, v, table[s:s + 1], [length], [0, new], dim ** -0.5, True, 0)
        close(out[rows], *want[:2], f"sequence {s}")
        close(lse[rows], *want[2:], f"lse of sequence {s}")


@pytest.mark.parametrize("kernel", list(HINTS))
def test_scores_of_minus_infinity(kernel):
    """Keys whose scores are -infinity weigh nothing: the bits of the same call with their pages absent. A row
    whose scores are all -infinity gives zeros, and -infinity for the log of their sum."""
    g = gen(4)
    lens, new, page = [700, 600, 90], [90, 70, 40], 16
    k, v, table = make_cache(g, lens, page, 2, 128, BF, fill=0.0)
    starts = [0, 90, 160, 200]
    q = torch.randn((200, 8, 128), generator=g, device=DEV).to(BF)
    q[..., 0] = q[..., 0].abs() + 0.1
    gone = [(0, 0), (0, 9), (0, 43), *((1, j) for j in range(20))] + [(2, j) for j in range(6)]   # all of sequence 2
    absent = table.clone()
    for s, j in gone:
        k[table[s, j].long(), ..., 0] = -math.inf
        absent[s, j] = -1
    call = lambda t: r.rope3d_paged_attention(q, k, v, t, ints(lens), ints(starts), max_new=HINTS[kernel], lse=True)  # noqa: E731
    out, lse = call(table)
    want, want_lse = call(absent)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert bool((out[160:] == 0).all()) and bool((lse[160:] == -math.inf).all()) and bool(lse[:160].isfinite().all())
