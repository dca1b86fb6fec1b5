"""The operators around a paged cache at the ends of their ranges: places far below zero and far up."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import rope_rope3d_apply_gb300 as r  # noqa: E402
from tests.paged_reference import close, rotate64  # noqa: E402

DEV = torch.device("cuda:0")


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
