"""The operators around a paged cache at the edges of what they take (no GPU)."""
from __future__ import annotations

import ctypes

import pytest

import rope_rope3d_apply_gb300 as r


def test_empty_sections_are_refused_by_name():
    """No counts at all: the binding's own refusal, as for counts that do not make up the frequencies."""
    torch = pytest.importorskip("torch")
    q, f = torch.zeros((4, 4, 32), dtype=torch.bfloat16), torch.zeros(16)
    pos = torch.zeros((3, 4), dtype=torch.int64)
    for sections in ((), [], (0,), (0, 0, 0)):
        with pytest.raises(ValueError, match="sections"):
            r.rope3d_apply_axes(q, None, pos, f, sections)


def workspace(**kw):
    """The attention's workspace for 1000 tokens of one sequence, 4 / 2 heads of 64."""
    mb = 1 << 20
    args = dict(page_table=100 * mb, seq_lens=101 * mb, seqs=1, pages=12, page_size=16, q=1 * mb, k_cache=20 * mb, v_cache=40 * mb,
                out=2 * mb, tokens=1000, q_heads=4, kv_heads=2, head_dim=64, q_token_stride=256, q_head_stride=64, out_token_stride=256,
                out_head_stride=64, k_page_stride=2048, k_slot_stride=128, k_cache_head_stride=64, v_page_stride=2048, v_slot_stride=128,
                v_cache_head_stride=64, scale=0.125, dtype=r.BF16, causal=1, **kw)
    need = ctypes.c_int64()
    assert r.load_library().rope3d_paged_attention_workspace(ctypes.byref(r._AttentionArgs(**args)), ctypes.byref(need)) == 0
    return need.value


def test_rows_that_no_bounded_wait_can_outlast():
    """Tables of more than 2^23 places a sequence: an item of the tiles could take longer than a wait in
    it may (10^9 clocks), so such a call goes to the kernel for few rows, whatever its rows. Seen by
    the workspace: two slots of 16 rows for each of 456 parts there, of 128 rows for each of 152 in tiles."""
    up256 = lambda n: -(-n // 256) * 256  # noqa: E731
    slots = lambda parts, rows: up256(2 * parts * rows * 66 * 4)  # noqa: E731
    notes = workspace(table_width=1 << 19, table_stride=1 << 19) - slots(152, 128)
    assert 0 < notes == up256(152 * (notes // 152))
    for width in ((1 << 19) + 1, 1 << 26):
        assert 0 < workspace(table_width=width, table_stride=width) - slots(456, 16) == up256(456 * (notes // 152))
