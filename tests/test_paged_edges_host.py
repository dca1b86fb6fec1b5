"""The operators around a paged cache at the edges of what they take (no GPU)."""
from __future__ import annotations

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
