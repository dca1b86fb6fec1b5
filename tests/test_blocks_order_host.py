"""Orders that the block operators' kernels have to keep in their source, and that
a run on an idle GPU does not show."""
from __future__ import annotations

import pytest

from tests import kernel_source as src

FFN, NORM, BACK = "rope3d_ffn.cu", "rope3d_norm.cu", "rope3d_norm_back.cu"


@pytest.mark.parametrize("file,kernel", [
    (FFN, "ffn_tile_kernel"), (FFN, "ffn_stream_kernel"), (NORM, "block_norm_ring_kernel"),
    (BACK, "block_norm_back_ring_kernel"),
])
def test_bounded_waits_begin_after_earlier_kernels(file, kernel):
    """A wait's limit runs from its first try. The kernels start before the one ahead
    of them in the stream is done, and their copies (all of them, or the tokens')
    only afterwards: a wait that begins earlier would run out under a long kernel
    with nothing wrong. So each thread that waits is past grid_wait() first."""
    body = src.kernel(file, kernel)
    _, missing = src.before_each(body, "mbar_wait", "grid_wait")
    assert "mbar_wait" in src.flat(body)
    assert not missing, missing
