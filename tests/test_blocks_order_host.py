"""Orders that the block operators' kernels have to keep in their source, and that
a run on an idle GPU does not show."""
from __future__ import annotations

import os
import re

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


@pytest.mark.parametrize("file,kernel", [
    (FFN, "ffn_tile_kernel"), (FFN, "ffn_stream_kernel"), (NORM, "block_norm_ring_kernel"),
    (BACK, "block_norm_back_ring_kernel"),
])
def test_a_wait_that_runs_out_does_not_part_a_warp(file, kernel):
    """Lanes of a warp try a barrier one by one: a wait can run out for some of them
    while others see it complete. Where its result decides the way, either a single
    lane waits or the warp takes one answer; else some lanes would leave and the
    others wait for them, without a limit, in their next warp-wide operation."""
    def walk(block, one_lane):
        for part in block.parts:
            if isinstance(part, str):
                for m in re.finditer(r"if\s*\(\s*!\s*mbar_wait\(|=\s*mbar_wait\(", part):
                    rest = part[m.start():]
                    if one_lane or re.search(r"__all_sync\(0xffffffffu, ready\)\) break;", rest):
                        continue
                    # (a result that is only noted decides no way)
                    assert re.match(r"if \(!mbar_wait\([^;]*\) && lost < 0\) lost = [^;]*;", rest), rest[:120]
            else:
                walk(part, one_lane or re.search(r"lane == 0\b", part.head) is not None)

    walk(src.kernel(file, kernel), False)


def test_warp_aligned_instructions_are_behind_a_syncwarp():
    """PTX wants every lane of a warp at an .aligned instruction, and promises no
    reconvergence behind branches and loops that lanes leave one by one. The helpers
    that hold such instructions bring the lanes together themselves, and the kernels
    have none outside of them."""
    with open(os.path.join(src.CSRC, "rope3d_tc.cuh")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    functions = re.split(r"(?=__device__ __forceinline__)", text)
    aligned = [f for f in functions if ".aligned" in f]
    assert len(aligned) == 5
    for f in aligned:
        assert re.search(r"\)\s*\{\s*(\w+ \*?\w+ = [^;]*;\s*)?__syncwarp\(\);", f), f[:120]
    for name in (FFN, NORM, BACK, "rope3d_norm.cuh"):
        with open(os.path.join(src.CSRC, name)) as f:
            assert ".aligned" not in re.sub(r"//[^\n]*", "", f.read()), name


def test_finish_reads_only_sums_that_were_written():
    """Chunks of whole groups finish their groups' gradients themselves and leave only
    the weights' sums (1 and 3 of the three rows) for block_norm_finish_kernel. The
    kernel's own expression says which rows it reads."""
    want = re.search(r"const bool want\[3\] = \{([^;]*)\};", src.flat(src.kernel(BACK, "block_norm_finish_kernel"))).group(1)
    names = ("d_pre_weight", "d_scale", "d_shift", "d_post_weight", "d_gate")
    for bits in range(64):
        given = {n: bool(bits >> i & 1) for i, n in enumerate(names)}
        whole = bool(bits >> 5)
        text = re.sub(r"p\.(\w+)\s*!=\s*nullptr", r"p.\1", want)
        text = re.sub(r"p\.(\w+)", lambda m: str(whole if m.group(1) == "groups_per_chunk" else given[m.group(1)]), text)
        text = text.replace("&&", " and ").replace("||", " or ").replace("!", " not ").replace("split", str(not whole))
        read = eval("(" + text + ")")   # noqa: S307 (the kernel's own expression)
        assert read == ((given["d_pre_weight"] or not whole and given["d_scale"]), not whole and given["d_shift"],
                        (given["d_post_weight"] or not whole and given["d_gate"])), (given, whole)
