"""The division of the attention over pages, the kernels' own source (rope3d_paged.cuh) compiled for
the host and run against brute force (tests/paged_line.cu): costs in 32 and 64 bits with and
without windows, lines on both sides of 2^21 and 2^31, lengths shorter than the new tokens, damaged
lengths and starts."""
from __future__ import annotations

import os
import subprocess

import pytest

from rope_rope3d_apply_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("line") / "paged_line")
    subprocess.run([build._nvcc(), "-std=c++17", "-O2", f"-I{build.CSRC}", os.path.join(HERE, "paged_line.cu"), "-o", out], check=True)
    return out


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_against_brute_force(program, seed):
    run = subprocess.run([program, str(seed), "300"], capture_output=True, text=True, timeout=600)
    assert run.returncode == 0, run.stdout
    taken = dict(line.rsplit(": ", 1) for line in run.stdout.splitlines())
    for bits in ("32 bits", "64 bits"):
        for case in (bits, bits + ", window", bits + ", causal", bits + ", window, causal"):
            assert int(taken[case]) > 100, case
    for case in ("lines below 2^21", "lines below 2^31", "lines of 2^31", "heads of 2^31", "divided items"):
        assert int(taken[case]) > 0, case
