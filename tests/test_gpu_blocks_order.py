"""The block operators behind a kernel that lets them start early and then runs for
longer than the limit of their own waits."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import rope_rope3d_apply_gb300 as r  # noqa: E402

DEV = torch.device("cuda:0")
BF = torch.bfloat16


@pytest.fixture(scope="module")
def long_kernel(tmp_path_factory):
    from rope_rope3d_apply_gb300 import build

    here = os.path.dirname(os.path.abspath(__file__))
    lib = str(tmp_path_factory.mktemp("long") / "liblong.so")
    subprocess.run([build._nvcc(), *build.ARCH, "-O2", "-shared", "-Xcompiler", "-fPIC",
                    os.path.join(here, "long_predecessor.cu"), "-o", lib], check=True)
    fn = ctypes.CDLL(lib).launch_long_predecessor
    fn.argtypes, fn.restype = [ctypes.c_longlong, ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int
    return fn


@pytest.mark.parametrize("tokens", [1, 24, 130, 300])
def test_waits_do_not_count_an_earlier_kernels_time(long_kernel, tokens):
    """Limits are 10^9 clocks; the kernel ahead takes 1.5 * 10^9. Few tokens (weights
    streamed), the mixed range, tiles, and the norms' ring of many rows."""
    g = torch.Generator(device=DEV).manual_seed(tokens)
    normal = lambda *shape: torch.randn(shape, generator=g, device=DEV).to(BF)  # noqa: E731
    x, dy = normal(tokens, 256), normal(tokens, 256)
    w = (normal(512, 256) / 16, normal(512, 256) / 16, normal(256, 512) / 16)
    rows = normal(5000, 768)
    calls = [lambda: (r.rope3d_gated_ffn(x, *w),), lambda: r.rope3d_gated_ffn_backward(dy, x, *w)]
    if tokens == 1:
        calls.append(lambda: r.rope3d_block_norm(rows, rows, post=r.NORM_RMS))
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        assert long_kernel(1_500_000_000, flag.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        got = call()
        torch.cuda.synchronize()
        assert int(flag) == 1
        assert r.rope3d_testing_ffn_wait_timeouts() == 0 and r.rope3d_testing_norm_wait_timeouts() == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want))
