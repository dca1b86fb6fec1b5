"""rope3d_gated_ffn and its backward pass on the GPU against 64 bits, within
bounds derived rounding by rounding (block_reference.py): one token to several
tiles of them, odd and ragged sizes, strided and unaligned matrices, kept and
recomputed projections, other streams, captured graphs."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import rope_rope3d_apply_gb300 as r  # noqa: E402
from tests import block_reference as ref  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(autouse=True)
def no_timeouts():
    yield
    assert r.rope3d_testing_ffn_wait_timeouts() == 0


def normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def make(tokens, width, hidden, dtype, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + tokens * 7 + width * 3 + hidden)
    dt = DT[dtype]
    return dict(x=normal(g, (tokens, width), dt), w_gate=normal(g, (hidden, width), dt, width ** -0.5),
                w_up=normal(g, (hidden, width), dt, width ** -0.5),
                w_down=normal(g, (width, hidden), dt, hidden ** -0.5)), normal(g, (tokens, width), dt)


SHAPES = [
    # tokens, width, hidden: few tokens (weights streamed) ...
    (1, 64, 128), (1, 8, 8), (1, 2048, 512), (2, 136, 264), (17, 512, 1024), (33, 72, 1000), (64, 256, 640),
    (100, 320, 192), (128, 128, 256),
    # ... and tiles of many
    (129, 64, 128), (150, 1032, 392), (200, 72, 520), (256, 128, 256), (257, 96, 64), (300, 200, 328), (515, 136, 264), (777, 520, 1096), (1024, 1024, 2048),
]
ODD = [(1, 1, 1), (1, 37, 131), (5, 129, 1), (40, 67, 259), (130, 1, 3), (200, 131, 259), (333, 77, 130)]


@pytest.mark.parametrize("act", [r.ACT_SILU, r.ACT_GELU_TANH, r.ACT_GELU_ERF])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES + ODD, ids=str)
def test_forward(shape, dtype, act):
    w, _ = make(*shape, dtype)
    y, g, u = r.rope3d_gated_ffn(**w, act=act, keep=True)
    torch.cuda.synchronize()
    assert r.rope3d_gated_ffn_last_kernel() == (2 if shape[0] <= 96 else 1)
    want = ref.ffn64(**w, act=act)
    ref.check(g, want["g"], "gate_pre")
    ref.check(u, want["u"], "up_pre")
    ref.check(y, want["y"], "y")
    # without the kept projections: the same bits
    assert torch.equal(r.rope3d_gated_ffn(**w, act=act), y)


@pytest.mark.parametrize("hidden", [1, 64, 250, 255])
def test_kept_shapes(hidden):
    """Kept projections are [tokens, hidden] for any shape of x, as the backward pass takes them."""
    w, dy = make(6, 40, hidden, "bf16")
    y, g, u = r.rope3d_gated_ffn(**w, keep=True)
    x = w.pop("x").view(2, 3, 40)
    y3, g3, u3 = r.rope3d_gated_ffn(x, **w, keep=True)
    assert y3.shape == x.shape and g3.shape == u3.shape == (6, hidden)
    assert torch.equal(y3.view(6, 40), y) and torch.equal(g3, g) and torch.equal(u3, u)
    got = r.rope3d_gated_ffn_backward(dy.view(2, 3, 40), x, *w.values(), g3, u3)
    want = r.rope3d_gated_ffn_backward(dy, x.view(6, 40), *w.values(), g.contiguous(), u.contiguous())
    assert got[0].shape == x.shape
    for a, b in zip(got, want):
        assert torch.equal(a.view(b.shape), b)


@pytest.mark.parametrize("kept", ["f32", "half", "again"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES + ODD, ids=str)
def test_backward(shape, dtype, kept):
    w, dy = make(*shape, dtype)
    act = (sum(shape) + len(kept)) % 3
    pre = ()
    if kept != "again":
        pre = r.rope3d_gated_ffn(**w, act=act, keep=True if kept == "f32" else DT[dtype])[1:]
    got = r.rope3d_gated_ffn_backward(dy, *w.values(), *pre, act=act)
    torch.cuda.synchronize()
    want = ref.ffn_backward64(dy, *w.values(), act, *pre)
    for name, t in zip(("dx", "dw_gate", "dw_up", "dw_down"), got):
        ref.check(t, want[name], name)
    # the same call again: the same bits; each gradient alone (their shared launch
    # is divided another way then): within the bound
    for a, b in zip(r.rope3d_gated_ffn_backward(dy, *w.values(), *pre, act=act), got):
        assert torch.equal(a, b)
    for need in ((True, False, False), (False, True, False), (False, False, True), (False, True, True)):
        alone = r.rope3d_gated_ffn_backward(dy, *w.values(), *pre, act=act, need=need)
        wanted = (need[0], need[1], need[1], need[2])
        for name, t, n in zip(("dx", "dw_gate", "dw_up", "dw_down"), alone, wanted):
            assert (t is not None) == n
            if n:
                ref.check(t, want[name], name)
