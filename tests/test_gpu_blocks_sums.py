"""Sums over many rows of the block operators' backward passes, where a bound on
rounding errors is too wide to see one row: exactly, on small whole numbers, for the
norms' column sums; and the feed-forward's weight gradients whose only terms lie far
apart, past 2^31 elements of the arrays in between."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import rope_rope3d_apply_gb300 as r  # noqa: E402
from tests import block_reference as ref  # noqa: E402

DEV = torch.device("cuda:0")
BF = torch.bfloat16
DT = {"bf16": BF, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def no_timeouts():
    yield
    assert r.rope3d_testing_ffn_wait_timeouts() == 0
    assert r.rope3d_testing_norm_wait_timeouts() == 0


def whole(g, shape, lo, hi, dtype):
    """Whole numbers from lo to hi, each as likely."""
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV, dtype=torch.int8).to(dtype)


def exact_sums(rows, channels, dtype, rpg, seed=0, step=50_000):
    """Without norms every value of the backward pass is a whole number:
        e = dn wq (1 + scale),  dR = dr + e,  dx = dR,  dy = dR gate,
        S = sum dn r,  T = sum dn,  U = sum dR y,  r = x + gate y
    With |x|, |y| <= 2, |dr|, |dn|, |gate| <= 1, wq and 1 + scale in {1, 2}: |dR| <= 5,
    |r| <= 4, so a row adds at most 4 to S, 10 to U and 2 * 4 to a weight's gradient,
    and the sums of up to 600,000 rows times wq stay below 2^24: every fp32 partial sum
    in any order is exact, and dx and dy are exact in 16 bits."""
    assert rows * 10 * 2 < 1 << 24
    g = torch.Generator(device=DEV).manual_seed(seed + rows + channels)
    dt, f32 = DT[dtype], torch.float32
    groups = -(-rows // rpg)
    x, y = whole(g, (rows, channels), -2, 2, dt), whole(g, (rows, channels), -2, 2, dt)
    dr, dn = whole(g, (rows, channels), -1, 1, dt), whole(g, (rows, channels), -1, 1, dt)
    gate, scale = whole(g, (groups, channels), -1, 1, f32), whole(g, (groups, channels), 0, 1, f32)
    wq, shift = whole(g, (channels,), 1, 2, f32), torch.zeros((groups, channels), device=DEV)
    got = r.rope3d_block_norm_backward(x, y, dr, dn, post=r.NORM_NONE, pre=r.NORM_NONE, gate=gate, pre_weight=wq,
                                       scale=scale, shift=shift, rows_per_group=rpg)
    S, T, U = (torch.zeros((groups, channels), dtype=torch.float64, device=DEV) for _ in range(3))
    for lo in range(0, rows, step):   # in pieces: the 64-bit arrays of 600,000 rows are large
        part = slice(lo, min(lo + step, rows))
        of = torch.arange(part.start, part.stop, device=DEV) // rpg
        xs, ys, drs, dns = (t[part].double() for t in (x, y, dr, dn))
        gs = gate.double()[of]
        dR = drs + dns * wq * (1 + scale.double()[of])
        assert torch.equal(got["dx"][part].double(), dR) and torch.equal(got["dy"][part].double(), dR * gs)
        S.index_add_(0, of, dns * (xs + gs * ys))
        T.index_add_(0, of, dns)
        U.index_add_(0, of, dR * ys)
    want = {"d_scale": wq * S, "d_shift": T, "d_gate": U, "d_pre_weight": ((1 + scale) * S).sum(0)}
    for name, t in want.items():
        assert torch.equal(got[name].double(), t), (name, int((got[name].double() != t).sum()))


@pytest.mark.parametrize("rows,channels,dtype,rpg", [
    # teams of lanes, whole warps, single elements; one group, ragged groups, groups of few rows
    (30000, 33, "bf16", 30000), (30000, 64, "f16", 7), (20000, 128, "bf16", 9999), (12000, 8, "f32", 12000), (20000, 256, "bf16", 20000),
    (20000, 200, "f32", 61), (4000, 1999, "f16", 1500), (3001, 777, "f32", 3001), (2000, 4001, "bf16", 700),
    # the ring: one group, a few, a ragged last one, many small ones, one row each
    (6000, 2048, "f16", 6000), (12000, 512, "bf16", 12000), (5000, 1032, "bf16", 1250), (8191, 768, "f32", 3000), (5000, 520, "f16", 5),
    (2432, 2048, "bf16", 1), (700, 8192, "bf16", 700), (20001, 384, "bf16", 20001),
    # too few rows for it, and the general kernels
    (301, 4096, "bf16", 301), (77, 8192, "f16", 20), (1, 2048, "bf16", 1), (300, 9001, "f32", 300), (123, 20000, "bf16", 41),
    (40, 65536, "f16", 7),
])
def test_every_row_counts_once(rows, channels, dtype, rpg):
    exact_sums(rows, channels, dtype, rpg)


@pytest.mark.parametrize("rpg", [600_000, 599_001])
def test_every_row_counts_once_past_32_bits(rpg):
    """Tensors of more than 2^32 bytes and 2^31 elements."""
    exact_sums(600_000, 4096, "bf16", rpg)


@pytest.mark.parametrize("kept", [BF, None], ids=["kept", "again"])
def test_weight_gradients_of_far_tokens(kept):
    """tokens x hidden past 2^31 elements: dy is zero but for three runs of 32 tokens
    (at the start, past the middle, at the end), so that the weights' gradients are
    those of the 96 tokens alone; kept projections, and (in fp32) computed again."""
    tokens, width, hidden = 300_000, 64, 8192
    assert 262_144 * hidden == 1 << 31
    g = torch.Generator(device=DEV).manual_seed(17)

    def normal(shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * scale).to(BF)

    x = normal((tokens, width))
    w = (normal((hidden, width), width ** -0.5), normal((hidden, width), width ** -0.5), normal((width, hidden), hidden ** -0.5))
    # (runs of whole 16s, so that the 96 tokens are added in as few steps as alone)
    far = torch.cat([torch.arange(a, a + 32, device=DEV) for a in (0, 262_160, tokens - 32)])
    dy = torch.zeros((tokens, width), dtype=BF, device=DEV)
    dy[far] = normal((96, width))
    pre = () if kept is None else r.rope3d_gated_ffn(x, *w, act=1, keep=kept)[1:]
    got = r.rope3d_gated_ffn_backward(dy, x, *w, *pre, act=1)
    want = ref.ffn_backward64(dy[far], x[far], *w, 1, *(t[far] for t in pre))
    ref.check(got[0][far], want["dx"], "dx")
    rest = torch.ones(tokens, dtype=torch.bool, device=DEV)
    rest[far] = False
    assert not bool(got[0][rest].any())
    for name, t in zip(("dw_gate", "dw_up", "dw_down"), got[1:]):
        ref.check(t, want[name], name)
