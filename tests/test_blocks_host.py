"""Host-side checks of the transformer-block operators (no GPU): what
rope3d_block_norm, rope3d_gated_ffn and their backward passes refuse, and the
sizes of their workspaces."""
from __future__ import annotations

import ctypes

import pytest

import rope_rope3d_apply_gb300 as r


@pytest.fixture(scope="module", autouse=True)
def lib():
    from rope_rope3d_apply_gb300 import build

    build.build()
    return r.load_library()


MB = 1 << 20


def norm_args(**kw):
    """A valid call on made-up addresses: 12 rows of 32 bf16 channels, 3 groups."""
    a = dict(x=1 * MB, y=2 * MB, r=3 * MB, n=4 * MB, post_weight=5 * MB, pre_weight=6 * MB, gate=7 * MB, scale=8 * MB,
             shift=9 * MB, rows=12, channels=32, rows_per_group=4, x_stride=32, y_stride=32, r_stride=32, n_stride=32,
             gate_stride=96, scale_stride=96, shift_stride=96, eps=1e-6, residual_scale=1.0, weight_offset=1.0,
             dtype=r.BF16, param_dtype=r.BF16, post_kind=r.NORM_RMS, pre_kind=r.NORM_LAYER)
    a.update(kw)
    return a


NORM_OK = [
    {}, dict(n=0), dict(r=0), dict(y=0, post_weight=0, gate=0, r=0), dict(post_kind=r.NORM_NONE, post_weight=0),
    dict(param_dtype=r.F32), dict(dtype=r.F32, param_dtype=r.F32), dict(x_stride=1000), dict(rows_per_group=100),
    dict(r=1 * MB), dict(n=2 * MB), dict(r=2 * MB, n=1 * MB), dict(eps=0.0), dict(residual_scale=-0.5),
    dict(x=1 * MB + 2), dict(rows=1, rows_per_group=1), dict(channels=1),
]
NORM_BAD = [
    (dict(x=0), "ERR_NULL"), (dict(r=0, n=0), "ERR_NULL"),
    (dict(rows=0), "ERR_SHAPE"), (dict(rows=-1), "ERR_SHAPE"), (dict(channels=0), "ERR_SHAPE"),
    (dict(channels=65537, x_stride=65537), "ERR_SHAPE"), (dict(rows_per_group=0), "ERR_SHAPE"),
    (dict(rows=1 << 31), "ERR_SHAPE"), (dict(x_stride=31), "ERR_SHAPE"), (dict(y_stride=31), "ERR_SHAPE"),
    (dict(r_stride=31), "ERR_SHAPE"), (dict(n_stride=0), "ERR_SHAPE"), (dict(gate_stride=31), "ERR_SHAPE"),
    (dict(scale_stride=-96), "ERR_SHAPE"), (dict(shift_stride=(1 << 31) + 1), "ERR_SHAPE"),
    (dict(dtype=3), "ERR_DTYPE"), (dict(param_dtype=r.F16), "ERR_DTYPE"), (dict(dtype=r.F32), "ERR_DTYPE"),
    (dict(post_kind=3), "ERR_ARG"), (dict(pre_kind=-1), "ERR_ARG"), (dict(eps=-1e-6), "ERR_ARG"),
    (dict(eps=float("nan")), "ERR_ARG"), (dict(residual_scale=float("inf")), "ERR_ARG"),
    (dict(weight_offset=float("nan")), "ERR_ARG"), (dict(y=0), "ERR_ARG"), (dict(y=0, post_weight=0), "ERR_ARG"),
    (dict(post_kind=r.NORM_NONE), "ERR_ARG"),
    (dict(x=1 * MB + 1), "ERR_ALIGN"), (dict(gate=7 * MB + 1), "ERR_ALIGN"),
    (dict(dtype=r.F32, param_dtype=r.F32, n=4 * MB + 2), "ERR_ALIGN"),
    (dict(r=1 * MB + 64), "ERR_ALIAS"), (dict(r=1 * MB, r_stride=64), "ERR_ALIAS"), (dict(n=3 * MB), "ERR_ALIAS"),
    (dict(n=5 * MB), "ERR_ALIAS"), (dict(r=8 * MB), "ERR_ALIAS"), (dict(r=1 * MB, n=1 * MB), "ERR_ALIAS"),
]


@pytest.mark.parametrize("change", NORM_OK, ids=str)
def test_norm_accepts(change):
    assert r.rope3d_block_norm_check(**norm_args(**change)) == "OK"


@pytest.mark.parametrize("change,status", NORM_BAD, ids=str)
def test_norm_refuses(change, status):
    assert r.rope3d_block_norm_check(**norm_args(**change)) == status


def norm_back_args(**kw):
    a = norm_args(r=0, n=0)
    a.update(dr=10 * MB, dn=11 * MB, dx=12 * MB, dy=13 * MB, d_post_weight=14 * MB, d_pre_weight=15 * MB, d_gate=16 * MB,
             d_scale=16 * MB + 64, d_shift=16 * MB + 128, dr_stride=32, dn_stride=32, dx_stride=32, dy_stride=32,
             grad_stride=96, workspace=20 * MB, workspace_bytes=4 * MB)
    a.update(kw)
    return a


def test_norm_backward_accepts():
    for change in ({}, dict(dr=0), dict(dn=0), dict(dx=10 * MB, dy=11 * MB), dict(dx=11 * MB, dy=10 * MB),
                   dict(d_gate=0, d_scale=0, d_shift=0, grad_stride=0),
                   dict(y=0, dy=0, gate=0, d_gate=0, post_weight=0, d_post_weight=0),
                   dict(d_gate=0, d_scale=0, d_shift=0, d_pre_weight=0, d_post_weight=0, workspace=0, workspace_bytes=0)):
        assert r.rope3d_block_norm_backward_check(**norm_back_args(**change)) == "OK", change


@pytest.mark.parametrize("change,status", [
    (dict(dx=0), "ERR_NULL"), (dict(dr=0, dn=0), "ERR_NULL"), (dict(dy=0), "ERR_NULL"), (dict(y=0), "ERR_NULL"),
    (dict(workspace=0), "ERR_NULL"),
    (dict(scale=0), "ERR_ARG"), (dict(pre_weight=0), "ERR_ARG"), (dict(gate=0), "ERR_ARG"),
    (dict(dr_stride=31), "ERR_SHAPE"), (dict(dx_stride=31), "ERR_SHAPE"), (dict(grad_stride=31), "ERR_SHAPE"),
    (dict(dx=10 * MB + 64), "ERR_ALIAS"), (dict(dx=10 * MB, dy=10 * MB), "ERR_ALIAS"), (dict(dx=1 * MB), "ERR_ALIAS"),
    (dict(d_gate=16 * MB + 32), "ERR_ALIAS"), (dict(grad_stride=64), "ERR_ALIAS"), (dict(d_pre_weight=14 * MB), "ERR_ALIAS"),
    (dict(workspace=12 * MB - 256), "ERR_ALIAS"),
    (dict(workspace_bytes=16), "ERR_SCRATCH"), (dict(workspace=20 * MB + 128), "ERR_ALIGN"),
    (dict(dn=11 * MB + 1), "ERR_ALIGN"),
], ids=str)
def test_norm_backward_refuses(change, status):
    assert r.rope3d_block_norm_backward_check(**norm_back_args(**change)) == status


def ffn_args(**kw):
    """A valid call on made-up addresses: 10 tokens, width 24, hidden 40."""
    a = dict(x=1 * MB, w_gate=2 * MB, w_up=3 * MB, w_down=4 * MB, y=5 * MB, gate_pre=6 * MB, up_pre=7 * MB, tokens=10,
             width=24, hidden=40, x_stride=24, w_gate_stride=24, w_up_stride=24, w_down_stride=40, y_stride=24,
             pre_stride=40, workspace=20 * MB, workspace_bytes=16 * MB, dtype=r.BF16, pre_dtype=r.F32, act=r.ACT_SILU)
    a.update(kw)
    return a


def test_ffn_accepts():
    for change in ({}, dict(gate_pre=0, up_pre=0, pre_dtype=99, pre_stride=0), dict(pre_dtype=r.BF16), dict(dtype=r.F16),
                   dict(w_up=2 * MB + 24 * 40 * 2), dict(x=1 * MB + 2, x_stride=25), dict(act=r.ACT_GELU_ERF),
                   dict(tokens=1, width=1, hidden=1)):
        assert r.rope3d_gated_ffn_check(**ffn_args(**change)) == "OK", change


FFN_BAD = [
    (dict(x=0), "ERR_NULL"), (dict(w_gate=0), "ERR_NULL"), (dict(w_up=0), "ERR_NULL"), (dict(w_down=0), "ERR_NULL"),
    (dict(workspace=0), "ERR_NULL"), (dict(gate_pre=0), "ERR_NULL"), (dict(up_pre=0), "ERR_NULL"),
    (dict(tokens=0), "ERR_SHAPE"), (dict(width=0), "ERR_SHAPE"), (dict(hidden=-1), "ERR_SHAPE"),
    (dict(tokens=(1 << 28) + 1), "ERR_SHAPE"), (dict(width=(1 << 20) + 1), "ERR_SHAPE"), (dict(x_stride=23), "ERR_SHAPE"),
    (dict(w_gate_stride=0), "ERR_SHAPE"), (dict(w_down_stride=39), "ERR_SHAPE"), (dict(pre_stride=39), "ERR_SHAPE"),
    (dict(w_up_stride=(1 << 31) + 8), "ERR_SHAPE"),
    (dict(dtype=r.F32), "ERR_DTYPE"), (dict(dtype=7), "ERR_DTYPE"), (dict(pre_dtype=r.F16), "ERR_DTYPE"),
    (dict(act=3), "ERR_ARG"), (dict(act=-1), "ERR_ARG"),
    (dict(x=1 * MB + 1), "ERR_ALIGN"), (dict(w_down=4 * MB + 1), "ERR_ALIGN"), (dict(gate_pre=6 * MB + 2), "ERR_ALIGN"),
    (dict(workspace=20 * MB + 128), "ERR_ALIGN"),
    (dict(workspace_bytes=100), "ERR_SCRATCH"),
]


@pytest.mark.parametrize("change,status", FFN_BAD + [
    (dict(y=0), "ERR_NULL"), (dict(y_stride=23), "ERR_SHAPE"), (dict(y=1 * MB), "ERR_ALIAS"), (dict(y=4 * MB + 64), "ERR_ALIAS"),
    (dict(up_pre=6 * MB), "ERR_ALIAS"), (dict(workspace=5 * MB), "ERR_ALIAS"), (dict(workspace=4 * MB - 256), "ERR_ALIAS"),
], ids=str)
def test_ffn_refuses(change, status):
    assert r.rope3d_gated_ffn_check(**ffn_args(**change)) == status


def ffn_back_args(**kw):
    a = ffn_args()
    for k in ("y", "y_stride"):
        del a[k]
    a.update(dy=8 * MB, dx=9 * MB, dw_gate=10 * MB, dw_up=11 * MB, dw_down=12 * MB, dy_stride=24, dx_stride=24,
             dw_gate_stride=24, dw_up_stride=24, dw_down_stride=40)
    a.update(kw)
    return a


def test_ffn_backward_accepts():
    for change in ({}, dict(gate_pre=0, up_pre=0), dict(dx=0, dx_stride=0), dict(dw_gate=0, dw_up=0), dict(dw_down=0),
                   dict(dw_up=10 * MB + 24 * 40 * 2)):
        assert r.rope3d_gated_ffn_backward_check(**ffn_back_args(**change)) == "OK", change


@pytest.mark.parametrize("change,status", FFN_BAD + [
    (dict(dy=0), "ERR_NULL"), (dict(dx=0, dw_gate=0, dw_up=0, dw_down=0), "ERR_NULL"), (dict(dw_up=0), "ERR_NULL"),
    (dict(dy_stride=23), "ERR_SHAPE"), (dict(dw_down_stride=39), "ERR_SHAPE"), (dict(dx=8 * MB), "ERR_ALIAS"),
    (dict(dw_gate=2 * MB), "ERR_ALIAS"), (dict(dw_up=10 * MB + 64), "ERR_ALIAS"), (dict(dw_down=6 * MB), "ERR_ALIAS"),
    (dict(workspace=9 * MB - 256), "ERR_ALIAS"),
], ids=str)
def test_ffn_backward_refuses(change, status):
    assert r.rope3d_gated_ffn_backward_check(**ffn_back_args(**change)) == status


def workspace(cls, query, **fields):
    n = ctypes.c_int64()
    assert getattr(r.load_library(), query)(ctypes.byref(cls(**fields)), ctypes.byref(n)) == 0
    return n.value


def test_workspaces_grow_with_what_is_kept_there():
    """act(g) * u of every token; copies of matrices whose rows are unaligned;
    in the backward pass three such arrays, and the projections where they are
    computed again."""
    def fwd(**kw):
        return workspace(r._FfnArgs, "rope3d_gated_ffn_workspace", **ffn_args(**kw))

    def back(**kw):
        return workspace(r._FfnBackArgs, "rope3d_gated_ffn_backward_workspace", **ffn_back_args(**kw))

    assert fwd() >= 10 * 40 * 2
    assert fwd(x=1 * MB + 2) >= fwd() + 10 * 24 * 2
    assert fwd(w_down_stride=41) >= fwd() + 24 * 40 * 2
    assert back() >= 3 * 10 * 40 * 2
    assert back(gate_pre=0, up_pre=0) >= back() + 2 * 10 * 40 * 4
    # the workspace itself is not looked at
    assert fwd(workspace=0, workspace_bytes=0) == fwd()
    # parameter gradients of the norms need partial sums, others nothing
    def norm(**kw):
        return workspace(r._NormBackArgs, "rope3d_block_norm_backward_workspace", **norm_back_args(**kw))

    assert norm() > 0
    assert norm(d_gate=0, d_scale=0, d_shift=0, d_pre_weight=0, d_post_weight=0) == 0


def test_null_arguments():
    lib = r.load_library()
    n = ctypes.c_int64()
    for name in ("rope3d_block_norm", "rope3d_block_norm_backward", "rope3d_gated_ffn", "rope3d_gated_ffn_backward"):
        assert getattr(lib, name)(None, None) == -1
        assert getattr(lib, name + "_check")(None, 0) == -1
    for name in ("rope3d_block_norm_backward", "rope3d_gated_ffn", "rope3d_gated_ffn_backward"):
        assert getattr(lib, name + "_workspace")(None, ctypes.byref(n)) == -1
    assert lib.rope3d_testing_ffn_wait_timeouts(None, 0) == -1
    assert lib.rope3d_testing_norm_wait_timeouts(None, 0) == -1


def test_binding_refuses_mismatched_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    w = torch.zeros(6, 8, dtype=torch.bfloat16)
    d = torch.zeros(8, 6, dtype=torch.bfloat16)
    for call in (
        lambda: r.rope3d_gated_ffn(x, w, w, d.T, act=0), lambda: r.rope3d_gated_ffn(x, w, w[:5], d),
        lambda: r.rope3d_gated_ffn(x.T, w, w, d), lambda: r.rope3d_gated_ffn(x[0], w, w, d),
        lambda: r.rope3d_gated_ffn(x, w, w, d, gate_pre=torch.zeros(4, 6)),
        lambda: r.rope3d_block_norm(x, x[:3]), lambda: r.rope3d_block_norm(x, pre_weight=torch.zeros(7)),
        lambda: r.rope3d_block_norm(x, scale=torch.zeros(3, 8)), lambda: r.rope3d_block_norm(x.T),
        lambda: r.rope3d_block_norm(x, scale=torch.zeros(2, 8), shift=torch.zeros(4, 8)),
        lambda: r.rope3d_block_norm(x, scale=torch.zeros(2, 8), rows_per_group=4),
    ):
        with pytest.raises((ValueError, r.Rope3dError)) as e:
            call()
        assert not isinstance(e.value, r.Rope3dError) or e.value.name == "ERR_SHAPE"
    for call in (
        lambda: r.rope3d_gated_ffn(x, w.half(), w, d), lambda: r.rope3d_block_norm(x, x.float()),
        lambda: r.rope3d_block_norm(x, pre_weight=torch.zeros(8), scale=torch.zeros(1, 8, dtype=torch.bfloat16)),
        lambda: r.rope3d_block_norm(x.to(torch.float64)),
    ):
        with pytest.raises(TypeError):
            call()
