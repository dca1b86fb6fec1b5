"""rope3d_block_norm and its backward pass on the GPU against 64 bits, within
bounds derived rounding by rounding (block_reference.py): both norms, each alone,
with and without weights, gate, scale and shift, groups of every size down to one
row, rows of one channel to rows too long for registers, unaligned and strided
views, in place."""
from __future__ import annotations

import itertools

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import rope_rope3d_apply_gb300 as r  # noqa: E402
from tests import block_reference as ref  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def make(rows, channels, dtype, groups=1, y=True, post=1, pre=1, weights=True, mod=True, params=None, rpg=None, seed=0,
         **kw):
    """Keyword arguments of a call, and dr, dn. groups: rows / groups rows each,
    or rpg rows each (the last shorter)."""
    g = torch.Generator(device=DEV).manual_seed(seed + 31 * rows + channels)
    dt, pt = DT[dtype], DT[params or dtype]
    rpg = rpg or rows // groups
    n_groups = -(-rows // rpg)

    def normal(shape, dtype, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=g, device=DEV) * scale + shift).to(dtype)

    a = dict(x=normal((rows, channels), dt, 2.0, 0.3), y=normal((rows, channels), dt, 0.7, -0.2) if y else None,
             post=post, pre=pre, rows_per_group=rpg, **kw)
    off = kw.get("weight_offset", 0.0)
    if weights:
        a["pre_weight"] = normal((channels,), pt, 0.1, 1.0 - off)
        if y and post:
            a["post_weight"] = normal((channels,), pt, 0.1, 1.0 - off)
    if mod:
        m = normal((n_groups, 3, channels), pt, 0.3)   # rows of one modulation tensor: strided views
        a["scale"], a["shift"] = m[:, 0], m[:, 1]
        if y:
            a["gate"] = m[:, 2]
    return a, normal((rows, channels), dt, 0.5), normal((rows, channels), dt, 0.5)


@pytest.fixture(autouse=True)
def no_timeouts():
    yield
    assert r.rope3d_testing_norm_wait_timeouts() == 0


def both(a, dr, dn, kernel):
    """Forward and backward against 64 bits. kernel 1: rows in registers or (many
    rows) through shared memory, 2: the general kernels, 3: through shared memory."""
    def last():
        k = r.rope3d_block_norm_last_kernel()
        return k == kernel or (kernel == 1 and k == 3)

    got = dict(zip(("r", "n"), r.rope3d_block_norm(**a)))
    assert last()
    want = ref.norm64(**a)
    for name, t in got.items():
        if t is not None:
            ref.check(t, want[name], name)
    got = r.rope3d_block_norm_backward(dr=dr, dn=dn, **a)
    assert last()
    torch.cuda.synchronize()
    want = ref.norm64(dr=dr, dn=dn, grads=True, **a)
    assert set(got) == set(want)
    for name, t in got.items():
        ref.check(t, want[name], name)
    again = r.rope3d_block_norm_backward(dr=dr, dn=dn, **a)
    for name, t in got.items():
        assert torch.equal(t, again[name]), name


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("post,pre", list(itertools.product((0, 1, 2), (0, 1, 2))))
@pytest.mark.parametrize("channels,kernel", [(256, 1), (77, 1), (20000, 2)])
def test_kinds(post, pre, channels, kernel, dtype):
    both(*make(37 if channels < 1000 else 5, channels, dtype, post=post, pre=pre, residual_scale=0.5), kernel)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("y,weights,mod", list(itertools.product((True, False), repeat=3)))
@pytest.mark.parametrize("channels,kernel", [(512, 1), (130, 1), (16390, 2)])
def test_absent_parts(y, weights, mod, channels, kernel, dtype):
    both(*make(24, channels, dtype, groups=3, y=y, weights=weights, mod=mod, weight_offset=1.0), kernel)


@pytest.mark.parametrize("dtype,channels,kernel", [
    # one channel, one vector, whole warps and their neighbours, each team size, the longest rows in registers, longer
    ("bf16", 1, 1), ("f32", 3, 1), ("f16", 63, 1), ("bf16", 65, 1), ("f32", 257, 1), ("bf16", 511, 1), ("f16", 513, 1),
    ("f32", 1157, 1), ("bf16", 2047, 1), ("f32", 2049, 1), ("f32", 4097, 1), ("f32", 8191, 1), ("bf16", 8, 1), ("f32", 4, 1), ("bf16", 248, 1), ("bf16", 264, 1), ("f16", 520, 1),
    ("bf16", 1000, 1), ("bf16", 1032, 1), ("f32", 1028, 1), ("bf16", 2048, 1), ("f16", 4096, 1), ("bf16", 4104, 1),
    ("bf16", 8192, 1), ("f32", 2052, 1), ("f32", 4096, 1), ("f32", 8192, 1), ("bf16", 65536, 2), ("f16", 20001, 2),
    ("bf16", 2049, 1), ("bf16", 4097, 1), ("f16", 6635, 1), ("f16", 8191, 1),
])
def test_channels(dtype, channels, kernel):
    both(*make(5, channels, dtype, post=2, pre=2), kernel)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("channels", [1, 64, 200, 500, 1024, 1157, 2048, 4096, 4001, 6635, 8192, 9000])
@pytest.mark.parametrize("rows,rpg", [(1, 1), (2, 1), (3, 2)])
def test_few_rows(rows, rpg, channels, dtype):
    """One row a group: chunks of whole groups, at every team size."""
    a, dr, dn = make(rows, channels, dtype, rpg=rpg)
    want = ref.norm64(**a)
    out = r.rope3d_block_norm(**a)
    ref.check(out[0], want["r"], "r")
    ref.check(out[1], want["n"], "n")
    want = ref.norm64(dr=dr, dn=dn, grads=True, **a)
    for name, t in r.rope3d_block_norm_backward(dr=dr, dn=dn, **a).items():
        ref.check(t, want[name], name)


@pytest.mark.parametrize("dtype,channels,forward,backward", [
    ("bf16", 16384, 1, 2), ("f32", 9001, 1, 2), ("f16", 9001, 1, 2), ("bf16", 16383, 1, 2),
])
def test_other_kernel_backward(dtype, channels, forward, backward):
    """Sizes whose forward and backward passes take different kernels."""
    a, dr, dn = make(3, channels, dtype)
    want = ref.norm64(**a)
    out = r.rope3d_block_norm(**a)
    assert r.rope3d_block_norm_last_kernel() == forward
    ref.check(out[0], want["r"], "r")
    ref.check(out[1], want["n"], "n")
    got = r.rope3d_block_norm_backward(dr=dr, dn=dn, **a)
    assert r.rope3d_block_norm_last_kernel() == backward
    want = ref.norm64(dr=dr, dn=dn, grads=True, **a)
    for name, t in got.items():
        ref.check(t, want[name], name)


@pytest.mark.parametrize("params", ["f32", None])
@pytest.mark.parametrize("dtype,channels,kernel", [("bf16", 320, 1), ("f16", 1152, 1), ("bf16", 45, 1), ("f16", 64, 1), ("f32", 700, 1)])
@pytest.mark.parametrize("rows,rpg", [(1, 1), (2, 1), (700, 1), (700, 3), (700, 64), (701, 350), (3000, 1500), (3000, 7)])
def test_groups(rows, rpg, dtype, channels, kernel, params):
    both(*make(rows, channels, dtype, rpg=rpg, params=params), kernel)


RING = [
    # rows, channels, dtype, groups: one warp a row, absent threads, each type's longest rows, one and several groups
    (20000, 128, "bf16", 2), (12000, 8, "bf16", 1), (6000, 2048, "f16", 1), (5000, 1032, "bf16", 4),
    (3000, 4096, "bf16", 3), (12000, 4, "f32", 5), (3000, 1156, "f32", 2), (700, 8192, "bf16", 1), (700, 8192, "f32", 1),
    (2432, 2048, "bf16", 2432), (5000, 520, "f16", 1000), (3001, 777, "f32", 1), (30000, 33, "bf16", 3), (4000, 1999, "f16", 1),
]


@pytest.mark.parametrize("rows,channels,dtype,groups", RING)
@pytest.mark.parametrize("post,pre,weights,mod", [(1, 1, True, False), (0, 1, False, True), (2, 2, True, True)])
def test_many_rows(rows, channels, dtype, groups, post, pre, weights, mod):
    a, dr, dn = make(rows, channels, dtype, groups=groups, post=post, pre=pre, weights=weights, mod=mod,
                     residual_scale=0.75)
    both(a, dr, dn, 3 if 384 <= channels < 8192 and channels % 4 == 0 else 1)


@pytest.mark.parametrize("y,pre", [(False, 1), (False, 2), (True, 0), (False, 0)])
def test_many_rows_absent_parts(y, pre):
    a, dr, dn = make(5000, 768, "bf16", groups=2, y=y, post=0, pre=pre)
    both(a, dr, dn, 3)
    # no gradient of one output, or of the parameters
    for d in (dict(dr=dr), dict(dn=dn)):
        want = ref.norm64(grads=True, **d, **a)
        for name, t in r.rope3d_block_norm_backward(**d, **a).items():
            ref.check(t, want[name], name)
    got = r.rope3d_block_norm_backward(dr=dr, dn=dn, param_grads=False, **a)
    want = ref.norm64(dr=dr, dn=dn, grads=True, **a)
    for name, t in got.items():
        ref.check(t, want[name], name)
