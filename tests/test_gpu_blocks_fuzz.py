"""Seeded random calls of the block operators against 64 bits: sizes, types, kinds,
groups, absent parts, row strides and offsets, in-place outputs, and the memory
beside every output."""
from __future__ import annotations

import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import rope_rope3d_apply_gb300 as r  # noqa: E402
from tests import block_reference as ref  # noqa: E402

DEV = torch.device("cuda:0")
TYPES = (torch.bfloat16, torch.float16, torch.float32)


@pytest.fixture(autouse=True)
def no_timeouts():
    yield
    assert r.rope3d_testing_ffn_wait_timeouts() == 0
    assert r.rope3d_testing_norm_wait_timeouts() == 0


class Views:
    """Matrices as views of wider buffers (or contiguous), filled with normal values;
    `untouched` checks what lies beside them."""

    def __init__(self, rng):
        self.rng, self.kept = rng, []
        self.gen = torch.Generator(device=DEV).manual_seed(rng.randrange(1 << 30))

    def __call__(self, rows, cols, dtype, scale=1.0, shift=0.0):
        off, pad = self.rng.choice(((0, 0), (0, 0), (8, 8), (self.rng.randint(0, 9), self.rng.randint(0, 17))))
        buf = (torch.randn((rows + 2, cols + off + pad), generator=self.gen, device=DEV) * scale + shift).to(dtype)
        view = buf[1:-1, off:off + cols]
        self.kept.append((buf, view, buf.clone()))
        return view

    def untouched(self):
        for buf, view, was in self.kept:
            view.fill_(0.0)
            was[1:-1][:, view.storage_offset() % buf.stride(0):][:, :view.shape[1]] = 0.0
            assert torch.equal(buf, was)


def size(rng, top):
    n = int(top ** rng.random())
    return max(1, n if rng.random() < 0.5 else -(-n // 8) * 8)


@pytest.mark.parametrize("seed", range(80))
def test_norms(seed):
    rng = random.Random(1000 + seed)
    views = Views(rng)
    channels = size(rng, 9000)
    rows = min(size(rng, 8000), max(1, 3_000_000 // channels))
    dt = rng.choice(TYPES)
    pt = rng.choice((dt, torch.float32))
    y, post, pre = rng.random() < 0.75, rng.randrange(3), rng.randrange(3)
    a = dict(x=views(rows, channels, dt, 2.0, 0.3), post=post, pre=pre, eps=1e-5, residual_scale=rng.choice((1.0, 0.5, -1.5)),
             weight_offset=rng.choice((0.0, 1.0)), rows_per_group=rng.choice((rows, 1, 2, rng.randint(1, rows))))
    if y:
        a["y"] = views(rows, channels, dt, 0.7, -0.2)
    groups = -(-rows // a["rows_per_group"])
    for name, wanted in (("post_weight", y and post), ("pre_weight", True)):
        if wanted and rng.random() < 0.6:
            a[name] = (torch.randn(channels, generator=views.gen, device=DEV) * 0.1 + 1.0).to(pt)
    for name, wanted in (("gate", y), ("scale", True), ("shift", True)):
        if wanted and rng.random() < 0.5:
            a[name] = views(groups, channels, pt, 0.3)
    out = dict(r=views(rows, channels, dt), n=views(rows, channels, dt))
    got = r.rope3d_block_norm(**a, **out)
    want = ref.norm64(**a)
    for name, t in zip("rn", got):
        ref.check(t, want[name], name)
    dr, dn = views(rows, channels, dt), views(rows, channels, dt)
    given = dict(dr=None if rng.random() < 0.2 else dr.clone(), dn=dn.clone())
    want = ref.norm64(**a, **given, grads=True)
    in_place = given["dr"] is not None and rng.random() < 0.3
    to = dict(dx=dr if in_place else views(rows, channels, dt))
    if y:
        to["dy"] = dn if in_place else views(rows, channels, dt)
    grads = r.rope3d_block_norm_backward(**a, dr=None if given["dr"] is None else dr, dn=dn, **to)
    assert set(grads) == set(want)
    for name, t in grads.items():
        ref.check(t, want[name], name)
    views.untouched()


@pytest.mark.parametrize("seed", range(60))
def test_feed_forward(seed):
    rng = random.Random(2000 + seed)
    views = Views(rng)
    tokens, width, hidden = size(rng, 900), size(rng, 700), size(rng, 1500)
    dt, act = rng.choice(TYPES[:2]), rng.randrange(3)
    x, dy = views(tokens, width, dt), views(tokens, width, dt)
    w = [views(hidden, width, dt, width ** -0.5), views(hidden, width, dt, width ** -0.5),
         views(width, hidden, dt, hidden ** -0.5)]
    kept = rng.choice((None, dt, torch.float32))
    pre = () if kept is None else views(2 * tokens, hidden, kept).split(tokens)   # (they share a row stride)
    y = views(tokens, width, dt)
    r.rope3d_gated_ffn(x, *w, act=act, y=y, **dict(zip(("gate_pre", "up_pre"), pre)))
    want = ref.ffn64(x, *w, act)
    ref.check(y, want["y"], "y")
    for t, name in zip(pre, "gu"):
        value, bound = want[name]
        if kept is not torch.float32:
            bound = bound + ref.half_step(kept) * (value.abs() + bound) + ref.tiny(kept)
        ref.check(t, (value, bound), name)
    need = rng.choice(((True, True, True), (True, False, False), (False, True, True), (True, True, False)))
    names = ("dx", "dw_gate", "dw_up", "dw_down")
    out = {}
    for name, wanted, like in zip(names, (need[0], need[1], need[1], need[2]), (x, *w)):
        if wanted:
            out[name] = views(*like.shape, dt)
    grads = r.rope3d_gated_ffn_backward(dy, x, *w, *pre, act=act, need=need, **out)
    want = ref.ffn_backward64(dy, x, *w, act, *pre)
    for name, t in zip(names, grads):
        assert (t is None) == (name not in out)
        if t is not None:
            ref.check(t, want[name], name)
    views.untouched()
