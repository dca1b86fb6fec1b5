"""The transformer-block operators as a program uses them: a whole block half
(norm, feed-forward, norm with gate and residual) forward and backward, other
streams, captured graphs, in-place and strided views, memory next to outputs,
special values, offsets past 32 bits, two calls at once, refusals on the device."""
from __future__ import annotations

import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import rope_rope3d_apply_gb300 as r  # noqa: E402
from tests import block_reference as ref  # noqa: E402

DEV = torch.device("cuda:0")
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def no_timeouts():
    yield
    assert r.rope3d_testing_ffn_wait_timeouts() == 0
    assert r.rope3d_testing_norm_wait_timeouts() == 0


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, shape, dtype=BF, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def ffn_weights(g, width, hidden, dtype=BF):
    return (normal(g, (hidden, width), dtype, width ** -0.5), normal(g, (hidden, width), dtype, width ** -0.5),
            normal(g, (width, hidden), dtype, hidden ** -0.5))


class Half:
    """The feed-forward half of a block: n = mod(rms(x)); y = ffn(n); out, next =
    x + gate * rms(y) and its norm. Forward, and backward by hand."""

    def __init__(self, tokens, width, hidden, dtype=BF, groups=2, seed=0):
        g = gen(seed)
        self.x = normal(g, (tokens, width), dtype)
        self.w = ffn_weights(g, width, hidden, dtype)
        self.mod = normal(g, (groups, 3, width), dtype, 0.3)
        self.pw, self.qw = normal(g, (width,), dtype, 0.1), normal(g, (width,), dtype, 0.1)
        self.d_out, self.d_next = normal(g, (tokens, width), dtype), normal(g, (tokens, width), dtype)
        self.pre = dict(pre=r.NORM_RMS, scale=self.mod[:, 0], shift=self.mod[:, 1])
        self.post = dict(post=r.NORM_RMS, pre=r.NORM_RMS, post_weight=self.pw, pre_weight=self.qw, gate=self.mod[:, 2],
                         weight_offset=1.0)

    def forward(self, stream=None):
        _, n = r.rope3d_block_norm(self.x, **self.pre, stream=stream)
        y, g, u = r.rope3d_gated_ffn(n, *self.w, act=r.ACT_GELU_TANH, keep=True, stream=stream)
        out, nxt = r.rope3d_block_norm(self.x, y, **self.post, stream=stream)
        return out, nxt, (n, y, g, u)

    def backward(self, kept, stream=None):
        n, y, g, u = kept
        a = r.rope3d_block_norm_backward(self.x, y, self.d_out, self.d_next, **self.post, stream=stream)
        dn, *dw = r.rope3d_gated_ffn_backward(a["dy"], n, *self.w, g, u, act=r.ACT_GELU_TANH, stream=stream)
        b = r.rope3d_block_norm_backward(self.x, dr=a["dx"], dn=dn, **self.pre, stream=stream)
        return dict(dx=b["dx"], dw_gate=dw[0], dw_up=dw[1], dw_down=dw[2], d_scale=b["d_scale"], d_shift=b["d_shift"],
                    d_gate=a["d_gate"], d_post_weight=a["d_post_weight"], d_pre_weight=a["d_pre_weight"])

    def reference(self):
        """Outputs and gradients in 64 bits, by automatic differentiation."""
        leaf = {k: v.double().requires_grad_() for k, v in
                dict(x=self.x, wg=self.w[0], wu=self.w[1], wd=self.w[2], mod=self.mod, pw=self.pw, qw=self.qw).items()}
        rows, G = self.x.shape[0], self.mod.shape[0]
        rms = lambda v: v * (v.square().mean(1, keepdim=True) + 1e-6).rsqrt()  # noqa: E731
        m = leaf["mod"].repeat_interleave(rows // G, 0)
        n = rms(leaf["x"]) * (1 + m[:, 0]) + m[:, 1]
        h = torch.nn.functional.gelu(n @ leaf["wg"].T, approximate="tanh") * (n @ leaf["wu"].T)
        y = h @ leaf["wd"].T
        out = leaf["x"] + m[:, 2] * (rms(y) * (1 + leaf["pw"]))
        nxt = rms(out) * (1 + leaf["qw"])
        got = torch.autograd.grad([out, nxt], list(leaf.values()), [self.d_out.double(), self.d_next.double()])
        d = dict(zip(leaf, got))
        return out.detach(), nxt.detach(), dict(
            dx=d["x"], dw_gate=d["wg"], dw_up=d["wu"], dw_down=d["wd"], d_scale=d["mod"][:, 0], d_shift=d["mod"][:, 1],
            d_gate=d["mod"][:, 2], d_post_weight=d["pw"], d_pre_weight=d["qw"])


# Roundings to the 16-bit type along the longest path of a block half: n, h, y (and
# the kept sums of nothing), the output; backward dy, dg and du, dn, dr, the result.
# Each is off by at most u = half a step of its value, at random; their sum in the
# 2-norm of a whole output is below u times their number (the norms and the products
# do not enlarge a relative error of a whole row by more than their condition, here
# below 2: rms and gelu slopes of at most 1.13 between orthogonal-like weights).
def near(got, want, roundings, dtype):
    off = float((got.double() - want).norm() / want.norm())
    assert off <= 2 * roundings * ref.half_step(dtype), off


@pytest.mark.parametrize("tokens,width,hidden,dtype", [(2, 256, 512, BF), (64, 512, 1024, BF), (400, 512, 1536, BF),
                                                       (1024, 1024, 2048, torch.float16), (90, 101, 307, BF)])
def test_block_half(tokens, width, hidden, dtype):
    half = Half(tokens, width, hidden, dtype)
    out, nxt, kept = half.forward()
    grads = half.backward(kept)
    want_out, want_nxt, want = half.reference()
    near(out, want_out, 4, dtype)
    near(nxt, want_nxt, 4, dtype)
    for k, v in grads.items():
        near(v, want[k], 9, dtype)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_other_streams():
    """The whole half on a side stream, by the stream argument and by torch's
    current stream, while the default stream is busy with other work."""
    half = Half(700, 512, 1024)
    want_f = half.forward()
    want_b = half.backward(want_f[2])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.zeros(1 << 26, device=DEV)
    for how in ("argument", "handle", "current"):
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(8):
            busy.add_(1.0)
        if how == "current":
            with torch.cuda.stream(side):
                f = half.forward()
                b = half.backward(f[2])
        else:
            s = side if how == "argument" else side.cuda_stream
            f = half.forward(stream=s)
            b = half.backward(f[2], stream=s)
        for _ in range(8):   # (workspaces freed by now must not be handed to this)
            torch.empty(1 << 22, device=DEV).fill_(-1.0)
        torch.cuda.synchronize()
        assert same(f[:2], want_f[:2]) and same(b.values(), want_b.values()), how


def test_other_stream_takes_no_pending_memory():
    """Memory freed on the current stream whose reader is still pending there is not
    what a call on another stream writes to; what such a call returned is not given
    away while the current stream still reads it."""
    rows, channels, hidden = 512, 1024, 2048
    g = gen(21)
    x, y, w = normal(g, (rows, channels)), normal(g, (rows, channels)), ffn_weights(g, channels, hidden)
    calls = {
        "norm": lambda **k: r.rope3d_block_norm(x, y, post=r.NORM_RMS, **k),
        "norm backward": lambda **k: tuple(r.rope3d_block_norm_backward(x, y, x, y, post=r.NORM_RMS, **k).values()),
        "ffn": lambda **k: r.rope3d_gated_ffn(x, *w, keep=BF, **k),
        "ffn backward": lambda **k: r.rope3d_gated_ffn_backward(y, x, *w, **k),
    }
    side = torch.cuda.Stream()
    for name, call in calls.items():
        want = call(stream=side)   # (memory of every size is there afterwards)
        torch.cuda.synchronize()
        sizes = [t.numel() for t in want] + [rows * hidden, rows * hidden * 2, 1 << 23]
        held = [torch.full((n,), 3.0, dtype=BF, device=DEV) for n in sizes]
        copies = [torch.empty_like(t) for t in held]
        torch.cuda.synchronize()
        torch.cuda._sleep(200_000_000)
        for c, t in zip(copies, held):
            c.copy_(t)
        del held, t
        out = call(stream=side.cuda_stream)
        side.synchronize()
        torch.cuda.synchronize()
        assert all(bool((c == 3.0).all()) for c in copies), name
        assert same(out, want), name
        # read behind a delay on the current stream, freed before that, then other work on the side stream
        torch.cuda._sleep(200_000_000)
        copies = [t.clone() for t in out]
        del out
        with torch.cuda.stream(side):
            for t in want:
                torch.empty_like(t).fill_(-1.0)
        torch.cuda.synchronize()
        assert same(copies, want), name


@pytest.mark.parametrize("tokens", [1, 50, 300])
def test_captured_graphs(tokens):
    """Forward and backward captured and replayed with new inputs; a second graph of
    other sizes replayed in between; eager calls before and after."""
    half, other = Half(tokens, 256, 768, groups=1), Half(tokens + 100, 512, 256, groups=1, seed=3)
    graphs = []
    for h in (half, other):
        h.backward(h.forward()[2])   # (the first call of a kernel sets its attributes)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f = h.forward()
            b = h.backward(f[2])
        graphs.append((h, g, f, b))
    for seed in (11, 12):
        for h, g, f, b in graphs:
            h.x.copy_(normal(gen(seed), h.x.shape))
            h.d_out.copy_(normal(gen(seed + 100), h.x.shape))
        for h, g, f, b in graphs:
            g.replay()
        graphs[0][1].replay()
        torch.cuda.synchronize()
        for h, g, f, b in graphs:
            want_f = h.forward()
            want_b = h.backward(want_f[2])
            torch.cuda.synchronize()
            assert same(f[:2], want_f[:2])
            assert same(b.values(), want_b.values())


def test_two_calls_at_once():
    """Threads with streams of their own: the same bits as one after the other."""
    halves = [Half(300, 256, 512, seed=s) for s in range(4)] + [Half(20, 512, 256, seed=9), Half(1, 256, 1024, groups=1)]
    want = [(h.forward(), h) for h in halves]
    want = [(f, h.backward(f[2]), h) for f, h in want]
    torch.cuda.synchronize()
    errors = []

    def work(f, b, h):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                f2 = h.forward()
                b2 = h.backward(f2[2])
                s.synchronize()
                if not (same(f2[:2], f[:2]) and same(b2.values(), b.values())):
                    errors.append(h.x.shape)

    threads = [threading.Thread(target=work, args=w) for w in want]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors


@pytest.mark.parametrize("rows,channels,dtype", [(9, 256, BF), (9, 77, BF), (3, 20000, BF), (5000, 768, BF), (9, 77, torch.float32)])
def test_norm_in_place(rows, channels, dtype):
    g = gen(1)
    x, y, w = normal(g, (rows, channels), dtype), normal(g, (rows, channels), dtype), normal(g, (channels,), dtype)
    kw = dict(post=r.NORM_LAYER, pre=r.NORM_RMS, post_weight=w, pre_weight=w)
    want = r.rope3d_block_norm(x, y, **kw)
    for r_is_x in (True, False):
        a, b = x.clone(), y.clone()
        r.rope3d_block_norm(a, b, **kw, r=a if r_is_x else b, n=b if r_is_x else a)
        assert torch.equal(a if r_is_x else b, want[0]) and torch.equal(b if r_is_x else a, want[1])
    dr, dn = normal(g, (rows, channels), dtype), normal(g, (rows, channels), dtype)
    want = r.rope3d_block_norm_backward(x, y, dr, dn, **kw)
    for dx_is_dr in (True, False):
        a, b = dr.clone(), dn.clone()
        got = r.rope3d_block_norm_backward(x, y, a, b, **kw, dx=a if dx_is_dr else b, dy=b if dx_is_dr else a)
        for k, v in got.items():
            assert torch.equal(v, want[k]), k


@pytest.mark.parametrize("rows,channels,off", [(40, 256, 8), (40, 256, 3), (5000, 512, 16), (40, 91, 5)])
def test_norm_strided_views_and_their_neighbours(rows, channels, off):
    """Column slices of wider buffers: the same bits as contiguous tensors, and
    nothing beside the outputs changes."""
    g = gen(2)

    def wide(fill=None):
        t = normal(g, (rows + 2, channels + off + 24)) if fill is None else torch.full((rows + 2, channels + off + 24), fill, dtype=BF, device=DEV)
        return t, t[1:-1, off:off + channels]

    (_, x), (_, y), (_, dr), (_, dn) = (wide() for _ in range(4))
    w = normal(g, (channels,))
    kw = dict(post=r.NORM_RMS, pre=r.NORM_LAYER, post_weight=w, pre_weight=w)
    want = r.rope3d_block_norm(x.contiguous(), y.contiguous(), **kw)
    (rb, ro), (nb, no) = wide(7.0), wide(9.0)
    r.rope3d_block_norm(x, y, **kw, r=ro, n=no)
    if (channels + off + 24) % 8 == 0 and off % 8 == 0 or channels % 8:
        assert torch.equal(ro, want[0]) and torch.equal(no, want[1])
    for (buf, view, fill), v in zip(((rb, ro, 7.0), (nb, no, 9.0)), (ref.norm64(x, y, **kw)["r"], ref.norm64(x, y, **kw)["n"])):
        ref.check(view, v)
        keep = buf.clone()
        keep[1:-1, off:off + channels] = fill
        assert bool((keep == fill).all())
    (xb, dx), (yb, dy) = wide(7.0), wide(9.0)
    got = r.rope3d_block_norm_backward(x, y, dr, dn, **kw, dx=dx, dy=dy)
    want = ref.norm64(x, y, dr, dn, grads=True, **kw)
    for k, v in got.items():
        ref.check(v, want[k], k)
    for buf, fill in ((xb, 7.0), (yb, 9.0)):
        buf[1:-1, off:off + channels] = fill
        assert bool((buf == fill).all())


@pytest.mark.parametrize("tokens,width,hidden,off", [(7, 64, 128, 8), (7, 64, 128, 1), (300, 136, 264, 8), (300, 136, 264, 3),
                                                     (200, 65, 33, 2)])
def test_ffn_strided_views_and_their_neighbours(tokens, width, hidden, off):
    """Slices of wider buffers, gate and up halves of one matrix, and the memory
    around every output."""
    g = gen(5)

    def wide(rows, cols, fill=None, scale=1.0):
        shape = (rows + 2, cols + off + 16)
        t = normal(g, shape, BF, scale) if fill is None else torch.full(shape, fill, dtype=BF, device=DEV)
        return t, t[1:-1, off:off + cols]

    x, dy = wide(tokens, width)[1], wide(tokens, width)[1]
    w2 = wide(2 * hidden, width, scale=width ** -0.5)[1]
    wg, wu, wd = w2[:hidden], w2[hidden:], wide(width, hidden, scale=hidden ** -0.5)[1]
    bufs = {n: wide(rows, cols, 5.0) for n, rows, cols in (
        ("y", tokens, width), ("g", tokens, hidden), ("u", tokens, hidden), ("dx", tokens, width), ("dg", 2 * hidden, width),
        ("dd", width, hidden))}
    v = {k: b[1] for k, b in bufs.items()}
    r.rope3d_gated_ffn(x, wg, wu, wd, act=r.ACT_SILU, y=v["y"], gate_pre=v["g"], up_pre=v["u"])
    r.rope3d_gated_ffn_backward(dy, x, wg, wu, wd, v["g"], v["u"], act=r.ACT_SILU, dx=v["dx"], dw_gate=v["dg"][:hidden],
                                dw_up=v["dg"][hidden:], dw_down=v["dd"])
    want = ref.ffn64(x, wg, wu, wd, 0)
    ref.check(v["y"], want["y"], "y")
    for k in "gu":
        val, err = want[k]
        ref.check(v[k], (val, err + ref.half_step(BF) * val.abs()), k)
    want = ref.ffn_backward64(dy, x, wg, wu, wd, 0, v["g"], v["u"])
    ref.check(v["dx"], want["dx"], "dx")
    ref.check(v["dg"][:hidden], want["dw_gate"], "dw_gate")
    ref.check(v["dg"][hidden:], want["dw_up"], "dw_up")
    ref.check(v["dd"], want["dw_down"], "dw_down")
    for name, (buf, view) in bufs.items():
        view.fill_(5.0)
        assert bool((buf == 5.0).all()), name


@pytest.mark.parametrize("pre", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("mod,off", [(2, 2), (4, 4), (4, 2), (6, 1), (1, 4), (0, 4), (0, 8)])
@pytest.mark.parametrize("tokens,width,hidden", [(5, 67, 131), (140, 65, 130), (300, 131, 67), (600, 523, 1301)])
def test_ffn_rows_of_every_alignment(tokens, width, hidden, mod, off, pre):
    """Rows that start on 2, 4 and 8 bytes and end inside a word, and their neighbours."""
    g = gen(tokens + mod + off)

    def wide(rows, cols, fill=None, scale=1.0, dtype=BF):
        ld = cols + off + 1
        ld += (mod - ld) % 8
        t = normal(g, (rows + 2, ld), BF, scale) if fill is None else torch.full((rows + 2, ld), fill, dtype=dtype, device=DEV)
        return t, t[1:-1, off:off + cols]

    x, dy = wide(tokens, width)[1], wide(tokens, width)[1]
    wg, wu = (wide(hidden, width, scale=width ** -0.5)[1] for _ in range(2))
    wd = wide(width, hidden, scale=hidden ** -0.5)[1]
    bufs = {n: wide(rows, cols, 5.0, dtype=dt) for n, rows, cols, dt in (
        ("y", tokens, width, BF), ("g", tokens, hidden, pre), ("u", tokens, hidden, pre), ("dx", tokens, width, BF),
        ("dw_gate", hidden, width, BF), ("dw_up", hidden, width, BF), ("dw_down", width, hidden, BF))}
    v = {k: b[1] for k, b in bufs.items()}
    r.rope3d_gated_ffn(x, wg, wu, wd, act=r.ACT_SILU, y=v["y"], gate_pre=v["g"], up_pre=v["u"])
    r.rope3d_gated_ffn_backward(dy, x, wg, wu, wd, v["g"], v["u"], act=r.ACT_SILU,
                                **{k: v[k] for k in ("dx", "dw_gate", "dw_up", "dw_down")})
    want = ref.ffn64(x, wg, wu, wd, 0)
    ref.check(v["y"], want["y"], "y")
    for k in "gu":
        val, err = want[k]
        ref.check(v[k], (val, err + (ref.half_step(BF) * val.abs() if pre is BF else 0.0)), k)
    want = ref.ffn_backward64(dy, x, wg, wu, wd, 0, v["g"], v["u"])
    for k in ("dx", "dw_gate", "dw_up", "dw_down"):
        ref.check(v[k], want[k], k)
    for name, (buf, view) in bufs.items():
        view.fill_(5.0)
        assert bool((buf == 5.0).all()), name


@pytest.mark.parametrize("tokens", [5, 300])
def test_special_values_stay_in_their_rows(tokens):
    """A NaN or an infinity in one token's row reaches that token's outputs alone."""
    g = gen(6)
    x, w = normal(g, (tokens, 192)), ffn_weights(g, 192, 320)
    y, gp, up = r.rope3d_gated_ffn(x, *w, keep=True)
    _, n = r.rope3d_block_norm(x)
    for bad in (float("nan"), float("inf"), -float("inf")):
        z = x.clone()
        z[2, 17] = bad
        y2, gp2, up2 = r.rope3d_gated_ffn(z, *w, keep=True)
        keep = torch.arange(tokens, device=DEV) != 2
        assert torch.equal(y2[keep], y[keep]) and torch.equal(gp2[keep], gp[keep]) and torch.equal(up2[keep], up[keep])
        assert bool((~torch.isfinite(gp2[2])).all()) and bool((~torch.isfinite(y2[2])).all())
        _, n2 = r.rope3d_block_norm(z)
        assert torch.equal(n2[keep], n[keep])
        assert not bool(torch.isfinite(n2[2]).all())
    # large pre-activations of either sign: the activation saturates, nothing turns NaN
    big = torch.full((tokens, 192), 3e4, dtype=BF, device=DEV)
    one = torch.zeros_like(w[0])
    one[:, 0] = torch.linspace(-1e4, 1e4, 320, device=DEV).to(BF)
    for act in (0, 1, 2):
        out = r.rope3d_gated_ffn(big, one, w[1], w[2], act=act)
        assert bool(torch.isfinite(out).all())
        grads = r.rope3d_gated_ffn_backward(x, big, one, w[1], w[2], act=act)
        assert all(bool(torch.isfinite(t).all()) for t in grads)
    # rows of zeros: their norm is zero, and their gradient finite
    zero = torch.zeros_like(x)
    _, n0 = r.rope3d_block_norm(zero)
    assert bool((n0 == 0).all())
    d = r.rope3d_block_norm_backward(zero, dn=x)
    assert bool(torch.isfinite(d["dx"]).all())


def test_gradients_against_differences():
    """<gradient, direction> against central differences of the 64-bit forward pass:
    off by at most the gradient's own bound along the direction, and the difference
    quotient's error (third derivative, here below 1e-5 of its value)."""
    g = gen(8)
    x, w, dy = normal(g, (150, 96)), ffn_weights(g, 96, 160), normal(g, (150, 96))
    got = r.rope3d_gated_ffn_backward(dy, x, *w, act=1)
    bound = ref.ffn_backward64(dy, x, *w, 1)
    args = [t.double() for t in (x, *w)]
    loss = lambda a: ((ref.act64(a[0] @ a[1].T, 1)[0] * (a[0] @ a[2].T)) @ a[3].T * dy.double()).sum()  # noqa: E731
    for i, name in enumerate(("dx", "dw_gate", "dw_up", "dw_down")):
        v = torch.randn(args[i].shape, generator=g, device=DEV, dtype=torch.float64)
        e = 1e-4
        lo, hi = list(args), list(args)
        lo[i], hi[i] = args[i] - e * v, args[i] + e * v
        diff = float((loss(hi) - loss(lo)) / (2 * e))
        own = float((got[i].double() * v).sum())
        assert abs(own - diff) <= float((bound[name][1] * v.abs()).sum()) + 1e-5 * abs(diff) + 1e-6, name
    y, dr, dn, wt = normal(g, (150, 96)), normal(g, (150, 96)), normal(g, (150, 96)), normal(g, (96,))
    kw = dict(post=2, pre=1, post_weight=wt, pre_weight=wt)
    out = r.rope3d_block_norm_backward(x, y, dr, dn, **kw)
    bound = ref.norm64(x, y, dr, dn, grads=True, **kw)

    def norm_loss(a, b):
        v = ref.norm64(a, b, **kw)
        return (v["r"][0] * dr.double()).sum() + (v["n"][0] * dn.double()).sum()

    for name, pick in (("dx", 0), ("dy", 1)):
        v = torch.randn(150, 96, generator=g, device=DEV, dtype=torch.float64)
        e = 1e-4
        moved = [(x.double() + s * e * v * (1 - pick), y.double() + s * e * v * pick) for s in (1, -1)]
        diff = float((norm_loss(*moved[0]) - norm_loss(*moved[1])) / (2 * e))
        own = float((out[name].double() * v).sum())
        assert abs(own - diff) <= float((bound[name][1] * v.abs()).sum()) + 1e-4 * abs(diff) + 1e-5, name


def test_norm_offsets_past_32_bits():
    """More than 2^32 bytes and 2^31 elements a tensor: rows from the far end."""
    rows, channels = 600_000, 4096
    x = torch.empty((rows, channels), dtype=BF, device=DEV)
    x.view(-1)[:] = 1.0
    g = gen(9)
    far = normal(g, (2000, channels))
    x[-2000:] = far
    y, w = x.flip(0), normal(g, (channels,))
    kw = dict(post=r.NORM_RMS, pre=r.NORM_RMS, post_weight=w, pre_weight=w)
    a, b = r.rope3d_block_norm(x, y, **kw)
    want = r.rope3d_block_norm(far.clone(), y[-2000:].clone(), **kw)
    assert torch.equal(a[-2000:], want[0]) and torch.equal(b[-2000:], want[1])
    got = r.rope3d_block_norm_backward(x, y, a, b, **kw)
    del a, b
    few = r.rope3d_block_norm_backward(far.clone(), y[-2000:].clone(), *want, **kw)
    assert torch.equal(got["dx"][-2000:], few["dx"]) and torch.equal(got["dy"][-2000:], few["dy"])


def test_ffn_offsets_past_32_bits():
    """tokens x hidden past 2^31: the same bits as a call of the last tokens alone."""
    tokens, width, hidden = 300_000, 64, 8192
    g = gen(10)
    x, w, dy = normal(g, (tokens, width)), ffn_weights(g, width, hidden), normal(g, (tokens, width))
    y, gp, up = r.rope3d_gated_ffn(x, *w, act=0, keep=BF)
    last = slice(tokens - 512, tokens)
    want = ref.ffn64(x[last], *w, 0)
    ref.check(y[last], want["y"], "y")
    ref.check(gp[last].float(), (want["g"][0], want["g"][1] + ref.half_step(BF) * want["g"][0].abs()), "gate_pre")
    dx = r.rope3d_gated_ffn_backward(dy, x, *w, gp, up, act=0, need=(True, False, False))[0]
    ref.check(dx[last], ref.ffn_backward64(dy[last], x[last], *w, 0, gp[last], up[last])["dx"], "dx")


def test_device_refusals():
    g = gen(11)
    x, w = normal(g, (4, 64)), ffn_weights(g, 64, 128)

    def status(call):
        with pytest.raises(r.Rope3dError) as e:
            call()
        return e.value.name

    assert status(lambda: r.rope3d_gated_ffn(x, w[0].cpu(), w[1], w[2])) == "ERR_DEVICE"
    assert status(lambda: r.rope3d_gated_ffn(x, *w, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))) == "ERR_SCRATCH"
    assert status(lambda: r.rope3d_gated_ffn(x, *w, y=x)) == "ERR_ALIAS"
    assert status(lambda: r.rope3d_gated_ffn_backward(x, x, *w, dx=x)) == "ERR_ALIAS"
    assert status(lambda: r.rope3d_block_norm(x, x.cpu())) == "ERR_DEVICE"
    assert status(lambda: r.rope3d_block_norm(x, x.clone(), n=x, r=x)) == "ERR_ALIAS"
    assert status(lambda: r.rope3d_block_norm(x, post_weight=x[0])) == "ERR_ARG"
    # nothing was written, and a sound call still works
    y = r.rope3d_gated_ffn(x, *w)
    ref.check(y, ref.ffn64(x, *w, 1)["y"])
