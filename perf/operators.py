"""The transformer-block operators, as cases to measure: the norms around a block
(with gate, residual scale and modulation) and the gated feed-forward, each with
its backward pass.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, rounded once at the end) or, where ``own`` is true, through this
framework's entry points. ``exact`` computes the same outputs in 64 bits from
the definitions, with the gradients by automatic differentiation.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---- cases -----------------------------------------------------------------
#
# Norm cases (op "norm" / "norm_bwd"):
#   r = res * x + gate * post(y) * wp,  n = pre(r) * wq * (1 + scale) + shift
# post / pre: "rms", "layer" or "none" (post "none" is the identity; y is absent
# where has_y is false, and then r is not an output); weights: both norms have a
# weight of their own, applied as offset + w; mod: gate, scale and shift, one
# row per group of consecutive rows (one sample).
#
# Feed-forward cases (op "ffn" / "ffn_bwd" / "ffn_train"):
#   y = (act(x Wg^T) * (x Wu^T)) Wd^T
# saved: the backward gets x Wg^T and x Wu^T as the forward pass kept them (in
# the inputs' type); otherwise it computes them again. fused: Wg and Wu are the
# halves of one matrix.


def _norm(name, op, rows, channels, dtype, has_y, post, pre, weights, mod, groups, res=1.0, offset=0.0):
    c = {"op": op, "rows": rows, "channels": channels, "dtype": dtype, "has_y": has_y, "post": post,
         "pre": pre, "weights": weights, "mod": mod, "groups": groups, "res": res, "offset": offset}
    return dict(c, name=name) if name else c


def _ffn(name, op, tokens, width, hidden, dtype, act, saved=False, fused=False):
    c = {"op": op, "tokens": tokens, "width": width, "hidden": hidden, "dtype": dtype, "act": act,
         "saved": saved, "fused": fused}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decoded token of a text model with norms before and after each block: latency
        _norm("norm_sandwich_token", "norm", 1, 4096, "bf16", True, "rms", "rms", True, False, 1, offset=1.0),
        # two video clips of 8 x 32 x 32 tokens in a diffusion block: gate, residual and the next modulated norm
        _norm("norm_modulated_video", "norm", 16384, 2048, "bf16", True, "none", "rms", False, True, 2),
        # odd sizes in float32 with a layer norm, before the first block (nothing to add yet)
        _norm("norm_layer_odd_f32", "norm", 1021, 1157, "f32", False, "none", "layer", True, True, 1),
        # training the text model's blocks: both norms' gradients
        _norm("norm_sandwich_bwd", "norm_bwd", 16384, 4096, "bf16", True, "rms", "rms", True, False, 1, offset=1.0),
        # training the diffusion blocks on four samples: gradients of the modulation too
        _norm("norm_modulated_bwd_f16", "norm_bwd", 8192, 2048, "f16", True, "none", "layer", False, True, 4, res=0.5),
        # one decoded token
        _ffn("ffn_token", "ffn", 1, 4096, 16384, "bf16", "gelu_tanh"),
        # a few tokens at a time: small batches of decoding
        _ffn("ffn_tokens_f16", "ffn", 24, 2048, 8192, "f16", "silu", fused=True),
        # one clip of 8 x 32 x 32 tokens, or a long prompt
        _ffn("ffn_clip", "ffn", 8192, 2048, 8192, "bf16", "gelu_tanh"),
        # odd sizes: no row of any matrix but the first starts on a 16-byte boundary
        _ffn("ffn_odd_f16", "ffn", 777, 1029, 2731, "f16", "gelu_erf"),
        # the backward pass from kept projections
        _ffn("ffn_bwd", "ffn_bwd", 2048, 2048, 8192, "bf16", "gelu_tanh", saved=True),
        # the backward pass that computes the projections again, at ragged sizes
        _ffn("ffn_bwd_ragged_f16", "ffn_bwd", 515, 1032, 2744, "f16", "silu", fused=True),
        # a training step: forward and backward
        _ffn("ffn_train", "ffn_train", 4096, 4096, 16384, "bf16", "silu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size, a multiple of 64 in half of the cases, of 8 in a quarter, any otherwise."""
    n = _log(rng, lo, hi)
    m = rng.choice((64, 64, 8, 1))
    return max(lo, n // m * m)


def draw(rng):
    if rng.random() < 0.45:
        rows, channels = _log(rng, 1, 32768), _size(rng, 64, 8192)
        rows = max(1, min(rows, (1 << 26) // channels))
        op = rng.choice(("norm", "norm_bwd"))
        has_y = rng.random() < 0.75
        groups = rng.randint(1, min(rows, 8))
        rows = rows // groups * groups
        mod = rng.random() < 0.6
        return _norm(None, op, rows, channels, rng.choice(("bf16", "f16", "f32")), has_y,
                     rng.choice(("none", "rms", "layer")) if has_y else "none", rng.choice(("rms", "layer")),
                     rng.random() < 0.6, mod, groups if mod else 1, rng.choice((1.0, 0.5)), rng.choice((0.0, 1.0)))
    op = rng.choice(("ffn", "ffn", "ffn_bwd", "ffn_train"))
    tokens, width, hidden = _log(rng, 1, 8192), _size(rng, 128, 4096), _size(rng, 256, 16384)
    tokens = max(1, min(tokens, (1 << 37) // (width * hidden)))
    return _ffn(None, op, tokens, width, hidden, rng.choice(("bf16", "f16")),
                rng.choice(("silu", "gelu_tanh", "gelu_erf")), rng.random() < 0.5, rng.random() < 0.5)


# ---- inputs ----------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(DTYPES[dtype])


def prepare(case, seed):
    g = _gen(seed)
    t = case["dtype"]
    s = {"case": case}
    if case["op"].startswith("norm"):
        R, C, G = case["rows"], case["channels"], case["groups"]
        # a residual stream: a few channels much larger than the others
        spread = 1.0 + 8.0 * (torch.rand((C,), generator=g, device="cuda") > 0.99).float()
        s["x"] = (torch.randn((R, C), generator=g, device="cuda") * spread * 2.0).to(DTYPES[t])
        s["y"] = _normal(g, (R, C), t, 0.7) if case["has_y"] else None
        w = case["weights"]
        mean = 1.0 - case["offset"]
        s["pre_weight"] = (mean + 0.1 * _normal(g, (C,), "f32")).to(DTYPES[t]) if w else None
        s["post_weight"] = (mean + 0.1 * _normal(g, (C,), "f32")).to(DTYPES[t]) if w and case["post"] != "none" else None
        # shift, scale and gate as a model's modulation layer gives them: thirds of one row a sample
        m = _normal(g, (G, 3, C), t, 0.3) if case["mod"] else None
        s["shift"], s["scale"], s["gate"] = (m[:, 0], m[:, 1], m[:, 2] if case["has_y"] else None) if case["mod"] else (None,) * 3
        if case["op"] == "norm_bwd":
            s["dr"] = _normal(g, (R, C), t, 0.5) if case["has_y"] else None
            s["dn"] = _normal(g, (R, C), t, 0.5)
        return s
    M, D, F = case["tokens"], case["width"], case["hidden"]
    s["x"] = _normal(g, (M, D), t)
    if case["fused"]:
        w = _normal(g, (2 * F, D), t, D ** -0.5)
        s["w_gate"], s["w_up"] = w[:F], w[F:]
    else:
        s["w_gate"], s["w_up"] = _normal(g, (F, D), t, D ** -0.5), _normal(g, (F, D), t, D ** -0.5)
    s["w_down"] = _normal(g, (D, F), t, F ** -0.5)
    if case["op"] != "ffn":
        s["dy"] = _normal(g, (M, D), t)
    if case["op"] == "ffn_bwd" and case["saved"]:
        s["gate_pre"] = (s["x"].float() @ s["w_gate"].float().T).to(DTYPES[t])
        s["up_pre"] = (s["x"].float() @ s["w_up"].float().T).to(DTYPES[t])
    return s


# ---- plain forms -----------------------------------------------------------


def _plain_stats(v, kind, eps):
    if kind == "none":
        return v, None
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    k = torch.rsqrt((v * v).mean(1, keepdim=True) + eps)
    return v * k, k


def _plain_norm_back(e, z, k, kind):
    if kind == "none":
        return e
    d = e - z * (e * z).mean(1, keepdim=True)
    if kind == "layer":
        d = d - e.mean(1, keepdim=True)
    return k * d


def _f32(t):
    return None if t is None else t.float()


def _rows(t, rows):
    """A group's row for each of its rows."""
    return None if t is None else t.repeat_interleave(rows // t.shape[0], 0)


def _plain_norm(s, eps=1e-6):
    c = s["case"]
    R, G, off = c["rows"], c["groups"], c["offset"]
    x, y = _f32(s["x"]), _f32(s["y"])
    wq = 1.0 if s["pre_weight"] is None else _f32(s["pre_weight"]) + off
    wp = 1.0 if s["post_weight"] is None else _f32(s["post_weight"]) + off
    scale, shift, gate = (_rows(_f32(s[k]), R) for k in ("scale", "shift", "gate"))
    r = x * c["res"]
    if y is not None:
        yh, ky = _plain_stats(y, c["post"], eps)
        p = yh * wp
        r = r + (p if gate is None else gate * p)
    z, kr = _plain_stats(r, c["pre"], eps)
    if c["op"] == "norm":
        n = z * wq
        if scale is not None:
            n = n * (1.0 + scale) + shift
        t = s["x"].dtype
        return {"r": None if y is None else r.to(t), "n": n.to(t)}
    dn = _f32(s["dn"])
    e = dn * wq
    if scale is not None:
        e = e * (1.0 + scale)
    dR = _plain_norm_back(e, z, kr, c["pre"])
    if s["dr"] is not None:
        dR = dR + _f32(s["dr"])
    t = s["x"].dtype
    out = {"dx": (dR * c["res"]).to(t)}
    if y is not None:
        f = dR * wp
        if gate is not None:
            f = f * gate
        out["dy"] = _plain_norm_back(f, yh, ky, c["post"]).to(t)
    per_group = lambda v: v.reshape(G, R // G, -1).sum(1)  # noqa: E731
    dz = dn * z
    if s["pre_weight"] is not None:
        out["d_pre_weight"] = (dz if scale is None else dz * (1.0 + scale)).sum(0).to(t)
    if scale is not None:
        out["d_scale"] = per_group(dz * wq).to(t)
        out["d_shift"] = per_group(dn).to(t)
    if y is not None:
        dp = dR * yh
        if s["post_weight"] is not None:
            out["d_post_weight"] = (dp if gate is None else dp * gate).sum(0).to(t)
        if gate is not None:
            out["d_gate"] = per_group(dp * wp).to(t)
    return out


def _plain_act(g, kind):
    """act(g) and act'(g)."""
    if kind == "silu":
        q = 1.0 / (1.0 + torch.exp(-g))
        return g * q, q * (1.0 + g * (1.0 - q))
    if kind == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        th = torch.tanh(k * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * k * (1.0 + 3 * 0.044715 * g * g)
    cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)


def _plain_ffn(s):
    c = s["case"]
    t = s["x"].dtype
    x, wg, wu, wd = (_f32(s[k]) for k in ("x", "w_gate", "w_up", "w_down"))
    if "gate_pre" in s:
        g, u = _f32(s["gate_pre"]), _f32(s["up_pre"])
    else:
        g, u = x @ wg.T, x @ wu.T
    a, da = _plain_act(g, c["act"])
    h = a * u
    out = {}
    if c["op"] != "ffn_bwd":
        out["y"] = (h @ wd.T).to(t)
    if c["op"] != "ffn":
        dy = _f32(s["dy"])
        dh = dy @ wd
        dg, du = dh * u * da, dh * a
        out["dx"] = (dg @ wg + du @ wu).to(t)
        out["dw_gate"], out["dw_up"], out["dw_down"] = (dg.T @ x).to(t), (du.T @ x).to(t), (dy.T @ h).to(t)
    return out


# ---- one pass --------------------------------------------------------------


def _own_norm(s):
    import rope_rope3d_apply_gb300 as rope3d

    c = s["case"]
    kind = {"none": rope3d.NORM_NONE, "rms": rope3d.NORM_RMS, "layer": rope3d.NORM_LAYER}
    kw = dict(post=kind[c["post"]], pre=kind[c["pre"]], post_weight=s["post_weight"], gate=s["gate"],
              pre_weight=s["pre_weight"], scale=s["scale"], shift=s["shift"], eps=1e-6,
              residual_scale=c["res"], weight_offset=c["offset"])
    if c["op"] == "norm":
        r, n = rope3d.rope3d_block_norm(s["x"], s["y"], **kw)
        return {"r": r, "n": n}
    return rope3d.rope3d_block_norm_backward(s["x"], s["y"], s["dr"], s["dn"], **kw)


def _own_ffn(s):
    import rope_rope3d_apply_gb300 as rope3d

    c = s["case"]
    act = {"silu": rope3d.ACT_SILU, "gelu_tanh": rope3d.ACT_GELU_TANH, "gelu_erf": rope3d.ACT_GELU_ERF}[c["act"]]
    w = (s["w_gate"], s["w_up"], s["w_down"])
    out, kept = {}, (s.get("gate_pre"), s.get("up_pre"))
    if c["op"] == "ffn":
        out["y"] = rope3d.rope3d_gated_ffn(s["x"], *w, act=act)
    elif c["op"] == "ffn_train":
        out["y"], *kept = rope3d.rope3d_gated_ffn(s["x"], *w, act=act, keep=True)
    if c["op"] != "ffn":
        out["dx"], out["dw_gate"], out["dw_up"], out["dw_down"] = rope3d.rope3d_gated_ffn_backward(
            s["dy"], s["x"], *w, *kept, act=act)
    return out


def run(state):
    if state["case"]["op"].startswith("norm"):
        out = _own_norm(state) if own else _plain_norm(state)
    else:
        out = _own_ffn(state) if own else _plain_ffn(state)
    return {k: v for k, v in out.items() if v is not None}


# ---- what a pass cannot do without -----------------------------------------


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"].startswith("norm"):
        R, C, G = case["rows"], case["channels"], case["groups"]
        y = 1 if case["has_y"] else 0
        small = (C * (1 + (1 if case["post"] != "none" else 0)) if case["weights"] else 0) + \
            (G * C * (2 + y) if case["mod"] else 0)
        if case["op"] == "norm":
            return {"bytes": e * (R * C * (2 + 2 * y) + small), "flops": 12 * R * C}
        return {"bytes": e * (R * C * (3 + 3 * y) + 2 * small), "flops": 30 * R * C}
    M, D, F = case["tokens"], case["width"], case["hidden"]
    w, x, hid = 3 * D * F, M * D, M * F
    if case["op"] == "ffn":
        return {"bytes": e * (w + 2 * x), "flops": 6 * M * D * F}
    if case["op"] == "ffn_bwd":
        if case["saved"]:
            return {"bytes": e * (2 * w + 3 * x + 2 * hid), "flops": 12 * M * D * F}
        return {"bytes": e * (2 * w + 3 * x), "flops": 16 * M * D * F}
    return {"bytes": e * (2 * w + 4 * x), "flops": 18 * M * D * F}


# ---- in 64 bits ------------------------------------------------------------


def _exact_norm(s, case):
    leaf = {k: s[k].double().requires_grad_() for k in
            ("x", "y", "post_weight", "gate", "pre_weight", "scale", "shift") if s[k] is not None}
    R, G, C = case["rows"], case["groups"], case["channels"]

    def norm(v, kind):
        if kind == "layer":
            var, mean = torch.var_mean(v, dim=-1, correction=0, keepdim=True)
            return (v - mean) / (var + 1e-6).sqrt()
        return v / (v.square().mean(-1, keepdim=True) + 1e-6).sqrt() if kind == "rms" else v

    def grouped(v, by):
        return (v.view(G, R // G, C) * by.unsqueeze(1)).view(R, C)

    total = leaf["x"] * case["res"]
    if "y" in leaf:
        p = norm(leaf["y"], case["post"])
        if "post_weight" in leaf:
            p = p * (case["offset"] + leaf["post_weight"])
        total = total + (grouped(p, leaf["gate"]) if "gate" in leaf else p)
    n = norm(total, case["pre"])
    if "pre_weight" in leaf:
        n = n * (case["offset"] + leaf["pre_weight"])
    if "scale" in leaf:
        n = (grouped(n, 1 + leaf["scale"]).view(G, R // G, C) + leaf["shift"].unsqueeze(1)).view(R, C)
    if case["op"] == "norm":
        return {"n": n.detach(), **({"r": total.detach()} if "y" in leaf else {})}
    outs, grads = [n], [s["dn"].double()]
    if "y" in leaf:
        outs.append(total)
        grads.append(s["dr"].double())
    got = torch.autograd.grad(outs, list(leaf.values()), grads)
    names = {"x": "dx", "y": "dy"}
    return {names.get(k, "d_" + k): v for k, v in zip(leaf, got)}


def _exact_ffn(s, case):
    x, wg, wu, wd = (s[k].double().requires_grad_(case["op"] != "ffn") for k in ("x", "w_gate", "w_up", "w_down"))
    g, u = torch.nn.functional.linear(x, wg), torch.nn.functional.linear(x, wu)
    if "gate_pre" in s:  # the values kept are the ones that count; gradients pass through them
        g, u = g + (s["gate_pre"].double() - g).detach(), u + (s["up_pre"].double() - u).detach()
    act = {"silu": lambda v: torch.nn.functional.silu(v),
           "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh"),
           "gelu_erf": lambda v: torch.nn.functional.gelu(v)}[case["act"]]
    y = torch.nn.functional.linear(act(g) * u, wd)
    out = {"y": y.detach()} if case["op"] != "ffn_bwd" else {}
    if case["op"] != "ffn":
        out.update(zip(("dx", "dw_gate", "dw_up", "dw_down"),
                       torch.autograd.grad(y, (x, wg, wu, wd), s["dy"].double())))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s, case) if case["op"].startswith("norm") else _exact_ffn(s, case)
