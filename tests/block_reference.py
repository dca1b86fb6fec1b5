"""The transformer-block operators in 64 bits, from their definitions, with a
bound on how far the library's outputs may be off, element by element.

A bound counts every rounding of the computation once: u = half a step of the
16-bit type for each value rounded to it (2^-8 bf16, 2^-11 fp16; fp16 also half
of the smallest subnormal, 2^-25), and for a sum of K products accumulated in
fp32, in any order, `accumulation(K)` times the sum of the products' magnitudes.
Errors of inputs of a step go through its derivative to first order; the
products of two errors that this leaves out are covered by `SLACK`.
"""
from __future__ import annotations

import math

import torch

SLACK = 1.02
FP32 = 2.0 ** -24


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def tiny(dtype) -> float:
    """Half of the smallest subnormal: the absolute part of a rounding."""
    return 2.0 ** -25 if dtype == torch.float16 else 0.0


def accumulation(k: int) -> float:
    """A tensor-core step adds 16 products and the accumulator with the bits
    below about 2^-23 of the largest cut off: at most 17 cut terms a step, each
    below 2^-23 of the largest magnitude, over ceil(k / 16) steps (and the steps
    of a split sum). 2^-21 a step and four steps of slack cover 17 terms where
    they differ in size as products of normal values do; a plain fp32 sum of k
    terms is at most k 2^-24."""
    return (math.ceil(k / 16) + 4) * 2.0 ** -21


def act64(g, kind):
    """act(g), act'(g) in 64 bits. kind: 0 silu, 1 gelu (tanh), 2 gelu (erf)."""
    if kind == 0:
        q = torch.sigmoid(g)
        return g * q, q * (1 + g * (1 - q))
    if kind == 1:
        k = math.sqrt(2 / math.pi)
        z = k * (g + 0.044715 * g ** 3)
        th = torch.tanh(z)
        return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * k * (1 + 3 * 0.044715 * g * g)
    c = 0.5 * torch.erfc(-g / math.sqrt(2))
    return g * c, c + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)


# |act'| and |act''| of the three activations stay below these (act' peaks at
# 1.13, act'' at 0.80); evaluating them in fp32 from exp or erf and a handful of
# multiplies costs at most ACT_EVAL relative to max(1, |g|).
ACT_SLOPE, ACT_CURVE, ACT_EVAL = 1.13, 0.8, 2.0 ** -19


def ffn64(x, w_gate, w_up, w_down, act):
    """y and its bound, from 16-bit inputs."""
    u16, t16 = half_step(x.dtype), tiny(x.dtype)
    x, wg, wu, wd = (t.double() for t in (x, w_gate, w_up, w_down))
    g, u = x @ wg.T, x @ wu.T
    D, F = wg.shape[1], wg.shape[0]
    ge, ue = accumulation(D) * (x.abs() @ wg.abs().T), accumulation(D) * (x.abs() @ wu.abs().T)
    a, _ = act64(g, act)
    h = a * u
    ae = ACT_SLOPE * ge + ACT_EVAL * g.abs().clamp(min=1)
    he = (ae * u.abs() + a.abs() * ue) * SLACK + u16 * h.abs() + t16
    y = h @ wd.T
    ye = he @ wd.abs().T + accumulation(F) * ((h.abs() + he) @ wd.abs().T)
    return {"y": (y, ye * SLACK + u16 * y.abs() + t16), "g": (g, ge), "u": (u, ue)}


def ffn_backward64(dy, x, w_gate, w_up, w_down, act, gate_pre=None, up_pre=None):
    """dx, dw_gate, dw_up, dw_down and their bounds; gate_pre / up_pre as kept."""
    u16, t16 = half_step(x.dtype), tiny(x.dtype)
    M, D = x.shape
    F = w_gate.shape[0]
    dy, x, wg, wu, wd = (t.double() for t in (dy, x, w_gate, w_up, w_down))
    if gate_pre is None:
        g, u = x @ wg.T, x @ wu.T
        ge, ue = accumulation(D) * (x.abs() @ wg.abs().T), accumulation(D) * (x.abs() @ wu.abs().T)
    else:
        g, u = gate_pre.double(), up_pre.double()
        ge = ue = torch.zeros_like(g)
    a, s = act64(g, act)
    ev = ACT_EVAL * g.abs().clamp(min=1)
    ae, se = ACT_SLOPE * ge + ev, ACT_CURVE * ge + ev
    dh = dy @ wd
    dhe = accumulation(D) * (dy.abs() @ wd.abs())
    dg, du, h = dh * u * s, dh * a, a * u
    dge = ((u * s).abs() * dhe + (dh * s).abs() * ue + (dh * u).abs() * se) * SLACK + u16 * dg.abs() + t16
    due = (a.abs() * dhe + dh.abs() * ae) * SLACK + u16 * du.abs() + t16
    he = (ae * u.abs() + a.abs() * ue) * SLACK + u16 * h.abs() + t16
    out = {}

    def put(name, value, err, mag, k):
        out[name] = (value, (err + accumulation(k) * mag) * SLACK + u16 * value.abs() + t16)

    put("dx", dg @ wg + du @ wu, dge @ wg.abs() + due @ wu.abs(), dg.abs() @ wg.abs() + du.abs() @ wu.abs(), 2 * F)
    put("dw_gate", dg.T @ x, dge.T @ x.abs(), dg.abs().T @ x.abs(), M)
    put("dw_up", du.T @ x, due.T @ x.abs(), du.abs().T @ x.abs(), M)
    put("dw_down", dy.T @ h, dy.abs().T @ he, dy.abs().T @ h.abs(), M)
    return out


def check(got, want, name=""):
    value, bound = want
    assert got.shape == value.shape, (name, got.shape, value.shape)
    off = (got.double() - value).abs()
    bad = ~(off <= bound)
    if bad.any():
        i = int((off / bound.clamp(min=1e-300)).nan_to_num(nan=math.inf).argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} values outside the bound, worst at {i}: "
                             f"{float(got.reshape(-1)[i])} for {float(value.reshape(-1)[i])} "
                             f"+- {float(bound.reshape(-1)[i])}")


# ---- the norms around a block ------------------------------------------------


def sum_error(n: int) -> float:
    """A sum of n fp32 terms as the kernels add them: at most n / 256 in a row on
    a thread (16 where a row is kept in registers), then trees of 32 and of the
    warps; each addition is off by half a step. 8 more steps for the terms."""
    return (n / 256 + 40) * FP32


def _stats(v, ve, kind, eps):
    """Normalised rows, 1 / std, and the errors: (h, h_err, k, k_rel)."""
    if kind == 0:
        return v, ve, torch.ones_like(v[:, :1]), torch.zeros_like(v[:, :1])
    C = v.shape[1]
    s = sum_error(C)
    mean = v.mean(1, keepdim=True) if kind == 2 else torch.zeros_like(v[:, :1])
    me = ve.mean(1, keepdim=True) + s * v.abs().mean(1, keepdim=True) if kind == 2 else torch.zeros_like(mean)
    d = v - mean
    de = ve + me + FP32 * d.abs()
    var = (d * d).mean(1, keepdim=True) + eps
    var_rel = ((2 * d.abs() + de) * de).mean(1, keepdim=True) / var + s + 2 * FP32
    k, k_rel = var.rsqrt(), 0.5 * var_rel * SLACK + 4 * FP32
    h = d * k
    return h, (h.abs() * (k_rel + 2 * FP32) + de * k) * SLACK, k, k_rel


def _spread(t, rows, rpg, fill):
    if t is None:
        return fill
    return t.double().repeat_interleave(rpg, 0)[:rows]


def norm64(x, y=None, dr=None, dn=None, post=0, pre=1, post_weight=None, gate=None, pre_weight=None, scale=None,
           shift=None, rows_per_group=None, eps=1e-6, residual_scale=1.0, weight_offset=0.0, grads=False):
    """r and n (grads False) or every gradient, each with its bound."""
    R, C = x.shape
    dt, res = x.dtype, residual_scale
    params = [t for t in (post_weight, gate, pre_weight, scale, shift) if t is not None]
    pt = params[0].dtype if params else dt
    rpg = rows_per_group or R
    u, t, pu, ptiny = half_step(dt), tiny(dt), half_step(pt), tiny(pt)
    x64 = x.double()
    wq = 1.0 if pre_weight is None else pre_weight.double() + weight_offset
    wp = 1.0 if post_weight is None else post_weight.double() + weight_offset
    one = torch.ones(1, 1, dtype=torch.float64, device=x.device)
    wq, wp = wq * one, wp * one
    gt, sc = _spread(gate, R, rpg, 1.0) * one, 1.0 + _spread(scale, R, rpg, 0.0) * one
    sh = _spread(shift, R, rpg, 0.0) * one
    F = 8 * FP32   # the handful of fp32 operations of an element
    zero = torch.zeros_like(x64)
    r, re = res * x64, F * (res * x64).abs()
    if y is not None:
        yh, yhe, ky, ky_rel = _stats(y.double(), zero, post, eps)
        m = gt * wp
        r = r + m * yh
        re = re + (m.abs() * yhe + F * (m * yh).abs()) * SLACK
    z, ze, kr, kr_rel = _stats(r, re, pre, eps)
    if not grads:
        n = z * wq * sc + sh
        ne = ((wq * sc).abs() * ze + F * ((z * wq * sc).abs() + sh.abs())) * SLACK
        return {"r": (r, re + u * r.abs() + t), "n": (n, ne + u * n.abs() + t)}
    d_n = zero if dn is None else dn.double()
    d_r = zero if dr is None else dr.double()
    s = sum_error(C)
    e = d_n * wq * sc
    ee = F * e.abs()
    mean = lambda v: v.mean(1, keepdim=True)  # noqa: E731
    if pre == 0:
        dR, dRe = d_r + e, ee + F * d_r.abs()
    else:
        me = mean(e) if pre == 2 else torch.zeros_like(kr)
        mee = (mean(ee) + s * mean(e.abs())) if pre == 2 else torch.zeros_like(kr)
        mez = mean(e * z)
        meze = (mean(ee * z.abs() + e.abs() * ze) + s * mean((e * z).abs()) + 4 * FP32 * mez.abs()) * SLACK
        inner = e - me - z * mez
        innere = (ee + mee + ze * mez.abs() + z.abs() * meze + F * (e.abs() + me.abs() + (z * mez).abs())) * SLACK
        dR = d_r + kr * inner
        dRe = (kr * innere + kr * inner.abs() * kr_rel + F * (d_r.abs() + (kr * inner).abs())) * SLACK
    out = {"dx": (res * dR, abs(res) * dRe * (1 + F) + F * (res * dR).abs() + u * (res * dR).abs() + t)}
    if y is not None:
        f = dR * m
        fe = (dRe * m.abs() + F * f.abs()) * SLACK
        if post == 0:
            out["dy"] = (f, fe + u * f.abs() + t)
        else:
            mf = mean(f) if post == 2 else torch.zeros_like(ky)
            mfe = (mean(fe) + s * mean(f.abs())) if post == 2 else torch.zeros_like(ky)
            mfy = mean(f * yh)
            mfye = (mean(fe * yh.abs() + f.abs() * yhe) + s * mean((f * yh).abs()) + 4 * FP32 * mfy.abs()) * SLACK
            inner = f - mf - yh * mfy
            innere = (fe + mfe + yhe * mfy.abs() + yh.abs() * mfye + F * (f.abs() + mf.abs() + (yh * mfy).abs())) * SLACK
            dy = ky * inner
            out["dy"] = (dy, (ky * innere + dy.abs() * (ky_rel + F)) * SLACK + u * dy.abs() + t)

    G = -(-R // rpg)
    g_of = torch.arange(R, device=x.device) // rpg

    def by_group(v):
        return torch.zeros((G, C), dtype=torch.float64, device=x.device).index_add_(0, g_of, v.expand(R, C).contiguous())

    # rows are added one by one at most, then chunks and groups
    sr = (R + 40) * FP32

    def column(term, err):
        mag = by_group(term.abs())
        return by_group(term), by_group(err) + sr * (mag + by_group(err)), mag

    def put(name, value, err, mag):
        out[name] = (value, (err + F * mag) * SLACK + pu * value.abs() + ptiny)

    gs = lambda v: 1.0 if v is None else v.double()  # noqa: E731
    S, Se, Sm = column(d_n * z, d_n.abs() * ze + F * (d_n * z).abs())
    T, Te, Tm = column(d_n, zero)
    if scale is not None:
        put("d_scale", wq * S, wq.abs() * Se, wq.abs() * Sm)
    if shift is not None:
        put("d_shift", T, Te, Tm)
    if pre_weight is not None:
        w = (1.0 + scale.double()) if scale is not None else torch.ones_like(S)
        put("d_pre_weight", (w * S).sum(0), (w.abs() * Se).sum(0) + sr * (w.abs() * Sm).sum(0), (w.abs() * Sm).sum(0))
    if y is not None:
        U, Ue, Um = column(dR * yh, dRe * yh.abs() + dR.abs() * yhe + F * (dR * yh).abs())
        if gate is not None:
            put("d_gate", wp * U, wp.abs() * Ue, wp.abs() * Um)
        if post_weight is not None:
            w = gs(gate) * torch.ones_like(U)
            put("d_post_weight", (w * U).sum(0), (w.abs() * Ue).sum(0) + sr * (w.abs() * Um).sum(0), (w.abs() * Um).sum(0))
    return out
