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
