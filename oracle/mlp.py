"""Oracle of the gated feed-forward block, fp64: its definition and its gradients by the chain rule, each with a bound
on the error of an implementation with bf16 operands and results and fp32 arithmetic between them.

Half a step of bf16 is 2^-8 of the value; EPS32 = 2^-16 of the sum of the absolute terms covers fp32 products and sums
(a tensor-core sum over K terms and over the splits: below 2^-16 for K up to some 10^5 random terms), the activation's
approximation (relative error 1e-5 of Phi) and its exponential."""
from __future__ import annotations

import math

import torch

HALF = torch.finfo(torch.bfloat16).eps / 2
EPS32 = 2.0 ** -16


def _act(a, act):
    """(act, slope, bound of |slope| over small changes)"""
    if act == "silu":
        s = torch.sigmoid(a)
        return a * s, s * (1 + a * (1 - s))
    phi = torch.exp(-0.5 * a * a) / math.sqrt(2 * math.pi)
    cdf = 0.5 * torch.erfc(-a / math.sqrt(2.0))
    return a * cdf, cdf + a * phi


def full(x, w_gate, w_up, w_down, b_gate=None, b_up=None, b_down=None, act="silu", dy=None):
    """(results, bounds): y and, given dy, dx, dw_gate, dw_up, dw_down, db_gate, db_up, db_down (None if absent)."""
    d = lambda t: None if t is None else t.detach().cpu().double()  # noqa: E731
    x, wg, wu, wd, bg, bu, bd, dy = (d(t) for t in (x, w_gate, w_up, w_down, b_gate, b_up, b_down, dy))
    zero = lambda t, n: torch.zeros(n, dtype=torch.float64) if t is None else t  # noqa: E731
    F, C = wg.shape
    x = x.reshape(-1, C)
    a, u = x @ wg.t() + zero(bg, F), x @ wu.t() + zero(bu, F)
    ea = EPS32 * (x.abs() @ wg.abs().t() + zero(bg, F).abs())  # fp32 error of the two projections
    eu = EPS32 * (x.abs() @ wu.abs().t() + zero(bu, F).abs())
    f, slope = _act(a, act)
    # |act'| <= 1.13 and |act''| <= 1 for both activations
    ef = 1.13 * ea + EPS32 * (f.abs() + a.abs() * 2.0 ** -6)
    h = f * u
    eh = ef * u.abs() + f.abs() * eu + HALF * h.abs()
    y = h @ wd.t() + zero(bd, C)
    out = dict(y=y)
    err = dict(y=eh @ wd.abs().t() + EPS32 * (h.abs() @ wd.abs().t() + zero(bd, C).abs()) + HALF * y.abs())
    if dy is None:
        return out, err
    dy = dy.reshape(-1, C)
    dh = dy @ wd
    edh = EPS32 * (dy.abs() @ wd.abs())
    da, du = dh * u * slope, dh * f
    es = ea + EPS32
    eda = edh * (u * slope).abs() + dh.abs() * (eu * slope.abs() + u.abs() * es) + HALF * da.abs()
    edu = edh * f.abs() + dh.abs() * ef + HALF * du.abs()
    for name, v, e, terms in (
            ("dx", da @ wg + du @ wu, eda @ wg.abs() + edu @ wu.abs(), da.abs() @ wg.abs() + du.abs() @ wu.abs()),
            ("dw_gate", da.t() @ x, eda.t() @ x.abs(), da.abs().t() @ x.abs()),
            ("dw_up", du.t() @ x, edu.t() @ x.abs(), du.abs().t() @ x.abs()),
            ("dw_down", dy.t() @ h, dy.abs().t() @ eh, dy.abs().t() @ h.abs()),
            ("db_gate", da.sum(0), eda.sum(0), da.abs().sum(0)), ("db_up", du.sum(0), edu.sum(0), du.abs().sum(0)),
            ("db_down", dy.sum(0), 0 * dy.sum(0), dy.abs().sum(0))):
        out[name], err[name] = v, e + EPS32 * terms + HALF * v.abs()
    for name, b in (("db_gate", bg), ("db_up", bu), ("db_down", bd)):
        if b is None:
            out[name] = err[name] = None
    return out, err
