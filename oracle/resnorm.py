"""Oracle of the residual step, fp64: y = post(f), r = x + gate scale drop(y), n = pre(r), by its definition, and its
gradients by the chain rule.  Philox4x32-10 in Python integers.

`terms` has, for each result, the sum of the absolute values of the terms that it is made of.  An implementation in
fp32 is off by a few 2^-24 of those for each step of its sums: a sum over C <= 8192 channels held by L lanes, or over
the rows of a block, runs through at most some hundred additions, so 2^-16 of the terms covers it."""
from __future__ import annotations

import torch

M0, M1, W0, W1, LOW = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85, 0xFFFFFFFF


def philox4x32(counter, key):
    """Ten rounds on a 4-word counter with a 2-word key (J. K. Salmon et al., SC11)."""
    c, (k0, k1) = list(counter), key
    for _ in range(10):
        a, b = c[0] * M0, c[2] * M1
        c = [(b >> 32) ^ c[1] ^ k0, b & LOW, (a >> 32) ^ c[3] ^ k1, a & LOW]
        k0, k1 = (k0 + W0) & LOW, (k1 + W1) & LOW
    return c


def keep_mask(shape, p: float, seed: int, offset: int) -> torch.Tensor:
    total = 1
    for d in shape:
        total *= d
    seed, offset = seed & (2 ** 64 - 1), offset & (2 ** 64 - 1)
    words = []
    for i in range((total + 3) // 4):
        words += philox4x32((i & LOW, i >> 32, offset & LOW, offset >> 32), (seed & LOW, seed >> 32))
    thr = int(p * 2.0 ** 32)
    return torch.tensor([w >= thr for w in words[:total]]).reshape(shape)


def _norm(v, kind, eps, w, b):
    c = v - v.mean(-1, keepdim=True) if kind == "layer" else v
    dev = torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    hat = c / dev
    y = hat if w is None else hat * w
    return y if b is None else y + b, hat, dev


def _norm_back(dy, hat, dev, kind, w):
    t = dy if w is None else dy * w
    out = t - hat * (t * hat).mean(-1, keepdim=True)
    if kind == "layer":
        out = out - t.mean(-1, keepdim=True)
    return out / dev


def _norm_terms(a, hat, dev, w, b):
    t = (a + a.mean(-1, keepdim=True)) / dev + hat.abs()
    t = t if w is None else t * w.abs()
    return t if b is None else t + b.abs()


def _norm_back_terms(ady, hat, dev, w):
    t = ady if w is None else ady * w.abs()
    return (t + hat.abs() * (t * hat.abs()).mean(-1, keepdim=True) + t.mean(-1, keepdim=True)) / dev


def step(x, f, gate=None, scale=None, post=None, post_weight=None, post_bias=None, pre="layer", pre_weight=None,
         pre_bias=None, eps=1e-5, p=0.0, rng=None, dr=None, dn=None):
    """dict(r, n) and, given dr or dn, the gradients dx, df, dgate, dscale, dpost_weight, ... (fp64, CPU)."""
    d = lambda t: None if t is None else t.detach().cpu().double()  # noqa: E731
    x, f, gate, scale, post_weight, post_bias, pre_weight, pre_bias, dr, dn = (
        d(t) for t in (x, f, gate, scale, post_weight, post_bias, pre_weight, pre_bias, dr, dn))
    lead = (-1,) + (1,) * (x.dim() - 1)
    y, ay = f, f.abs()
    if post:
        y, hat_f, dev_f = _norm(f, post, eps, post_weight, post_bias)
        ay = _norm_terms(f.abs(), hat_f, dev_f, post_weight, post_bias)
    factor = torch.ones_like(x)
    if p > 0:
        factor = keep_mask(x.shape, p, *(int(t) for t in rng.tolist())).double() / (1.0 - p)
    y = torch.where(factor == 0, torch.zeros_like(y), y * factor)
    ay = torch.where(factor == 0, torch.zeros_like(y), ay * factor)
    au = ay if scale is None else ay * scale.abs()
    u = y if scale is None else y * scale
    g = None if gate is None else gate.reshape(lead).expand_as(x)
    r = x + (u if g is None else torch.where(g == 0, torch.zeros_like(u), g * u))
    out = dict(r=r, n=None)
    ar = x.abs() + (au if g is None else torch.where(g == 0, torch.zeros_like(u), g.abs() * au))
    terms = out["terms"] = dict(r=ar)
    if pre:
        out["n"], hat_r, dev_r = _norm(r, pre, eps, pre_weight, pre_bias)
        terms["n"] = _norm_terms(ar, hat_r, dev_r, pre_weight, pre_bias)
    if dr is None and dn is None:
        return out
    rows = tuple(range(x.dim() - 1))
    total = torch.zeros_like(x) if dr is None else dr
    at = total.abs()
    out |= dict.fromkeys(("dgate", "dscale", "dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias"))
    if pre and dn is not None:
        total = total + _norm_back(dn, hat_r, dev_r, pre, pre_weight)
        at = at + _norm_back_terms(dn.abs(), hat_r, dev_r, pre_weight)
    if pre:
        up = torch.zeros_like(x) if dn is None else dn
        out["dpre_weight"] = None if pre_weight is None else (up * hat_r).sum(rows)
        out["dpre_bias"] = None if pre_bias is None else up.sum(rows)
        terms["dpre_weight"] = (up.abs() * (_norm_terms(ar, hat_r, dev_r, None, None))).sum(rows)
        terms["dpre_bias"] = up.abs().sum(rows)
    du = total
    if g is not None:
        out["dgate"] = (total * u).sum(tuple(range(1, x.dim())))
        du = g * total
        terms["dgate"] = (at * au).sum(tuple(range(1, x.dim())))
    adu = at if g is None else at * g.abs()
    live = torch.ones_like(x, dtype=torch.bool) if g is None else g != 0
    if scale is not None:
        out["dscale"] = torch.where(live, du * y, torch.zeros_like(y)).sum(rows)
        terms["dscale"] = torch.where(live, adu * ay, torch.zeros_like(y)).sum(rows)
        du, adu = du * scale, adu * scale.abs()
    dy = torch.where(factor == 0, torch.zeros_like(du), du * factor)
    ady = adu * factor
    if post:
        out["dpost_weight"] = None if post_weight is None else torch.where(live, dy * hat_f, torch.zeros_like(dy)).sum(rows)
        out["dpost_bias"] = None if post_bias is None else dy.sum(rows)
        af = _norm_terms(f.abs(), hat_f, dev_f, None, None)
        terms["dpost_weight"] = torch.where(live, ady * af, torch.zeros_like(dy)).sum(rows)
        terms["dpost_bias"] = torch.where(live, ady, torch.zeros_like(dy)).sum(rows)
        dy = _norm_back(dy, hat_f, dev_f, post, post_weight)
        ady = _norm_back_terms(ady, hat_f, dev_f, post_weight)
    terms["dx"], terms["df"] = at, torch.where(live, ady, torch.zeros_like(dy))
    out["dx"], out["df"] = total, torch.where(live, dy, torch.zeros_like(dy))
    return out
