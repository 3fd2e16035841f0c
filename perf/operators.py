"""Cases that time and check the operators of a whole Swin layer around the windowed attention: attention with a
learned relative position bias, the residual step with its norms, gate, layer scale and dropout, and the gated
feed-forward block.

`run` computes them in plain elementary torch operations, or, where `own` is true, through this package."""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

D = 32  # channels of an attention head
BF16, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one small image through one layer: latency of a single inference call
        dict(name="relbias_fwd_tiny", op="relbias", train=False, B=1, H=16, W=16, heads=2, M=8, s=0, log=False),
        # first stage at patch 2 with 32 x 32 windows, shifted: the compute-bound forward
        dict(name="relbias_fwd_p2_m32", op="relbias", train=False, B=32, H=128, W=128, heads=3, M=32, s=16, log=False),
        # first stage at patch 4 with 8 x 8 windows, shifted: the memory-bound training step
        dict(name="relbias_train_p4_m8", op="relbias", train=True, B=64, H=64, W=64, heads=3, M=8, s=4, log=False),
        # detection grid (an 800 x 1333 image at patch 4), padded to the window; distances share log buckets
        dict(name="relbias_train_det_m16", op="relbias", train=True, B=2, H=200, W=334, heads=3, M=16, s=8, log=True),
        # the largest training step: 1024-token windows
        dict(name="relbias_train_p2_m32", op="relbias", train=True, B=16, H=128, W=128, heads=3, M=32, s=0, log=False),
        # one small image's residual step: latency
        dict(name="resnorm_fwd_tiny", op="resnorm", train=False, B=1, T=256, C=64, f32=False, pre="layer", post="none",
             affine=True, gate=False, scale=False, p=0.0),
        # first stage, stochastic depth per image
        dict(name="resnorm_fwd_stage1", op="resnorm", train=False, B=128, T=4096, C=96, f32=False, pre="layer",
             post="none", affine=True, gate=True, scale=False, p=0.0),
        # third stage in training: fp32 stream, bf16 branch, layer scale, dropout on the branch
        dict(name="resnorm_train_stage3", op="resnorm", train=True, B=64, T=256, C=384, f32=True, pre="layer",
             post="none", affine=True, gate=True, scale=True, p=0.1),
        # both norms (sandwich), an odd channel count that no vector width divides
        dict(name="resnorm_train_odd", op="resnorm", train=True, B=3, T=1111, C=1001, f32=False, pre="rms", post="rms",
             affine=True, gate=False, scale=False, p=0.0),
        # one small image's feed-forward block: latency
        dict(name="mlp_fwd_tiny", op="mlp", train=False, T=256, C=64, F=168, act="silu", bias=True),
        # first stage at inference: few channels, many tokens
        dict(name="mlp_fwd_stage1", op="mlp", train=False, T=524288, C=96, F=256, act="gelu", bias=True),
        # third stage in training
        dict(name="mlp_train_stage3", op="mlp", train=True, T=32768, C=384, F=1024, act="silu", bias=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["relbias", "resnorm", "mlp"])
    train = rng.random() < 0.5
    if op == "relbias":
        while True:
            M = rng.choice([4, 8, 16, 32, 64])
            c = dict(op=op, train=train, B=_log_uniform(rng, 1, 64), H=_log_uniform(rng, M, 256),
                     W=_log_uniform(rng, M, 256), heads=_log_uniform(rng, 1, 24), M=M, s=4 * rng.randrange(M // 4),
                     log=rng.random() < 0.4)
            Hp, Wp = -(-c["H"] // M) * M, -(-c["W"] // M) * M
            rows = c["B"] * Hp * Wp * c["heads"]
            if rows * M * M <= 1 << 29 and rows <= 1 << 20:
                return c
    if op == "resnorm":
        while True:
            C = _log_uniform(rng, 8, 2048)
            if rng.random() < 0.6:
                C = max(8, C // 8 * 8)
            pre = rng.choice(["layer", "rms", "none"])
            post = rng.choice(["layer", "rms", "none"])
            c = dict(op=op, train=train, B=_log_uniform(rng, 1, 128), T=_log_uniform(rng, 1, 16384), C=C,
                     f32=rng.random() < 0.4, pre=pre, post=post, affine=rng.random() < 0.8, gate=rng.random() < 0.5,
                     scale=rng.random() < 0.5, p=rng.choice([0.0, 0.0, 0.1, 0.5]))
            if c["B"] * c["T"] * C <= (1 << 24 if train or c["p"] else 3 << 24):
                return c
    while True:
        c = dict(op=op, train=train, T=_log_uniform(rng, 1, 262144), C=8 * _log_uniform(rng, 4, 128),
                 F=8 * _log_uniform(rng, 4, 512), act=rng.choice(["silu", "gelu"]), bias=rng.random() < 0.6)
        if c["T"] * c["C"] * c["F"] <= 12 << 30 and c["T"] * c["F"] <= 1 << 27:
            return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def _log_buckets(M):
    """Bucket of every displacement (row, column): per axis, distances up to 3 apart each, then by octaves, signed."""
    def axis(d):
        a = abs(d)
        b = a if a < 4 else 4 + int(math.floor(math.log2(a / 4.0)))
        return b if d >= 0 else -b

    one = [axis(d) for d in range(-(M - 1), M)]
    lo = min(one)
    n = max(one) - lo + 1
    ids = [[(a - lo) * n + (b - lo) for b in one] for a in one]
    return ids, n * n


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    if case["op"] == "relbias":
        shape = (case["B"], case["H"], case["W"], case["heads"], D)
        for name in ("q", "k", "v"):
            st[name] = _randn(g, shape, BF16)
        M = case["M"]
        n, st["buckets"] = (2 * M - 1) ** 2, None
        if case["log"]:
            ids, n = _log_buckets(M)
            st["buckets"] = torch.tensor(ids, dtype=torch.int32, device="cuda")
        st["table"] = _randn(g, (case["heads"], n), BF16, 0.7)
        if case["train"]:
            st["dout"] = _randn(g, shape, BF16)
    elif case["op"] == "resnorm":
        B, T, C = case["B"], case["T"], case["C"]
        stream = F32 if case["f32"] else BF16
        st["x"] = _randn(g, (B, T, C), stream, 1.5)
        st["f"] = _randn(g, (B, T, C), BF16)
        st["gate"] = st["scale"] = st["rng"] = None
        if case["gate"]:  # stochastic depth at rate 0.2: one in five samples drops its branch
            keep = torch.rand((B,), generator=g, device="cuda") >= 0.2
            st["gate"] = (keep.float() * 1.25).to(stream)
        if case["scale"]:
            st["scale"] = _randn(g, (C,), stream, 0.1, 0.5)
        for k in ("pre", "post"):
            st[k + "_weight"] = st[k + "_bias"] = None
            if case["affine"] and case[k] != "none":
                st[k + "_weight"] = _randn(g, (C,), stream, 0.1, 1.0)
                if case[k] == "layer":
                    st[k + "_bias"] = _randn(g, (C,), stream, 0.1)
        if case["p"] > 0:
            st["rng"] = torch.randint(0, 1 << 62, (2,), generator=g, device="cuda", dtype=torch.int64)
        if case["train"]:
            st["dr"] = _randn(g, (B, T, C), stream)
            st["dn"] = _randn(g, (B, T, C), BF16) if case["pre"] != "none" else None
    else:
        T, C, F = case["T"], case["C"], case["F"]
        st["x"] = _randn(g, (T, C), BF16)
        st["w_gate"] = _randn(g, (F, C), BF16, C ** -0.5)
        st["w_up"] = _randn(g, (F, C), BF16, C ** -0.5)
        st["w_down"] = _randn(g, (C, F), BF16, F ** -0.5)
        for name, n in (("b_gate", F), ("b_up", F), ("b_down", C)):
            st[name] = _randn(g, (n,), BF16, 0.1) if case["bias"] else None
        if case["train"]:
            st["dy"] = _randn(g, (T, C), BF16)
    return st


# ------------------------------------------------------------------ the passes
def run(st):
    case = st["case"]
    if case["op"] == "relbias":
        return _run_relbias(st, case)
    if case["op"] == "resnorm":
        return _run_resnorm(st, case)
    return _run_mlp(st, case)


def _run_relbias(st, case):
    if own:
        from vision_transformer_windowed_b200 import ops
        a = (st["q"], st["k"], st["v"])
        M, s, tab, bk = case["M"], case["s"], st["table"], st["buckets"]
        if not case["train"]:
            return ops.winattn_relbias_fwd(*a, tab, M, s, buckets=bk, need_lse=False)[0]
        o, lse = ops.winattn_relbias_fwd(*a, tab, M, s, buckets=bk)
        dq, dk, dv, dtable = ops.winattn_relbias_bwd(*a, o, st["dout"], lse, tab, M, s, buckets=bk)
        return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv, dtable=dtable)
    return _plain_relbias(st, case)


def _windows(t, M, s):
    """[B, H, W, heads, D] -> [B, windows, heads, M*M, D], padded, rolled, in 32 bits."""
    B, H, W, h, d = t.shape
    Hp, Wp = -(-H // M) * M, -(-W // M) * M
    x = torch.zeros((B, Hp, Wp, h, d), device=t.device, dtype=F32)
    x[:, :H, :W] = t.float()
    if s:
        x = torch.roll(x, (-s, -s), (1, 2))
    x = x.reshape(B, Hp // M, M, Wp // M, M, h, d)
    return x.permute(0, 1, 3, 5, 2, 4, 6).reshape(B, (Hp // M) * (Wp // M), h, M * M, d)


def _grid(x, like, M, s):
    """The inverse of _windows, cut back to the real grid; the last axis may have any size."""
    B, H, W, h = like.shape[:4]
    Hp, Wp = -(-H // M) * M, -(-W // M) * M
    d = x.shape[-1]
    x = x.reshape(B, Hp // M, Wp // M, h, M, M, d).permute(0, 1, 4, 2, 5, 3, 6).reshape(B, Hp, Wp, h, d)
    if s:
        x = torch.roll(x, (s, s), (1, 2))
    return x[:, :H, :W].contiguous()


def _region_labels(H, W, M, s, device):
    """Shift-region label of every token of every window: [windows, M*M]."""
    Hp, Wp = -(-H // M) * M, -(-W // M) * M

    def side(n):
        i = torch.arange(n, device=device)
        return (i >= n - M).long() + (i >= n - s).long()

    lab = 3 * side(Hp)[:, None] + side(Wp)[None, :]
    return lab.reshape(Hp // M, M, Wp // M, M).permute(0, 2, 1, 3).reshape(-1, M * M)


def _displacements(M, device):
    """Index of the displacement (query minus key) of every pair of window positions: [M*M, M*M]."""
    i = torch.arange(M * M, device=device) // M
    j = torch.arange(M * M, device=device) % M
    return (i[:, None] - i[None, :] + M - 1) * (2 * M - 1) + (j[:, None] - j[None, :] + M - 1)


def _plain_relbias(st, case):
    M, s = case["M"], case["s"]
    q, k, v = (_windows(st[n], M, s) for n in ("q", "k", "v"))
    scale = 1.0 / math.sqrt(D)
    idx = _displacements(M, q.device)
    if st["buckets"] is not None:
        idx = st["buckets"].reshape(-1).long()[idx]
    S = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    S += st["table"].float()[:, idx]
    if s:
        lab = _region_labels(case["H"], case["W"], M, s, q.device)
        S.masked_fill_((lab[:, :, None] != lab[:, None, :])[None, :, None], -math.inf)
    m = S.amax(-1, keepdim=True)
    P = torch.exp(S.sub_(m))
    del S
    total = P.sum(-1, keepdim=True)
    P /= total
    o = torch.matmul(P, v)
    out = _grid(o, st["q"], M, s).to(BF16)
    if not case["train"]:
        return out
    lse = _grid(m + torch.log(total), st["q"], M, s)[..., 0].contiguous()
    do = _windows(st["dout"], M, s)
    dv = torch.matmul(P.transpose(-1, -2), do)
    dS = torch.matmul(do, v.transpose(-1, -2))
    dS -= (do * o).sum(-1, keepdim=True)
    dS *= P
    del P
    dq = torch.matmul(dS, k).mul_(scale)
    dk = torch.matmul(dS.transpose(-1, -2), q).mul_(scale)
    pairs = dS.sum((0, 1)).double().reshape(case["heads"], -1)
    dtable = torch.zeros(st["table"].shape, device=q.device, dtype=torch.float64)
    dtable.index_add_(1, idx.reshape(-1), pairs)
    dq, dk, dv = (_grid(t, st["q"], M, s).to(BF16) for t in (dq, dk, dv))
    return dict(o=out, lse=lse, dq=dq, dk=dk, dv=dv, dtable=dtable.to(BF16))


_EPS = 1e-5


def _run_resnorm(st, case):
    pre, post = (None if case[k] == "none" else case[k] for k in ("pre", "post"))
    if own:
        from vision_transformer_windowed_b200 import ops
        kw = dict(gate=st["gate"], scale=st["scale"], pre=pre, post=post, post_weight=st["post_weight"],
                  post_bias=st["post_bias"], pre_weight=st["pre_weight"], eps=_EPS, p=case["p"], rng=st["rng"])
        r, n = ops.residual_norm_fwd(st["x"], st["f"], pre_bias=st["pre_bias"], **kw)
        if not case["train"]:
            return dict(r=r, n=n)
        g = ops.residual_norm_bwd(st["dr"], st["dn"], r, st["f"], pre_bias=st["pre_bias"], **kw)
        return dict(r=r, n=n, **g._asdict())
    return _plain_resnorm(st, case, pre, post)


def _philox_keep(rng, total, p):
    """Keep mask of `total` elements: Philox4x32-10, counter (element // 4, offset), key seed, one word an element."""
    low = 0xFFFFFFFF
    n4 = (total + 3) // 4
    i = torch.arange(n4, device=rng.device, dtype=torch.int64)
    c = [i & low, i >> 32, (rng[1] & low).expand(n4), ((rng[1] >> 32) & low).expand(n4)]
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # wraps modulo 2^64; the low and high halves are exact
        c = [((b >> 32) & low) ^ c[1] ^ k0, b & low, ((a >> 32) & low) ^ c[3] ^ k1, a & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack(c, 1).reshape(-1)[:total]
    return words >= int(p * 4294967296.0)


def _plain_norm(x, kind, w, b):
    """(normalised row, its inverse deviation, output with weight and bias)."""
    c = x - x.mean(-1, keepdim=True) if kind == "layer" else x
    inv = torch.rsqrt((c * c).mean(-1, keepdim=True) + _EPS)
    hat = c * inv
    y = hat if w is None else hat * w.float()
    return hat, inv, y if b is None else y + b.float()


def _plain_norm_grad(dy, hat, inv, kind, w, b):
    """(gradient of the row, of the weight, of the bias)."""
    dw = None if w is None else (dy * hat).sum((0, 1)).to(w.dtype)
    db = None if b is None else dy.sum((0, 1)).to(b.dtype)
    t = dy if w is None else dy * w.float()
    dx = t - hat * (t * hat).mean(-1, keepdim=True)
    if kind == "layer":
        dx = dx - t.mean(-1, keepdim=True)
    return dx * inv, dw, db


def _plain_resnorm(st, case, pre, post):
    x, f = st["x"].float(), st["f"].float()
    y = f
    if post:
        hat_f, inv_f, y = _plain_norm(f, post, st["post_weight"], st["post_bias"])
    keep = _philox_keep(st["rng"], y.numel(), case["p"]).reshape(y.shape) if case["p"] > 0 else None
    if keep is not None:
        y = torch.where(keep, y * (1.0 / (1.0 - case["p"])), 0.0)
    u = y if st["scale"] is None else y * st["scale"].float()
    gate = None if st["gate"] is None else st["gate"].float()[:, None, None]
    r = x + (u if gate is None else torch.where(gate == 0, 0.0, gate * u))
    if pre:
        hat_r, inv_r, n = _plain_norm(r, pre, st["pre_weight"], st["pre_bias"])
    out = dict(r=r.to(st["x"].dtype), n=n.to(BF16) if pre else None)
    if not case["train"]:
        return out
    dr = st["dr"].float()
    dpre_w = dpre_b = dpost_w = dpost_b = dgate = dscale = None
    if pre:
        d, dpre_w, dpre_b = _plain_norm_grad(st["dn"].float(), hat_r, inv_r, pre, st["pre_weight"], st["pre_bias"])
        dr = dr + d
    du = dr
    if gate is not None:
        dgate = (dr * u).sum((1, 2)).to(st["gate"].dtype)
        du = torch.where(gate == 0, 0.0, gate * dr)
    dy = du
    if st["scale"] is not None:
        dscale = (du * y).sum((0, 1)).to(st["scale"].dtype)
        dy = du * st["scale"].float()
    if keep is not None:
        dy = torch.where(keep, dy * (1.0 / (1.0 - case["p"])), 0.0)
    if post:
        dy, dpost_w, dpost_b = _plain_norm_grad(dy, hat_f, inv_f, post, st["post_weight"], st["post_bias"])
    return dict(out, dx=dr.to(st["x"].dtype), df=dy.to(BF16), dgate=dgate, dscale=dscale, dpost_weight=dpost_w,
                dpost_bias=dpost_b, dpre_weight=dpre_w, dpre_bias=dpre_b)


_MLP = ("w_gate", "w_up", "w_down", "b_gate", "b_up", "b_down")


def _run_mlp(st, case):
    if own:
        from vision_transformer_windowed_b200 import ops
        y = ops.gated_mlp_fwd(st["x"], *(st[n] for n in _MLP), act=case["act"])
        if not case["train"]:
            return y
        g = ops.gated_mlp_bwd(st["dy"], st["x"], *(st[n] for n in _MLP), act=case["act"])
        return dict(y=y, **g._asdict())
    x = st["x"].float()
    wg, wu, wd = (st[n].float() for n in ("w_gate", "w_up", "w_down"))
    a, u = x @ wg.t(), x @ wu.t()
    if case["bias"]:
        a, u = a + st["b_gate"].float(), u + st["b_up"].float()
    if case["act"] == "silu":
        sg = 1.0 / (1.0 + torch.exp(-a))
        act, slope = a * sg, sg * (1.0 + a * (1.0 - sg))
    else:
        cdf = 0.5 * (1.0 + torch.erf(a * math.sqrt(0.5)))
        act, slope = a * cdf, cdf + a * torch.exp(-0.5 * a * a) * (1.0 / math.sqrt(2.0 * math.pi))
    h = act * u
    y = h @ wd.t()
    if case["bias"]:
        y = y + st["b_down"].float()
    if not case["train"]:
        return y.to(BF16)
    dy = st["dy"].float()
    dh = dy @ wd
    da, du = dh * u * slope, dh * act
    grads = dict(dx=da @ wg + du @ wu, dw_gate=da.t() @ x, dw_up=du.t() @ x, dw_down=dy.t() @ h)
    for n, t in (("db_gate", da), ("db_up", du), ("db_down", dy)):
        grads[n] = t.sum(0) if case["bias"] else None
    return {n: None if t is None else t.to(BF16) for n, t in dict(grads, y=y).items()}


# ------------------------------------------------------------------ the least work
def _pairs(case):
    """Pairs (query, key) that attend, over the padded grid of one image and head."""
    M, s = case["M"], case["s"]

    def axis(n):
        w = -(-n // M)
        return (w - 1) * M * M + ((M - s) ** 2 + s * s if s else M * M)

    # a pair attends when both its row and its column parts match, so the sums over the two axes multiply
    return axis(case["H"]) * axis(case["W"])


def work(case):
    if case["op"] == "relbias":
        rows = case["B"] * case["H"] * case["W"] * case["heads"]
        pairs = case["B"] * case["heads"] * _pairs(case)
        table = case["heads"] * (2 * case["M"] - 1) ** 2 * 2
        if not case["train"]:
            return dict(bytes=rows * 4 * 2 * D + table, flops=4 * D * pairs)
        # q, k, v, dout read; o, lse, dq, dk, dv written
        return dict(bytes=rows * (8 * 2 * D + 4) + 2 * table, flops=14 * D * pairs)
    if case["op"] == "resnorm":
        n = case["B"] * case["T"] * case["C"]
        xs = 4 if case["f32"] else 2
        pre = case["pre"] != "none"
        fwd = xs + 2 + xs + (2 if pre else 0)
        bwd = xs + (2 if pre else 0) + xs + 2
        return dict(bytes=n * (fwd + (bwd if case["train"] else 0)), flops=n * (40 if case["train"] else 12))
    T, C, F = case["T"], case["C"], case["F"]
    if not case["train"]:
        return dict(bytes=2 * (2 * T * C + 3 * C * F), flops=6 * T * C * F)
    return dict(bytes=2 * (4 * T * C + 6 * C * F), flops=18 * T * C * F)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "relbias":
        return _exact_relbias(st, case)
    if case["op"] == "resnorm":
        return _exact_resnorm(st, case)
    return _exact_mlp(st, case)


def _exact_relbias(st, case):
    """Window by window from token coordinates, a slice of the windows at a time, gradients by differentiation."""
    B, H, W, h, M, s = (case[k] for k in ("B", "H", "W", "heads", "M", "s"))
    dev, N = st["q"].device, M * M
    nh, nw = -(-H // M), -(-W // M)
    a = torch.arange(M, device=dev)
    i, j = a.repeat_interleave(M), a.repeat(M)
    delta = (i[:, None] - i[None] + M - 1) * (2 * M - 1) + j[:, None] - j[None] + M - 1
    ids = delta if st["buckets"] is None else st["buckets"].flatten()[delta].long()
    flat = {n: st[n].reshape(B * H * W, h, D) for n in ("q", "k", "v") + (("dout",) if case["train"] else ())}
    table = st["table"].double().requires_grad_(case["train"])
    names = ("o", "dq", "dk", "dv") if case["train"] else ("o",)
    res = {n: torch.empty((B * H * W, h, D), device=dev, dtype=torch.float64) for n in names}
    lse = torch.empty((B * H * W, h), device=dev, dtype=torch.float64)
    dtable = torch.zeros_like(table)
    step = max(1, (1 << 27) // (h * N * N))
    for w0 in range(0, B * nh * nw, step):
        w = torch.arange(w0, min(w0 + step, B * nh * nw), device=dev)
        b, wr, wc = w // (nh * nw), w // nw % nh, w % nw
        rr, cc = wr[:, None] * M + i, wc[:, None] * M + j
        row, col = (rr + s) % (nh * M), (cc + s) % (nw * M)
        real = (row < H) & (col < W)
        tok = ((b[:, None] * H + row) * W + col)[real]
        part = []
        for n in flat:
            t = torch.zeros((len(w), N, h, D), device=dev, dtype=torch.float64)
            t[real] = flat[n][tok].double()
            part.append(t.transpose(1, 2))
        q, k, v = (t.requires_grad_(case["train"]) for t in part[:3])
        z = torch.einsum("whtd,whud->whtu", q, k) / math.sqrt(D) + table[:, ids]
        if s:  # the tokens that wrapped around the grid's edge are strangers to the others
            up, left = row < s, col < s
            same = (up[:, :, None] == up[:, None, :]) & (left[:, :, None] == left[:, None, :])
            z = torch.where(same[:, None], z, torch.full((), -math.inf, device=dev, dtype=torch.float64))
        L = torch.logsumexp(z, -1, keepdim=True)
        o = torch.einsum("whtu,whud->whtd", torch.exp(z - L), v)
        got = [o]
        if case["train"]:
            *grads, dt = torch.autograd.grad(o, (q, k, v, table), part[3])
            got += grads
            dtable += dt
        for n, t in zip(names, got):
            res[n][tok] = t.detach().transpose(1, 2)[real]
        lse[tok] = L.detach()[..., 0].transpose(1, 2)[real]
        del part, q, k, v, z, L, o, got
    grid = {n: t.reshape(B, H, W, h, D) for n, t in res.items()}
    if not case["train"]:
        return grid["o"]
    return dict(grid, lse=lse.reshape(B, H, W, h), dtable=dtable)


def _exact_keep(rng, shape, p):
    """The same generator in unsigned arithmetic on the host."""
    seed, off = (int(t) & (2 ** 64 - 1) for t in rng.tolist())
    total = int(np.prod(shape))
    n4 = -(-total // 4)
    m32 = np.uint64(0xFFFFFFFF)
    i = np.arange(n4, dtype=np.uint64)
    x0, x1 = i & m32, i >> np.uint64(32)
    x2, x3 = np.full(n4, off & 0xFFFFFFFF, np.uint64), np.full(n4, off >> 32, np.uint64)
    key0, key1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        p0, p1 = x0 * np.uint64(0xD2511F53), x2 * np.uint64(0xCD9E8D57)
        x0, x1, x2, x3 = ((p1 >> np.uint64(32)) ^ x1 ^ np.uint64(key0), p1 & m32,
                          (p0 >> np.uint64(32)) ^ x3 ^ np.uint64(key1), p0 & m32)
        key0, key1 = (key0 + 0x9E3779B9) % 2 ** 32, (key1 + 0xBB67AE85) % 2 ** 32
    words = np.empty((n4, 4), np.uint64)
    for n, x in enumerate((x0, x1, x2, x3)):
        words[:, n] = x
    keep = words.reshape(-1)[:total] >= np.uint64(int(p * 2.0 ** 32))
    return torch.from_numpy(keep.reshape(shape)).to(rng.device)


def _exact_norm(x, kind, w, b):
    if kind == "layer":
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        x = (x - mean) / torch.sqrt(var + _EPS)
    else:
        x = x / torch.sqrt(torch.mean(x.square(), -1, keepdim=True) + _EPS)
    x = x if w is None else x * w
    return x if b is None else x + b


def _exact_resnorm(st, case):
    names = ["x", "f"] + [n for n in ("gate", "scale", "post_weight", "post_bias", "pre_weight", "pre_bias")
                          if st[n] is not None]
    t = {n: st[n].double().requires_grad_(case["train"]) for n in names}
    y = t["f"]
    if case["post"] != "none":
        y = _exact_norm(y, case["post"], t.get("post_weight"), t.get("post_bias"))
    if case["p"] > 0:
        y = y * _exact_keep(st["rng"], y.shape, case["p"]) / (1.0 - case["p"])
    if "scale" in t:
        y = y * t["scale"]
    if "gate" in t:
        y = y * t["gate"].reshape(-1, 1, 1)
    r = t["x"] + y
    n = _exact_norm(r, case["pre"], t.get("pre_weight"), t.get("pre_bias")) if case["pre"] != "none" else None
    out = dict(r=r.detach(), n=None if n is None else n.detach())
    if not case["train"]:
        return out
    outs, ups = [r], [st["dr"].double()]
    if n is not None:
        outs, ups = outs + [n], ups + [st["dn"].double()]
    got = dict(zip(names, torch.autograd.grad(outs, [t[k] for k in names], ups)))
    every = ("x", "f", "gate", "scale", "post_weight", "post_bias", "pre_weight", "pre_bias")
    return dict(out, **{"d" + k: got.get(k) for k in every})


def _exact_mlp(st, case):
    T, C, F = case["T"], case["C"], case["F"]
    names = [n for n in _MLP if st[n] is not None]
    w = {n: st[n].double().requires_grad_(case["train"]) for n in names}
    total = {n: torch.zeros_like(w[n]) for n in names}
    y, dx = [], []
    step = max(1, (1 << 26) // F)
    for t0 in range(0, T, step):
        x = st["x"][t0:t0 + step].double().requires_grad_(case["train"])
        a = torch.nn.functional.linear(x, w["w_gate"], w.get("b_gate"))
        u = torch.nn.functional.linear(x, w["w_up"], w.get("b_up"))
        act = a * torch.sigmoid(a) if case["act"] == "silu" else a * torch.special.ndtr(a)
        z = torch.nn.functional.linear(act * u, w["w_down"], w.get("b_down"))
        y.append(z.detach())
        if case["train"]:
            gx, *gw = torch.autograd.grad(z, [x] + [w[n] for n in names], st["dy"][t0:t0 + step].double())
            dx.append(gx)
            for n, g in zip(names, gw):
                total[n] += g
        del x, a, u, act, z
    y = torch.cat(y)
    if not case["train"]:
        return y
    return dict(y=y, dx=torch.cat(dx), **{"d" + n: total.get(n) for n in _MLP})
