"""Oracle of the attention with a learned relative position bias by buckets, fp64,
one window and head at a time from token coordinates:

  S_tu = q_t.k_u / sqrt(d) + table[h][bucket(i_t - i_u, j_t - j_u)]   (shift-masked pairs: -inf)
  P = softmax(S), O = P V, lse = log sum exp S
  dV = P^T dO, dP = dO V^T, dS = P o (dP - rowsum(dO o O)), dQ = dS K / sqrt(d),
  dK = dS^T Q / sqrt(d), dtable[h][b] = sum of dS over the windows and the pairs of bucket b

A pair whose bucket lies outside the table has no bias; a query without a key has
O = 0, lse = -inf and no gradient.

Beside each result stands a bound on the error of an implementation that rounds as
the kernels do (bf16 operands of the products, bf16 outputs, the gradient's row
term from the rounded O, everything else in fp32), from the definition alone:
  half a step of bf16 is 2^-8 of the value;
  o:  2^-8 (sum P |v| + |o|)             the rounding of P, and of o
  D:  sum |dO| err(o) =: err(D)          the row term dO . O from the rounded o
  dS: P err(D) + 2^-8 |dS|               and its own rounding as an operand
  dq: (sum err(dS) |k|) / sqrt(d) + 2^-8 |dq|, dk likewise, dv: 2^-8 (sum P |dO| + |dv|)
  dtable: sum err(dS) + 2^-8 |dtable|
with EPS_P = 2^-14 of P beside them for the fp32 scores and the exponential (scores
up to about 100: 100 * 2^-23 in the argument, a few times)."""
from __future__ import annotations

import math

import torch

HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2
EPS_P = 2.0 ** -14


def displacement_index(M: int) -> torch.Tensor:
    """[M*M, M*M]: displacement index of (query position, key position)."""
    i = torch.arange(M * M) // M
    j = torch.arange(M * M) % M
    return (i[:, None] - i[None] + M - 1) * (2 * M - 1) + j[:, None] - j[None] + M - 1


def bias_matrix(table: torch.Tensor, M: int, buckets=None) -> torch.Tensor:
    """[heads, M*M, M*M] fp64 bias of every pair of window positions."""
    idx = displacement_index(M)
    if buckets is not None:
        idx = buckets.reshape(-1).long()[idx]
    inside = (idx >= 0) & (idx < table.shape[1])
    b = table.double()[:, idx.clamp(0, table.shape[1] - 1)]
    return torch.where(inside[None], b, torch.zeros((), dtype=torch.float64))


def full(q, k, v, table, M: int, s: int, buckets=None, dout=None):
    """(results, error bounds): dicts of fp64 CPU tensors shaped like the tensors they are for."""
    q, k, v, table = (t.detach().cpu() for t in (q, k, v, table))
    buckets = None if buckets is None else buckets.cpu()
    B, H, W, heads, d = q.shape
    nh, nw, N = -(-H // M), -(-W // M), M * M
    scale = 1.0 / math.sqrt(d)
    bias = bias_matrix(table, M, buckets)
    idx = displacement_index(M)
    if buckets is not None:
        idx = buckets.reshape(-1).long()[idx]
    n_buckets = table.shape[1]
    inside = (idx >= 0) & (idx < n_buckets)
    f64 = dict(dtype=torch.float64)
    names = ["o"] + (["dq", "dk", "dv"] if dout is not None else [])
    out = {n: torch.zeros((B, H, W, heads, d), **f64) for n in names}
    err = {n: torch.zeros((B, H, W, heads, d), **f64) for n in names}
    out["lse"] = torch.zeros((B, H, W, heads), **f64)
    if dout is not None:
        out["dtable"] = torch.zeros((heads, n_buckets), **f64)
        err["dtable"] = torch.zeros((heads, n_buckets), **f64)
    h8 = HALF_BF16

    def region(x, n):  # of a rolled coordinate
        return 0 if x < n - M else (1 if x < n - s else 2)

    for b in range(B):
        for wr in range(nh):
            for wc in range(nw):
                rr = [wr * M + i for i in range(M) for _ in range(M)]
                cc = [wc * M + j for _ in range(M) for j in range(M)]
                row = torch.tensor([(r + s) % (nh * M) for r in rr])
                col = torch.tensor([(c + s) % (nw * M) for c in cc])
                lab = torch.tensor([3 * region(r, nh * M) + region(c, nw * M) if s else 0 for r, c in zip(rr, cc)])
                real = (row < H) & (col < W)
                rows, cols = row[real], col[real]

                def rows_of(t, h):
                    x = torch.zeros((N, d), **f64)
                    x[real] = t[b, rows, cols, h].double()
                    return x

                apart = lab[:, None] != lab[None]
                for h in range(heads):
                    Q, K, V = rows_of(q, h), rows_of(k, h), rows_of(v, h)
                    S = Q @ K.t() * scale + bias[h]
                    S = torch.where(apart, torch.full((), -math.inf, **f64), S)
                    m = S.amax(1, keepdim=True)
                    none = m == -math.inf
                    e = torch.exp(S - torch.where(none, torch.zeros((), **f64), m))
                    total = e.sum(1, keepdim=True)
                    P = torch.where(none, torch.zeros((), **f64), e / total)
                    O = P @ V
                    PV = P @ V.abs()
                    out["o"][b, rows, cols, h] = O[real]
                    eo = (h8 + EPS_P) * PV + h8 * O.abs()
                    err["o"][b, rows, cols, h] = eo[real]
                    out["lse"][b, rows, cols, h] = (m + torch.log(total))[real, 0]
                    if dout is None:
                        continue
                    dO = rows_of(dout.detach().cpu(), h)
                    dP = dO @ V.t()
                    D = (dO * O).sum(1, keepdim=True)
                    dS = P * (dP - D)
                    dS = torch.where(P == 0, torch.zeros((), **f64), dS)
                    eD = (dO.abs() * eo).sum(1, keepdim=True)
                    eS = P * eD + (h8 + EPS_P) * dS.abs()
                    dQ, dK, dV = dS @ K * scale, dS.t() @ Q * scale, P.t() @ dO
                    for n, t, te in (("dq", dQ, eS @ K.abs() * scale), ("dk", dK, eS.t() @ Q.abs() * scale),
                                     ("dv", dV, (h8 + EPS_P) * (P.t() @ dO.abs()))):
                        out[n][b, rows, cols, h] = t[real]
                        err[n][b, rows, cols, h] = (te + h8 * t.abs())[real]
                    out["dtable"][h].index_add_(0, idx[inside], dS[inside])
                    err["dtable"][h].index_add_(0, idx[inside], eS[inside])
    if dout is not None:
        err["dtable"] += h8 * out["dtable"].abs()
    return out, err
