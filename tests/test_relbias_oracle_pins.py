"""Pins of the relative-position-bias oracle: against the low-rank-bias oracle with U = I and W the bias transposed,
autograd of a tensor restatement, and differences."""
import numpy as np
import pytest
import torch

import oracle
from oracle import relbias
from vision_transformer_windowed_b200.inputs import make_inputs

CASES = [(1, 8, 8, 2, 4, 0), (2, 16, 16, 2, 8, 4), (1, 10, 7, 2, 4, 0), (1, 13, 20, 1, 8, 4)]


def draw(B, H, W, heads, M, n=None, seed=3):
    inp = make_inputs(B, H, W, heads, 32)
    g = torch.Generator().manual_seed(seed)
    n = (2 * M - 1) ** 2 if n is None else n
    inp["table"] = (torch.randn((heads, n), generator=g) * 0.7).to(torch.bfloat16)
    return inp


@pytest.mark.parametrize("cfg", CASES)
def test_equals_low_rank_oracle_with_the_whole_bias_as_factors(cfg):
    B, H, W, heads, M, s = cfg
    inp = draw(B, H, W, heads, M)
    got, _ = relbias.full(inp["q"], inp["k"], inp["v"], inp["table"], M, s, dout=inp["dout"])
    b = relbias.bias_matrix(inp["table"], M)
    u = torch.eye(M * M, dtype=torch.float64).expand(heads, -1, -1).contiguous()
    ref = oracle.full(inp["q"], inp["k"], inp["v"], torch.zeros_like(inp["theta"]), M, s, dout=inp["dout"],
                      bias=(u, b.transpose(1, 2).contiguous()))
    for key in ("o", "lse", "dq", "dk", "dv"):
        want = np.asarray(ref[key], dtype=np.float64)
        assert np.abs(got[key].numpy() - want).max() <= 1e-6 * max(1.0, np.abs(want).max()), key
    # du with U = I is sum_u dS_tu W_u; through W = I instead dS itself would show: the table
    # gradient is checked against autograd and differences below


def restatement(q, k, v, table, M, s, idx):
    B, H, W, h, d = q.shape
    Hp, Wp = -(-H // M) * M, -(-W // M) * M

    def win(t):
        x = torch.nn.functional.pad(t, (0, 0, 0, 0, 0, Wp - W, 0, Hp - H)).roll((-s, -s), (1, 2))
        return x.reshape(B, Hp // M, M, Wp // M, M, h, d).permute(0, 1, 3, 5, 2, 4, 6).reshape(B, -1, h, M * M, d)

    S = win(q) @ win(k).transpose(-1, -2) / d ** 0.5 + table[:, idx]
    if s:
        lab = torch.zeros((Hp, Wp), dtype=torch.long)
        n = 0
        for a in (slice(0, -M), slice(-M, -s), slice(-s, None)):
            for b in (slice(0, -M), slice(-M, -s), slice(-s, None)):
                lab[a, b] = n
                n += 1
        lab = lab.reshape(Hp // M, M, Wp // M, M).permute(0, 2, 1, 3).reshape(-1, M * M)
        S = S.masked_fill((lab[:, :, None] != lab[:, None])[None, :, None], float("-inf"))
    o = torch.softmax(S, -1) @ win(v)
    o = o.reshape(B, Hp // M, Wp // M, h, M, M, d).permute(0, 1, 4, 2, 5, 3, 6).reshape(B, Hp, Wp, h, d)
    return o.roll((s, s), (1, 2))[:, :H, :W]


@pytest.mark.parametrize("log", [False, True])
@pytest.mark.parametrize("cfg", CASES)
def test_equals_autograd_of_a_restatement(cfg, log):
    B, H, W, heads, M, s = cfg
    buckets, n = (None, None)
    if log:
        from vision_transformer_windowed_b200 import ops
        buckets, n = ops.log_distance_buckets(M, exact=2, device="cpu")
    inp = draw(B, H, W, heads, M, n)
    got, err = relbias.full(inp["q"], inp["k"], inp["v"], inp["table"], M, s, buckets=buckets, dout=inp["dout"])
    leaves = [inp[n].double().requires_grad_() for n in ("q", "k", "v", "table")]
    idx = relbias.displacement_index(M) if buckets is None else buckets.reshape(-1).long()[relbias.displacement_index(M)]
    o = restatement(*leaves, M, s, idx)
    grads = torch.autograd.grad(o, leaves, inp["dout"].double())
    for key, t in zip(("o", "dq", "dk", "dv", "dtable"), (o, *grads)):
        assert (got[key] - t).abs().max() <= 1e-12 * max(1.0, t.abs().max()), key
        assert err[key].shape == got[key].shape and (err[key] >= 0).all()


def test_table_gradient_by_differences():
    B, H, W, heads, M, s = 1, 6, 7, 2, 4, 0
    inp = draw(B, H, W, heads, M)
    got, _ = relbias.full(inp["q"], inp["k"], inp["v"], inp["table"], M, s, dout=inp["dout"])
    t = inp["table"].double()
    for h, b in ((0, 24), (1, 10), (1, 48), (0, 0)):
        step = 1e-5
        f = []
        for sign in (1, -1):
            u = t.clone()
            u[h, b] += sign * step
            o, _ = relbias.full(inp["q"], inp["k"], inp["v"], u, M, s)
            f.append((o["o"] * inp["dout"].double()).sum())
        assert abs((f[0] - f[1]) / (2 * step) - got["dtable"][h, b]) <= 1e-6 * max(1.0, abs(got["dtable"][h, b]))


def test_row_without_a_key_and_bucket_outside_the_table():
    B, H, W, heads, M, s = 1, 4, 4, 1, 4, 0
    inp = draw(B, H, W, heads, M)
    inp["table"][:] = float("-inf")
    got, _ = relbias.full(inp["q"], inp["k"], inp["v"], inp["table"], M, s, dout=inp["dout"])
    assert (got["o"] == 0).all() and (got["lse"] == float("-inf")).all()
    assert all((got[k] == 0).all() for k in ("dq", "dk", "dv", "dtable"))
    outside = torch.full((7, 7), 49, dtype=torch.int32)
    a, _ = relbias.full(inp["q"], inp["k"], inp["v"], inp["table"], M, s, buckets=outside)
    b, _ = relbias.full(inp["q"], inp["k"], inp["v"], torch.zeros_like(inp["table"]), M, s)
    assert torch.equal(a["o"], b["o"])
