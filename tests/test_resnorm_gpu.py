"""GPU parity of the residual step against its fp64 oracle: 2^-16 of each result's terms for the fp32 arithmetic, and
half a step of the result's type (2^-8 for bf16, 2^-24 for fp32).  The backward is compared at the r it is given."""
import pytest
import torch

from oracle import resnorm
from vision_transformer_windowed_b200 import ops

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
PARAMS = ("gate", "scale", "post_weight", "post_bias", "pre_weight", "pre_bias")


def draw(B, T, C, stream, pre, post, affine=True, gate=True, scale=True, mean=0.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda shape, dt, std=1.0, mu=0.0: (torch.randn(shape, generator=g) * std + mu).to(dt)  # noqa: E731
    t = dict(x=n((B, T, C), stream, 1.5, mean), f=n((B, T, C), BF16, 1.0, mean))
    t["gate"] = ((torch.rand(B, generator=g) > 0.3).float() * 1.25).to(stream) if gate else None
    t["scale"] = n((C,), stream, 0.2, 0.5) if scale else None
    for which, kind in (("pre", pre), ("post", post)):
        t[which + "_weight"] = n((C,), stream, 0.2, 1.0) if affine and kind else None
        t[which + "_bias"] = n((C,), stream, 0.2) if affine and kind else None
    return t, n((B, T, C), stream), n((B, T, C), BF16) if pre else None


def cuda(t):
    return {k: None if v is None else v.cuda() for k, v in t.items()}


def close(name, got, want, terms, kind=None):
    assert (got is None) == (want is None), name
    if got is None:
        return
    kind = kind or got.dtype
    a = got.double().cpu()
    assert torch.isfinite(a).all(), name
    bound = 2.0 ** -16 * terms + torch.finfo(kind).eps / 2 * want.abs() + 1e-30
    over = (a - want).abs() - bound
    assert over.max() <= 0, f"{name}: {float(over.max()):.3g} over its bound"


def check(B, T, C, stream, pre, post, p=0.0, use_dr=True, use_dn=True, **kw):
    t, dr, dn = draw(B, T, C, stream, pre, post, **kw)
    rng = torch.tensor([0x123456789ABCDEF, (1 << 40) + 7]) if p else None
    opt = dict(pre=pre, post=post, p=p)
    d = cuda(t)
    r, n = ops.residual_norm_fwd(**d, **opt, rng=None if rng is None else rng.cuda())
    want = resnorm.step(**t, **opt, rng=rng)
    close("r", r, want["r"], want["terms"]["r"])
    close("n", n, want["n"], want["terms"].get("n"))
    dr, dn = dr if use_dr else None, dn if use_dn else None
    # the oracle at exactly this r
    branch = want["r"] - t["x"].double()
    at = resnorm.step(**{**t, "x": r.cpu().double() - branch}, **opt, rng=rng, dr=dr, dn=dn)
    g = ops.residual_norm_bwd(None if dr is None else dr.cuda(), None if dn is None else dn.cuda(), r,
                              *(d[k] for k in ("f",)), **{k: d[k] for k in PARAMS}, **opt,
                              rng=None if rng is None else rng.cuda())
    for name, got in g._asdict().items():
        close(name, got, at[name], at["terms"].get(name))
    torch.cuda.synchronize()


@pytest.mark.parametrize("stream", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("C", [1, 8, 24, 33, 64, 96, 97, 128, 192, 256, 384, 513, 520, 768, 1001, 1024, 1536, 2056, 4104,
                               5003, 8192])
def test_every_row_shape(C, stream):
    rows = 71 if C <= 1024 else 5
    check(2, rows, C, stream, "layer", None)
    check(3, (rows + 1) // 2, C, stream, "rms", "layer", gate=C % 2 == 0)


@pytest.mark.parametrize("stream", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("pre", [None, "layer", "rms"])
@pytest.mark.parametrize("post", [None, "layer", "rms"])
def test_every_kind(pre, post, stream):
    check(5, 13, 96, stream, pre, post)
    check(5, 13, 40, stream, pre, post, affine=False, gate=False, scale=False)
    check(2, 7, 50, stream, pre, post, scale=False, p=0.1)


@pytest.mark.parametrize("C,p", [(96, 0.1), (8, 0.5), (37, 0.9), (192, 0.999)])
def test_dropout(C, p):
    check(3, 21, C, BF16, "layer", None, p=p)
    check(1, 21, C, F32, None, "rms", p=p, gate=False)


@pytest.mark.parametrize("which", ["dr", "dn"])
def test_one_upstream_gradient(which):
    check(2, 9, 64, BF16, "layer", None, use_dr=which == "dr", use_dn=which == "dn")


def test_large_mean_and_one_row():
    check(1, 1, 96, F32, "layer", "layer", mean=1000.0)
    check(1, 1, 1000, BF16, "layer", None, mean=100.0)


def test_many_rows_sum_in_order_and_repeat():
    """More rows than the backward has blocks, twice: the same bits."""
    t, dr, dn = draw(64, 700, 96, BF16, "layer", "layer")
    d = cuda(t)
    r, _ = ops.residual_norm_fwd(**d, pre="layer", post="layer")
    kw = {k: d[k] for k in PARAMS}
    a, b = (ops.residual_norm_bwd(dr.cuda(), dn.cuda(), r, d["f"], **kw, pre="layer", post="layer") for _ in range(2))
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    want = resnorm.step(**{**t, "x": r.cpu().double() - (resnorm.step(**t, pre="layer", post="layer")["r"] - t["x"].double())},
                        pre="layer", post="layer", dr=dr, dn=dn)
    for name, got in a._asdict().items():
        close(name, got, want[name], want["terms"][name])


def test_dropped_sample_with_values_that_are_not_finite():
    t, dr, dn = draw(3, 5, 96, BF16, "layer", "layer")
    t["gate"] = torch.tensor([1.25, 0.0, 1.25]).to(BF16)
    t["f"][1] = float("nan")
    d = cuda(t)
    r, n = ops.residual_norm_fwd(**d, pre="layer", post="layer")
    assert torch.equal(r[1].cpu(), t["x"][1]) and torch.isfinite(n).all()
    g = ops.residual_norm_bwd(dr.cuda(), dn.cuda(), r, d["f"], **{k: d[k] for k in PARAMS}, pre="layer", post="layer")
    assert (g.df[1] == 0).all()
    assert all(torch.isfinite(x).all() for x in (g.dx, g.df, g.dscale, g.dpost_weight, g.dpost_bias, g.dpre_weight))
    assert torch.isfinite(g.dgate[0]) and torch.isfinite(g.dgate[2])


def test_in_place_unaligned_and_neighbours_left_alone():
    t, dr, dn = draw(2, 9, 96, BF16, "layer", None)
    d = cuda(t)
    r, n = ops.residual_norm_fwd(**d, pre="layer", p=0.0)
    size = r.numel()
    buf = torch.full((size + 16,), 3.0, device="cuda", dtype=BF16)
    view = buf[1:1 + size].view(r.shape)  # two-byte aligned: the narrow accesses
    view.copy_(d["x"])
    f = d["f"].clone()
    r2, n2 = ops.residual_norm_fwd(**{**d, "x": view, "f": f}, pre="layer", r=view, n=f)
    assert r2.data_ptr() == view.data_ptr()
    assert (r2.float() - r.float()).abs().max() <= 2.0 ** -7 * r.float().abs().max()
    assert (n2.float() - n.float()).abs().max() <= 2.0 ** -6 * n.float().abs().max()
    assert buf[0] == 3 and (buf[1 + size:] == 3).all()


def test_autograd_graph_and_generator_in_place():
    """The layer's step under autograd: the generator tensor may advance between forward and backward; a captured
    forward draws a new mask when the tensor changes."""
    t, dr, dn = draw(2, 6, 96, F32, "layer", None)
    d = cuda(t)
    rng = torch.tensor([3, 4], device="cuda")
    leaves = {k: v.clone().requires_grad_() for k, v in d.items() if v is not None}
    r, n = ops.residual_norm(**leaves, pre="layer", p=0.25, rng=rng)
    rng[1] += 1
    grads = torch.autograd.grad([r, n], list(leaves.values()), [dr.cuda(), dn.cuda()])
    want = resnorm.step(**t, pre="layer", p=0.25, rng=torch.tensor([3, 4]), dr=dr, dn=dn)
    for key, got in zip(leaves, grads):  # r is fp32: its rounding is inside the fp32 slack
        close("d" + key, got, want["d" + key], want["terms"]["d" + key])
    r, n = ops.residual_norm_fwd(**d, pre="layer", p=0.25, rng=rng)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.residual_norm_fwd(**d, pre="layer", p=0.25, rng=rng, r=r, n=n)
    rng.copy_(torch.tensor([8, 9]))
    g.replay()
    torch.cuda.synchronize()
    want = resnorm.step(**t, pre="layer", p=0.25, rng=torch.tensor([8, 9]))
    close("r", r, want["r"], want["terms"]["r"])
    only_x = torch.autograd.grad(ops.residual_norm(leaves["x"], d["f"], pre="rms")[0].sum(), leaves["x"])[0]
    assert (only_x == 1).all()


def test_empty_batch():
    t, dr, dn = draw(0, 5, 96, BF16, "layer", None)
    d = cuda(t)
    r, n = ops.residual_norm_fwd(**d, pre="layer")
    g = ops.residual_norm_bwd(dr.cuda(), dn.cuda(), r, d["f"], **{k: d[k] for k in PARAMS}, pre="layer")
    torch.cuda.synchronize()
    assert r.numel() == 0 and (g.dpre_weight == 0).all() and (g.dscale == 0).all() and g.dgate.numel() == 0


@pytest.mark.parametrize("C,rows", [(1, 3400), (7, 3400), (33, 1200), (100, 1300), (513, 250), (1001, 300), (4098, 120),
                                    (8178, 7), (8179, 7), (8190, 7)])
def test_rows_off_a_boundary_many_a_group(C, rows):
    """Channel counts that no chunk divides: every group of lanes walks several rows, the last group's is a part."""
    check(3, rows, C, F32, "layer", "rms", p=0.2)
    check(3, rows, C, BF16, "rms", None)


@pytest.mark.parametrize("C", [33, 1001])
def test_in_place_rows_off_a_boundary(C):
    t, dr, dn = draw(2, 37, C, BF16, "layer", None)
    d = cuda(t)
    r, n = ops.residual_norm_fwd(**d, pre="layer")
    x, f = d["x"].clone(), d["f"].clone()
    r2, n2 = ops.residual_norm_fwd(**{**d, "x": x, "f": f}, pre="layer", r=x, n=f)
    assert r2 is x and n2 is f and torch.equal(r2, r) and torch.equal(n2, n)


@pytest.mark.parametrize("stream", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("pre,post", [("layer", None), ("rms", "layer"), ("layer", "rms")])
@pytest.mark.parametrize("C,rows", [(33, 40), (36, 257), (97, 21), (1001, 3), (96, 5), (8, 70)])
def test_no_epsilon_and_groups_past_the_last_row(C, rows, pre, post, stream):
    """eps = 0 with a row count that leaves groups of lanes without a row: what those hold joins no sum."""
    t, dr, dn = draw(1, rows, C, stream, pre, post, gate=False)
    opt = dict(pre=pre, post=post, eps=0.0)
    d = cuda(t)
    r, n = ops.residual_norm_fwd(**d, **opt)
    want = resnorm.step(**t, **opt)
    close("r", r, want["r"], want["terms"]["r"])
    close("n", n, want["n"], want["terms"]["n"])
    at = resnorm.step(**{**t, "x": r.cpu().double() - (want["r"] - t["x"].double())}, **opt, dr=dr, dn=dn)
    g = ops.residual_norm_bwd(dr.cuda(), dn.cuda(), r, d["f"], **{k: d[k] for k in PARAMS}, **opt)
    for name, got in g._asdict().items():
        close(name, got, at[name], at["terms"].get(name))


@pytest.mark.parametrize("B,T", [(70001, 1), (70001, 2), (66000, 3)])
def test_more_samples_than_blocks_of_the_gate_sum(B, T):
    g = torch.Generator().manual_seed(1)
    f, dr = (torch.randn((B, T, 8), generator=g).to(BF16) for _ in "fd")
    gate = torch.randn(B, generator=g).to(BF16)
    got = ops.residual_norm_bwd(dr.cuda(), None, dr.cuda(), f.cuda(), gate=gate.cuda(), pre=None)
    terms = f.double() * dr.double()
    close("dgate", got.dgate, terms.sum((1, 2)), terms.abs().sum((1, 2)))
