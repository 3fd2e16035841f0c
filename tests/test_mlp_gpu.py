"""GPU parity of the gated feed-forward block against its fp64 oracle, element by element within the oracle's bounds."""
import pytest
import torch

from oracle import mlp
from vision_transformer_windowed_b200 import _lib, ops

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _device_status_clean():
    _lib.fs_set_wait_limit_ns(4_000_000_000)
    _lib.fs_device_status()
    yield
    torch.cuda.synchronize()
    assert _lib.fs_device_status() == 0


def draw(T, C, F, bias=True, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda shape, std=1.0: (torch.randn(shape, generator=g) * std).to(BF16)  # noqa: E731
    t = dict(x=n((T, C), scale), w_gate=n((F, C), C ** -0.5), w_up=n((F, C), C ** -0.5), w_down=n((C, F), F ** -0.5),
             b_gate=None, b_up=None, b_down=None)
    if bias:
        t.update(b_gate=n(F, 0.3), b_up=n(F, 0.3), b_down=n(C, 0.3))
    return t, n((T, C))


def compare(got, want, bound):
    for name, a in got.items():
        assert (a is None) == (want[name] is None), name
        if a is None:
            continue
        a = a.double().cpu().reshape(want[name].shape)
        assert torch.isfinite(a).all(), name
        over = (a - want[name]).abs() - bound[name] * (1 + 1e-3) - 1e-12
        assert over.max() <= 0, f"{name}: {float(over.max()):.3g} over its bound"


def check(T, C, F, act="silu", **kw):
    t, dy = draw(T, C, F, **kw)
    d = {k: None if v is None else v.cuda() for k, v in t.items()}
    y = ops.gated_mlp_fwd(**d, act=act)
    g = ops.gated_mlp_bwd(dy.cuda(), **d, act=act)
    torch.cuda.synchronize()
    want, bound = mlp.full(**t, act=act, dy=dy)
    compare(dict(y=y, **g._asdict()), want, bound)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,C,F", [(1, 8, 8), (2, 96, 256), (127, 64, 168), (128, 64, 64), (129, 72, 136), (300, 96, 384),
                                   (1000, 200, 520), (257, 384, 1024), (64, 1024, 256), (513, 264, 40), (700, 16, 1032),
                                   (2500, 136, 72)])
def test_parity(T, C, F, act):
    check(T, C, F, act)


@pytest.mark.parametrize("T,C,F", [(129, 72, 136), (300, 96, 384)])
def test_parity_without_biases(T, C, F):
    check(T, C, F, bias=False)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("scale", [1e-3, 30.0])
def test_small_and_large_preactivations(act, scale):
    check(200, 64, 128, act, scale=scale)


def test_many_tokens_repeat_and_neighbours_left_alone():
    t, dy = draw(40000, 96, 128)
    d = {k: v.cuda() for k, v in t.items()}
    big = torch.full((40000 * 96 + 256,), 5.0, device="cuda", dtype=BF16)
    view = big[128:-128].view(40000, 96)
    a = ops.gated_mlp_fwd(**d, y=view)
    b = ops.gated_mlp_fwd(**d)
    assert torch.equal(a, b) and (big[:128] == 5).all() and (big[-128:] == 5).all()
    g, h = (ops.gated_mlp_bwd(dy.cuda(), **d) for _ in range(2))
    for p, q in zip(g, h):
        assert torch.equal(p, q)
    want, bound = mlp.full(**t, dy=dy)
    compare(dict(y=b, **g._asdict()), want, bound)


def test_infinite_row_stays_a_row():
    t, _ = draw(300, 64, 128)
    d = {k: v.cuda() for k, v in t.items()}
    clean = ops.gated_mlp_fwd(**d)
    d["x"][7] = float("inf")
    y = ops.gated_mlp_fwd(**d)
    keep = torch.arange(300, device="cuda") != 7
    assert torch.equal(y[keep], clean[keep])


def test_autograd_stream_and_graph():
    t, dy = draw(333, 96, 256)
    want, bound = mlp.full(**t, act="gelu", dy=dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        leaf = {k: v.cuda().requires_grad_() for k, v in t.items()}
        y = ops.gated_mlp(**leaf, act="gelu")
        grads = torch.autograd.grad(y, list(leaf.values()), dy.cuda())
    torch.cuda.current_stream().wait_stream(side)
    compare(dict(zip(("d" + k for k in leaf), grads), y=y.detach()), want, bound)
    d = {k: v.cuda() for k, v in t.items()}
    y = ops.gated_mlp_fwd(**d, act="gelu")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.gated_mlp_fwd(**d, act="gelu", y=y)
    new, _ = draw(333, 96, 256, seed=5)
    d["x"].copy_(new["x"])
    g.replay()
    torch.cuda.synchronize()
    want, bound = mlp.full(**{**t, "x": new["x"]}, act="gelu")
    compare(dict(y=y), want, bound)


def test_no_tokens():
    t, dy = draw(0, 64, 128)
    d = {k: v.cuda() for k, v in t.items()}
    y = ops.gated_mlp_fwd(**d)
    g = ops.gated_mlp_bwd(dy.cuda(), **d)
    torch.cuda.synchronize()
    assert y.numel() == 0 and (g.dw_gate == 0).all() and (g.dw_down == 0).all() and (g.db_down == 0).all()


def test_long_contractions_over_many_tokens():
    # tiles of 256 rows in every product that has them, the last rows' half empty
    t, dy = draw(19001, 264, 1544)
    d = {k: v.cuda() for k, v in t.items()}
    y = ops.gated_mlp_fwd(**d)
    g = ops.gated_mlp_bwd(dy.cuda(), **d)
    want, bound = mlp.full(**d, act="silu", dy=dy.cuda())
    cpu = lambda x: {k: v.cpu() for k, v in x.items()}  # noqa: E731
    compare(dict(y=y, **g._asdict()), cpu(want), cpu(bound))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("C", [8, 136])
def test_every_digit_of_the_activation(C, act):
    """One hidden unit at every bf16 value from -12.5 to 12.5: y = act(g) and dx = act'(g), right to the rounding of the
    product's operand and of the result.  Sizes whose forward is one kernel, and two.  2^-14 of a value's terms for the
    fp32 steps (an exponent of up to 113 in fp32: 113 2^-24 ln 2 < 2^-17.6, and a few steps of 2^-20)."""
    bits = torch.arange(0, 0x4148 + 1, dtype=torch.int32).to(torch.int16)  # 0 .. 12.5
    g = bits.view(BF16)
    g = torch.cat([g[g >= 2.0 ** -20], -g[g >= 2.0 ** -20], torch.zeros(1, dtype=BF16)])
    assert g.max() == 12.5 and len(g) > 6000
    x = torch.zeros((len(g), C), dtype=BF16)
    x[:, 0] = g
    w_gate, w_up, w_down = (torch.zeros(n, dtype=BF16) for n in ((8, C), (8, C), (C, 8)))
    w_gate[0, 0] = w_down[0, 0] = 1
    b_up = torch.ones(8, dtype=BF16)
    d = [t.cuda() for t in (x, w_gate, w_up, w_down)]
    y = ops.gated_mlp_fwd(*d, b_up=b_up.cuda(), act=act)[:, 0].double().cpu()
    dy = torch.zeros_like(d[0])
    dy[:, 0] = 1
    dx = ops.gated_mlp_bwd(dy, *d, b_up=b_up.cuda(), act=act).dx[:, 0].double().cpu()
    a = g.double()
    if act == "silu":
        s = torch.sigmoid(a)
        want, slope, terms = a * s, s * (1 + a * (1 - s)), s * (1 + a.abs() * (1 - s))
    else:
        cdf = 0.5 * torch.erfc(-a / 2 ** 0.5)
        phi = torch.exp(-0.5 * a * a) / (2 * torch.pi) ** 0.5
        want, slope, terms = a * cdf, cdf + a * phi, cdf + a.abs() * phi
    half = torch.finfo(BF16).eps / 2
    # h is rounded, and y is h; dg is rounded, and dx is dg
    over = (y - want).abs() - (half + 2.0 ** -14) * want.abs()
    assert over.max() <= 0, f"act({float(a[over.argmax()])}): {float(y[over.argmax()])}, {float(want[over.argmax()])}"
    over = (dx - slope).abs() - half * slope.abs() - 2.0 ** -14 * terms
    assert over.max() <= 0, f"act'({float(a[over.argmax()])}): {float(dx[over.argmax()])}, {float(slope[over.argmax()])}"
