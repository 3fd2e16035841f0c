"""One transformer layer from the three operators, as a model would call them: residual step -> projections -> windowed
attention with a relative position bias -> residual step -> gated feed-forward -> residual step; outputs and gradients
against the same layer in fp64 by torch's autograd, captured and replayed, on two streams at once; and what the Python
functions refuse."""
import math

import pytest
import torch
import torch.nn.functional as F

from oracle.relbias import displacement_index
from oracle.resnorm import keep_mask
from vision_transformer_windowed_b200 import _lib, ops

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(autouse=True)
def _device_status_clean():
    _lib.fs_set_wait_limit_ns(4_000_000_000)
    _lib.fs_device_status()
    yield
    torch.cuda.synchronize()
    assert _lib.fs_device_status() == 0


def draw(B, H, W, heads, M, stream, hidden, seed=0):
    g = torch.Generator().manual_seed(seed)
    C = 32 * heads
    n = lambda *shape, std=1.0: torch.randn(shape, generator=g) * std  # noqa: E731
    t = dict(x=n(B, H, W, C).to(stream), f=n(B, H, W, C).to(BF16), w_qkv=n(3 * C, C, std=C ** -0.5).to(BF16),
             w_o=n(C, C, std=C ** -0.5).to(BF16), table=n(heads, (2 * M - 1) ** 2, std=0.5).to(BF16),
             w_gate=n(hidden, C, std=C ** -0.5).to(BF16), w_up=n(hidden, C, std=C ** -0.5).to(BF16),
             w_down=n(C, hidden, std=hidden ** -0.5).to(BF16), b_gate=n(hidden, std=0.2).to(BF16),
             b_up=n(hidden, std=0.2).to(BF16), b_down=n(C, std=0.2).to(BF16))
    for i in (1, 2):
        t[f"scale{i}"] = n(C, std=0.5).to(stream)
        t[f"norm{i}"] = (1 + n(C, std=0.2)).to(stream)
        t[f"shift{i}"] = n(C, std=0.2).to(stream)
    t["gate"] = torch.tensor([1.25 if b % 3 != 1 else 0.0 for b in range(B)]).to(stream)
    return t, n(B, H, W, C).to(BF16), n(B, H, W, C).to(stream)


def layer(t, M, s, p, rng):
    B, H, W, C = t["x"].shape
    heads = C // 32
    r0, n0 = ops.residual_norm(t["x"], t["f"], pre="layer", pre_weight=t["norm1"], pre_bias=t["shift1"])
    q, k, v = (x.contiguous().view(B, H, W, heads, 32) for x in F.linear(n0, t["w_qkv"]).chunk(3, -1))
    a = ops.window_attention_relbias(q, k, v, t["table"], M, s)
    a = F.linear(a.view(B, H, W, C), t["w_o"])
    r1, n1 = ops.residual_norm(r0, a, gate=t["gate"], scale=t["scale1"], pre="rms", pre_weight=t["norm2"], p=p, rng=rng)
    y = ops.gated_mlp(n1, t["w_gate"], t["w_up"], t["w_down"], t["b_gate"], t["b_up"], t["b_down"], act="gelu")
    r2, n2 = ops.residual_norm(r1, y, scale=t["scale2"], post="layer", post_bias=t["shift2"], pre="layer")
    return n2, r2


def plain(t, M, s, p, rng):
    """The layer in t's (64-bit) type."""
    B, H, W, C = t["x"].shape
    heads = C // 32

    def windows(x):  # [B, windows, heads, M*M, 32]
        x = torch.roll(x, (-s, -s), (1, 2)).view(B, H // M, M, W // M, M, heads, 32)
        return x.permute(0, 1, 3, 5, 2, 4, 6).reshape(B, (H // M) * (W // M), heads, M * M, 32)

    n0 = F.layer_norm(t["x"] + t["f"], (C,), t["norm1"], t["shift1"])
    q, k, v = (windows(x.view(B, H, W, heads, 32)) for x in F.linear(n0, t["w_qkv"]).chunk(3, -1))
    S = q @ k.transpose(-1, -2) / math.sqrt(32) + t["table"][:, displacement_index(M)][None, None]
    if s:
        cut = lambda n: torch.bucketize(torch.arange(n), torch.tensor([n - M, n - s]), right=True)  # noqa: E731
        lab = (3 * cut(H)[:, None] + cut(W)[None]).view(H // M, M, W // M, M).permute(0, 2, 1, 3).reshape(-1, M * M)
        S = S.masked_fill((lab[:, :, None] != lab[:, None])[None, :, None], -math.inf)
    a = (S.softmax(-1) @ v).view(B, H // M, W // M, heads, M, M, 32).permute(0, 1, 4, 2, 5, 3, 6).reshape(B, H, W, C)
    a = F.linear(torch.roll(a, (s, s), (1, 2)), t["w_o"])
    if p:
        a = a * keep_mask(a.shape, p, *rng.tolist()).to(a.dtype) / (1 - p)
    r1 = t["x"] + t["f"] + t["gate"].view(B, 1, 1, 1) * t["scale1"] * a
    n1 = r1 * torch.rsqrt((r1 * r1).mean(-1, keepdim=True) + 1e-5) * t["norm2"]
    y = F.linear(F.gelu(F.linear(n1, t["w_gate"], t["b_gate"])) * F.linear(n1, t["w_up"], t["b_up"]), t["w_down"],
                 t["b_down"])
    r2 = r1 + t["scale2"] * (F.layer_norm(y, (C,)) + t["shift2"])
    return F.layer_norm(r2, (C,)), r2


# Roundings to bf16 between an input and an output: n0, q/k/v, P, o, the projection, n1, h, y, n2 and, with a bf16
# stream, r three times; and as many on the way back, whose factors are the forward's rounded values.  Each is off by
# at most half a step, 2^-8 of its value, and norms, softmax and products pass a relative error on about as it is:
# in the L2 norm the sum of them all bounds an output (12) and a gradient (24).
HALF = torch.finfo(BF16).eps / 2


def near(name, got, want, roundings):
    got, want = got.detach().double().cpu(), want.detach()
    assert torch.isfinite(got).all(), name
    err = float((got - want).norm() / want.norm())
    assert err <= roundings * HALF, f"{name}: {err:.3g} over {roundings * HALF:.3g}"


@pytest.mark.parametrize("B,H,W,heads,M,s,stream,p", [(2, 16, 24, 2, 8, 4, F32, 0.0), (3, 16, 16, 3, 8, 0, BF16, 0.1),
                                                      (1, 32, 32, 2, 16, 8, BF16, 0.0), (2, 8, 8, 1, 4, 0, F32, 0.25),
                                                      (1, 64, 32, 1, 32, 16, F32, 0.0)])
def test_layer_and_its_gradients(B, H, W, heads, M, s, stream, p):
    t, dn, dr = draw(B, H, W, heads, M, stream, 32 * heads * 2 + 40)
    rng = torch.tensor([17, 5])
    leaves = {k: v.cuda().requires_grad_() for k, v in t.items()}
    n2, r2 = layer(leaves, M, s, p, rng.cuda())
    got = torch.autograd.grad([n2, r2], list(leaves.values()), [dn.cuda(), dr.cuda()])
    exact = {k: v.double().requires_grad_() for k, v in t.items()}
    n2_, r2_ = plain(exact, M, s, p, rng)
    want = torch.autograd.grad([n2_, r2_], list(exact.values()), [dn.double(), dr.double()])
    near("n2", n2, n2_, 12)
    near("r2", r2, r2_, 12)
    for k, a, b in zip(leaves, got, want):
        near("d" + k, a, b, 24)


def test_gradient_against_differences():
    """The layer's gradient along a direction is the slope of its fp64 form along it."""
    t, dn, dr = draw(1, 16, 16, 2, 8, F32, 104, seed=3)
    leaves = {k: v.cuda().requires_grad_() for k, v in t.items()}
    n2, r2 = layer(leaves, 8, 4, 0.0, None)
    got = torch.autograd.grad([n2, r2], list(leaves.values()), [dn.cuda(), dr.cuda()])
    g = torch.Generator().manual_seed(4)
    way = {k: torch.randn(v.shape, generator=g, dtype=F64) for k, v in t.items()}

    def at(h):
        n, r = plain({k: v.double() + h * way[k] for k, v in t.items()}, 8, 4, 0.0, None)
        return float((n * dn.double()).sum() + (r * dr.double()).sum())

    h = 1e-5
    slope = (at(h) - at(-h)) / (2 * h)
    ours = sum(float((a.double().cpu() * way[k]).sum()) for k, a in zip(leaves, got))
    # each gradient is within 24 half steps of its own in the L2 norm; a random direction sees its norm
    size = math.sqrt(sum(float(a.double().norm()) ** 2 for a in got))
    assert abs(slope - ours) <= 4 * 24 * HALF * size


def test_captured_and_replayed():
    t, dn, dr = draw(2, 16, 16, 2, 8, F32, 104)
    rng = torch.tensor([1, 2], device="cuda")
    d = {k: v.cuda().requires_grad_() for k, v in t.items()}
    dn, dr = dn.cuda(), dr.cuda()

    def step():
        n2, r2 = layer(d, 8, 4, 0.1, rng)
        return (n2, r2, *torch.autograd.grad([n2, r2], list(d.values()), [dn, dr]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (2, 3):
        rng[1] = seed
        graph.replay()
        torch.cuda.synchronize()
        kept = [x.clone() for x in out]
        for name, a, b in zip(("n2", "r2", *d), kept, step()):  # the projections may take another library kernel
            near(name, a, b.detach().double().cpu(), 2)


def test_two_streams_at_once():
    sets = [draw(2, 32, 32, 2, 16, BF16, 136, seed=i) for i in (0, 1)]
    cuda = [({k: v.cuda().requires_grad_() for k, v in t.items()}, dn.cuda(), dr.cuda()) for t, dn, dr in sets]

    def step(i):
        t, dn, dr = cuda[i]
        n2, r2 = layer(t, 16, 8, 0.0, None)
        return (n2, r2, *torch.autograd.grad([n2, r2], list(t.values()), [dn, dr]))

    alone = [[x.detach().clone() for x in step(i)] for i in (0, 1)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i] = step(i)
    torch.cuda.synchronize()
    for i in (0, 1):
        # the projections may take another library kernel, and dq of windows of 16 or more adds fp32 sums in
        # the order they come: what lies behind them may round the other way
        for name, a, b in zip(("n2", "r2", *cuda[i][0]), got[i], alone[i]):
            near(name, a, b.double().cpu(), 2)


# ------------------------------------------------------------------ refusals
def cuda(*shape, dtype=BF16):
    return torch.zeros(shape, device="cuda", dtype=dtype)


def test_refused_attention():
    q, table = cuda(1, 16, 16, 2, 32), cuda(2, 225)
    fwd = lambda *a, **kw: ops.winattn_relbias_fwd(*a, 8, 4, **kw)  # noqa: E731
    cases = [((q.float(), q, q, table), {}, "q must be"), ((q, q.float(), q, table), {}, "k must be"),
             ((q, cuda(1, 16, 16, 3, 32), q, table), {}, "k has shape"),
             ((q, q, q.transpose(1, 2), table), {}, "v must be contiguous"),
             ((q, q, q, table.float()), {}, "table must be"), ((q, q, q, cuda(3, 225)), {}, "table has shape"),
             ((q, q, q, table[0]), {}, "table must be"), ((q, q, q, cuda(2, 100)), {}, "225 entries"),
             ((q, q, q, table), dict(buckets=cuda(15, 15)), "buckets must be"),
             ((q, q, q, table), dict(buckets=cuda(15, 14, dtype=torch.int32)), "buckets has shape"),
             ((q, q, q, table), dict(o=cuda(1, 16, 16, 2, 32, dtype=F32)), "o must be"),
             ((q, q, q, table), dict(lse=cuda(1, 16, 16, 2)), "lse must be")]
    for args, kw, message in cases:
        with pytest.raises(ValueError, match=message):
            fwd(*args, **kw)
    with pytest.raises(_lib.FswinError):
        ops.winattn_relbias_fwd(q, q, q, cuda(2, 529), 12, 0)
    lse = cuda(1, 16, 16, 2, dtype=F32)
    with pytest.raises(ValueError, match="dout"):
        ops.winattn_relbias_bwd(q, q, q, q, q.float(), lse, table, 8, 4)
    with pytest.raises(ValueError, match="workspace"):
        ops.winattn_relbias_bwd(q, q, q, q, q, lse, table, 8, 4, workspace=cuda(64))
    with pytest.raises(_lib.FswinError):
        ops.winattn_relbias_bwd(q, q, q, q, q, lse, table, 8, 4, workspace=cuda(256, dtype=torch.uint8))


def test_refused_residual_step():
    x, f = cuda(2, 5, 96), cuda(2, 5, 96)
    cases = [((x, f.float()), {}, "f must be"), ((x, f[:, :4]), {}, "f has shape"),
             ((x.transpose(0, 1), f.transpose(0, 1)), {}, "contiguous"), ((x, f), dict(gate=cuda(3)), "gate has shape"),
             ((x, f), dict(scale=cuda(96, dtype=F32)), "scale must be"), ((x, f), dict(pre_weight=cuda(95)), "pre_weight"),
             ((x, f), dict(r=cuda(2, 5, 96, dtype=F32)), "r must be"), ((x, f), dict(n=cuda(2, 5, 95)), "n has shape"),
             ((x, f), dict(p=0.1), "rng"), ((x, f), dict(p=0.1, rng=cuda(2)), "rng"),
             ((x, f), dict(p=0.1, rng=cuda(3, dtype=torch.int64)), "rng")]
    for args, kw, message in cases:
        with pytest.raises(ValueError, match=message):
            ops.residual_norm_fwd(*args, **kw)
    for kw in (dict(p=1.0, rng=cuda(2, dtype=torch.int64)), dict(eps=-1.0), dict(pre=None, pre_weight=cuda(96)),
               dict(post_bias=cuda(96))):
        with pytest.raises((ValueError, _lib.FswinError)):
            ops.residual_norm_fwd(x, f, **kw)
    with pytest.raises(ValueError, match="dn without"):
        ops.residual_norm_bwd(x, f, x, f, pre=None)
    with pytest.raises(ValueError, match="workspace"):
        ops.residual_norm_bwd(x, f, x, f, workspace=cuda(64))


def test_refused_feed_forward():
    x, w, wd = cuda(5, 96), cuda(256, 96), cuda(96, 256)
    cases = [((x.float(), w, w, wd), {}, "x must be"), ((x, w, cuda(255, 96), wd), {}, "w_up has shape"),
             ((x, w, w, w), {}, "w_down has shape"), ((x, w, w, wd), dict(b_gate=cuda(96)), "b_gate has shape"),
             ((x, w, w, cuda(256, 96).t()), {}, "w_down must be contiguous"),
             ((x, w, w, wd), dict(y=cuda(5, 96, dtype=F32)), "y must be")]
    for args, kw, message in cases:
        with pytest.raises(ValueError, match=message):
            ops.gated_mlp_fwd(*args, **kw)
    with pytest.raises(_lib.FswinError):
        ops.gated_mlp_fwd(cuda(5, 92), cuda(256, 92), cuda(256, 92), cuda(92, 256))
    wide = cuda(5, 264), cuda(256, 264), cuda(256, 264), cuda(264, 256)  # weights beyond shared memory: h has a workspace
    with pytest.raises(_lib.FswinError):
        ops.gated_mlp_fwd(*wide, workspace=cuda(256, dtype=torch.uint8))
    with pytest.raises(_lib.FswinError):
        ops.gated_mlp_bwd(x, x, w, w, wd, workspace=cuda(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="dy has shape"):
        ops.gated_mlp_bwd(cuda(4, 96), x, w, w, wd)


@pytest.mark.parametrize("stream", [BF16, F32], ids=["bf16", "f32"])
def test_each_gradient_against_differences(stream):
    """Each input's gradient along a direction of its own against the slope of the layer's fp64 form: 24 half steps of
    that gradient's fp64 norm (as for the whole gradient, which this direction sees no more of than its norm)."""
    t, dn, dr = draw(2, 16, 16, 2, 8, stream, 104, seed=3)
    leaves = {k: v.cuda().requires_grad_() for k, v in t.items()}
    n2, r2 = layer(leaves, 8, 4, 0.0, None)
    got = dict(zip(leaves, torch.autograd.grad([n2, r2], list(leaves.values()), [dn.cuda(), dr.cuda()])))
    exact = {k: v.double().requires_grad_() for k, v in t.items()}
    n2_, r2_ = plain(exact, 8, 4, 0.0, None)
    want = dict(zip(exact, torch.autograd.grad([n2_, r2_], list(exact.values()), [dn.double(), dr.double()])))
    base = {k: v.double() for k, v in t.items()}
    for k, v in t.items():
        # along the gradient, where the slope is its norm, and as far across, where it is none
        along = want[k] / want[k].norm()
        way = torch.randn(v.shape, generator=torch.Generator().manual_seed(len(k)), dtype=F64)
        way -= (way * along).sum() * along
        way = way / way.norm() + along

        def at(h):
            n, r = plain({**base, k: base[k] + h * way}, 8, 4, 0.0, None)
            return float((n * dn.double()).sum() + (r * dr.double()).sum())

        h = 1e-4
        slope = (at(h) - at(-h)) / (2 * h)
        size = float(want[k].norm())
        ours = float((got[k].double().cpu() * way).sum())
        assert abs(slope - size) <= 1e-3 * size, k
        assert abs(slope - ours) <= 24 * HALF * size * float(way.norm()), f"{k}: {ours}, {slope}"


# ------------------------------------------------------------------ threads
def entry_points():
    """Calls with every output and workspace given, so that no allocation precedes them; M = 16 and the feed-forward
    read their tensors through TMA maps."""
    from vision_transformer_windowed_b200.inputs import make_inputs

    inp = {k: v.cuda() for k, v in make_inputs(1, 32, 32, 2, 32).items()}
    q, k, v, dout, theta = (inp[n] for n in ("q", "k", "v", "dout", "theta"))
    table = torch.zeros((2, 31 * 31), device="cuda", dtype=BF16)
    o, lse, dq, dk, dv = (torch.empty_like(q), torch.empty(q.shape[:4], device="cuda"), *(torch.empty_like(q) for _ in "qkv"))
    ws, ws_rb = ops.alloc_workspace(q, 16, 8), ops.alloc_relbias_workspace(q, 16, 8)
    x, w, wd, y = (torch.ones(s, device="cuda", dtype=BF16) for s in ((5, 264), (256, 264), (264, 256), (5, 264)))
    ws_mlp = torch.empty(1 << 16, device="cuda", dtype=torch.uint8)
    dtheta, dtable = torch.empty_like(theta), torch.empty_like(table)
    return dict(
        rope_fwd=lambda: ops.winattn_fwd(q, k, v, theta, 16, 8, o=o, lse=lse),
        rope_bwd=lambda: ops.winattn_bwd(q, k, v, o, dout, lse, theta, 16, 8, workspace=ws, dq=dq, dk=dk, dv=dv,
                                         dtheta=dtheta),
        relbias_fwd=lambda: ops.winattn_relbias_fwd(q, k, v, table, 16, 8, o=o, lse=lse),
        relbias_bwd=lambda: ops.winattn_relbias_bwd(q, k, v, o, dout, lse, table, 16, 8, workspace=ws_rb, dq=dq, dk=dk,
                                                    dv=dv, dtable=dtable),
        mlp_fwd=lambda: ops.gated_mlp_fwd(x, w, w, wd, y=y, workspace=ws_mlp))


def test_first_call_of_a_thread():
    """A thread that has made no CUDA call yet, as the autograd engine's may be: the library's call is its first."""
    from threading import Thread

    for name, call in entry_points().items():
        call()  # what a first call sets up is not at issue
        torch.cuda.synchronize()
        raised = []

        def body():
            try:
                call()
            except Exception as e:  # noqa: BLE001
                raised.append(e)

        t = Thread(target=body)
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert not raised, f"{name}: {raised[0]}"


# ------------------------------------------------------------------ second derivatives
def test_no_second_derivative_by_mistake():
    """The gradients have no gradient of their own: asking for one is refused, not answered with zero."""
    from vision_transformer_windowed_b200.inputs import make_inputs

    inp = {k: v.cuda().requires_grad_() for k, v in make_inputs(1, 16, 16, 2, 32).items()}
    q, k, v, theta = (inp[n] for n in ("q", "k", "v", "theta"))
    u = torch.randn((2, 256, 16), device="cuda", requires_grad=True)
    table = torch.randn((2, 31 * 31), device="cuda").to(BF16).requires_grad_()
    x, w, wd = (torch.randn(s, device="cuda").to(BF16).requires_grad_() for s in ((5, 64), (128, 64), (64, 128)))
    for name, out, leaf in (("rope", ops.window_attention(q, k, v, theta, 16, 0), theta),
                            ("low rank", ops.window_attention_lrbias(q, k, v, theta, u, u, 16, 0), u),
                            ("relative bias", ops.window_attention_relbias(q, k, v, table, 16, 0), table),
                            ("residual step", ops.residual_norm(x, x)[1], x), ("feed-forward", ops.gated_mlp(x, w, w, wd), w)):
        grad = torch.autograd.grad(out.float().square().sum(), leaf, create_graph=True)[0]
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (grad.float().square().sum() + leaf.float().sum()).backward()


def test_threads_at_once():
    """Four host threads, a stream and tensors each, the whole layer forward and backward."""
    from threading import Thread

    sets = [draw(2, 32, 32, 2, 16, BF16, 136, seed=i) for i in range(4)]
    cuda = [({k: v.cuda().requires_grad_() for k, v in t.items()}, dn.cuda(), dr.cuda()) for t, dn, dr in sets]

    def step(i):
        t, dn, dr = cuda[i]
        n2, r2 = layer(t, 16, 8, 0.0, None)
        return (n2, r2, *torch.autograd.grad([n2, r2], list(t.values()), [dn, dr]))

    alone = [[x.detach().clone() for x in step(i)] for i in range(4)]
    torch.cuda.synchronize()
    got, raised = [None] * 4, []

    def body(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    got[i] = step(i)
        except Exception as e:  # noqa: BLE001
            raised.append(e)

    threads = [Thread(target=body, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not raised, raised[0]
    for i in range(4):
        for name, a, b in zip(("n2", "r2", *cuda[i][0]), got[i], alone[i]):  # as for two streams
            near(name, a, b.double().cpu(), 2)
