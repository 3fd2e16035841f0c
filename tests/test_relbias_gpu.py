"""GPU parity of the relative-position-bias attention against its fp64 oracle, element by element within the oracle's
own error bounds; lse (fp32) within 2^-16 of the larger of 1 and its size (fp32 scores of a few tens, their sum and
the logarithm's and exponential's few steps of 2^-22)."""
import pytest
import torch

from oracle import relbias
from vision_transformer_windowed_b200 import _lib, ops
from vision_transformer_windowed_b200.inputs import make_inputs

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(autouse=True)
def _device_status_clean():
    _lib.fs_set_wait_limit_ns(4_000_000_000)
    _lib.fs_device_status()
    yield
    torch.cuda.synchronize()
    assert _lib.fs_device_status() == 0


def draw(B, H, W, heads, M, n=None, qk_scale=1.0, std=0.7, seed=3):
    inp = make_inputs(B, H, W, heads, 32, qk_scale=qk_scale)
    inp.pop("theta")
    g = torch.Generator().manual_seed(seed)
    n = (2 * M - 1) ** 2 if n is None else n
    inp["table"] = (torch.randn((heads, n), generator=g) * std).to(torch.bfloat16)
    return inp


def run(inp, M, s, buckets=None):
    d = {k: t.cuda() for k, t in inp.items()}
    bk = None if buckets is None else buckets.cuda()
    o, lse = ops.winattn_relbias_fwd(d["q"], d["k"], d["v"], d["table"], M, s, buckets=bk)
    dq, dk, dv, dt = ops.winattn_relbias_bwd(d["q"], d["k"], d["v"], o, d["dout"], lse, d["table"], M, s, buckets=bk)
    torch.cuda.synchronize()
    return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv, dtable=dt)


def compare(got, ref, err, keys=("o", "lse", "dq", "dk", "dv", "dtable")):
    for key in keys:
        a, b = got[key].double().cpu(), ref[key]
        assert a.shape == b.shape, key
        if key == "lse":
            fine = torch.isfinite(b)
            assert torch.equal(a[~fine], b[~fine])
            assert ((a - b)[fine].abs() <= 2.0 ** -16 * b[fine].abs().clamp(min=1.0)).all(), key
            continue
        assert torch.isfinite(a).all(), f"{key}: non-finite values"
        # 1e-6 of the largest: fp32 sums that cancel to near zero
        over = (a - b).abs() - (err[key] * (1 + 1e-3) + 1e-6 * max(1.0, float(b.abs().max())))
        assert over.max() <= 0, f"{key}: {float(over.max()):.3g} over its bound, error {float((a - b).abs().max()):.3g}"


CASES = [  # (B, H, W, heads, M, s)
    (1, 4, 4, 1, 4, 0),
    (1, 8, 12, 2, 4, 0),      # 6 windows: a ragged tile
    (2, 10, 6, 3, 4, 0),      # padded
    (1, 8, 8, 1, 8, 0),       # one window: half a tile
    (2, 16, 16, 2, 8, 0),
    (2, 16, 16, 3, 8, 4),
    (1, 8, 24, 1, 8, 4),      # three windows
    (1, 20, 13, 2, 8, 4),     # padded, shifted
    (1, 16, 16, 5, 16, 0),
    (1, 32, 32, 2, 16, 8),
    (1, 32, 48, 1, 16, 4),
    (1, 40, 36, 2, 16, 12),   # padded
    (1, 32, 32, 2, 32, 0),
    (1, 64, 64, 1, 32, 16),
    (1, 64, 40, 1, 32, 8),
    (1, 33, 64, 1, 32, 20),
    (1, 64, 64, 1, 64, 0),
    (1, 64, 64, 1, 64, 32),
    (1, 64, 70, 1, 64, 16),
    (1, 64, 64, 1, 64, 24),
    (1, 64, 64, 1, 64, 4),
]


@pytest.mark.parametrize("cfg", CASES)
def test_parity(cfg):
    inp = draw(*cfg[:5])
    compare(run(inp, *cfg[4:]), *relbias.full(inp["q"], inp["k"], inp["v"], inp["table"], *cfg[4:], dout=inp["dout"]))


@pytest.mark.parametrize("cfg", [(1, 8, 12, 2, 4, 0), (2, 16, 16, 3, 8, 4), (1, 32, 32, 2, 16, 8), (1, 32, 32, 40, 16, 0),
                                 (1, 64, 64, 1, 32, 16)])
def test_parity_by_buckets(cfg):
    """Shared buckets, with some displacements outside the table on either side."""
    B, H, W, heads, M, s = cfg
    buckets, n = ops.log_distance_buckets(M, exact=2, device="cpu")
    buckets[0, 0], buckets[-1, -1], buckets[M - 1, 0] = -1, n, 2 ** 31 - 1
    inp = draw(B, H, W, heads, M, n)
    compare(run(inp, M, s, buckets), *relbias.full(inp["q"], inp["k"], inp["v"], inp["table"], M, s, buckets=buckets,
                                                  dout=inp["dout"]))


@pytest.mark.parametrize("cfg", [(1, 8, 8, 2, 4, 0), (2, 16, 16, 3, 8, 4), (1, 32, 32, 2, 16, 8), (1, 64, 64, 1, 32, 16)])
def test_sharp_softmax_and_masked_displacements(cfg):
    """Peaked rows, a wide bias, entries of -inf and of the type's lowest value."""
    B, H, W, heads, M, s = cfg
    inp = draw(B, H, W, heads, M, qk_scale=3.0, std=4.0)
    n = inp["table"].shape[1]
    inp["table"][:, 1] = -INF
    inp["table"][0, n // 2 + 1] = -INF
    inp["table"][0, 2:n // 3] = torch.finfo(torch.bfloat16).min
    compare(run(inp, M, s), *relbias.full(inp["q"], inp["k"], inp["v"], inp["table"], M, s, dout=inp["dout"]))


@pytest.mark.parametrize("M", [4, 8, 16, 32])
def test_rows_without_a_key(M):
    """Head 0 attends nothing, head 1 only one displacement that the window's last rows lack."""
    inp = draw(1, M, M, 2, M)
    inp["table"][:] = -INF
    inp["table"][1, (M - 2) * (2 * M - 1) + M - 1] = 0.25  # the key one row below
    got = run(inp, M, 0)
    ref, err = relbias.full(inp["q"], inp["k"], inp["v"], inp["table"], M, 0, dout=inp["dout"])
    assert (ref["lse"][..., 0] == -INF).all() and torch.isfinite(ref["lse"][0, :-1, :, 1]).all()
    compare(got, ref, err)
    assert (got["o"][..., 0, :] == 0).all() and (got["dq"][..., 0, :] == 0).all()


@pytest.mark.parametrize("M", [4, 8, 16])
def test_every_entry_of_the_lowest_value_is_the_uniform_row(M):
    inp = draw(1, M, M, 1, M)
    inp["table"][:] = torch.finfo(torch.bfloat16).min
    o, _ = ops.winattn_relbias_fwd(*(inp[k].cuda() for k in ("q", "k", "v", "table")), M, 0, need_lse=False)
    mean = inp["v"].double().reshape(-1, 32).mean(0)
    bound = 2.0 ** -7 * inp["v"].double().abs().reshape(-1, 32).mean(0)  # P's rounding and o's
    assert ((o.double().cpu() - mean).abs() <= bound).all()


@pytest.mark.parametrize("M", [4, 8])
def test_values_that_are_not_finite_stay_in_their_window(M):
    """Small windows share a tile with their neighbours."""
    inp = draw(1, M, 4 * M, 1, M)
    clean = run(inp, M, 0)
    for name in ("q", "k", "v", "dout"):
        inp[name][:, :, M:2 * M] = INF if name == "v" else float("nan")
    got = run(inp, M, 0)
    for key in ("o", "lse", "dq", "dk", "dv"):
        for part in (slice(0, M), slice(2 * M, 4 * M)):
            assert torch.equal(got[key][:, :, part], clean[key][:, :, part]), key


def test_inference_forward_repeats_and_leaves_nothing_else_written():
    inp = draw(2, 40, 36, 2, 16)
    d = {k: t.cuda() for k, t in inp.items()}
    a = run(inp, 16, 8)
    b = run(inp, 16, 8)
    o, none = ops.winattn_relbias_fwd(d["q"], d["k"], d["v"], d["table"], 16, 8, need_lse=False)
    assert none is None and torch.equal(o, a["o"])
    for key in ("o", "lse", "dk", "dv", "dtable"):
        assert torch.equal(a[key], b[key]), key
    # outputs inside larger buffers: the bytes around them stay
    big = torch.full((o.numel() + 64,), 7.0, device="cuda", dtype=torch.bfloat16)
    view = big[32:-32].view(o.shape)
    ops.winattn_relbias_fwd(d["q"], d["k"], d["v"], d["table"], 16, 8, o=view, need_lse=False)
    assert torch.equal(view, o) and (big[:32] == 7).all() and (big[-32:] == 7).all()


@pytest.mark.parametrize("M", [8, 16])
def test_autograd_other_stream_and_graph(M):
    inp = draw(1, 32, 32, 2, M)
    want = run(inp, M, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        leaves = [inp[k].cuda().requires_grad_() for k in ("q", "k", "v", "table")]
        o = ops.window_attention_relbias(*leaves, M, 0)
        grads = torch.autograd.grad(o, leaves, inp["dout"].cuda())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(o.detach(), want["o"])
    for t, key in zip(grads, ("dq", "dk", "dv", "dtable")):
        if key == "dq" and M >= 16:  # two fp32 sums in either order: commutative, equal up to the zero they start from
            assert (t.float() - want[key].float()).abs().max() <= 2.0 ** -7 * want[key].float().abs().max()
        else:
            assert torch.equal(t, want[key]), key
    d = {k: t.cuda() for k, t in inp.items()}
    ws = ops.alloc_relbias_workspace(d["q"], M, 0)
    out, lse = ops.winattn_relbias_fwd(d["q"], d["k"], d["v"], d["table"], M, 0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.winattn_relbias_fwd(d["q"], d["k"], d["v"], d["table"], M, 0, o=out, lse=lse)
        dq, dk, dv, dt = ops.winattn_relbias_bwd(d["q"], d["k"], d["v"], out, d["dout"], lse, d["table"], M, 0,
                                                 workspace=ws)
    new = draw(1, 32, 32, 2, M, seed=9)
    d["table"].copy_(new["table"])
    inp["table"] = new["table"]
    g.replay()
    torch.cuda.synchronize()
    again = run(inp, M, 0)
    assert torch.equal(out, again["o"]) and torch.equal(dt, again["dtable"]) and torch.equal(dk, again["dk"])


def test_empty_batch_zeroes_the_table_gradient():
    inp = draw(0, 16, 16, 2, 8)
    got = run(inp, 8, 0)
    assert got["o"].numel() == 0 and (got["dtable"] == 0).all()


@pytest.mark.parametrize("cfg", [(1, 8, 8, 700, 8, 0), (1, 8, 8, 500, 4, 0), (1, 16, 16, 200, 16, 0)])
def test_more_heads_than_ctas(cfg):
    inp = draw(*cfg[:5])
    compare(run(inp, *cfg[4:]), *relbias.full(inp["q"], inp["k"], inp["v"], inp["table"], *cfg[4:], dout=inp["dout"]))


@pytest.mark.parametrize("cfg", [(1, 8, 8, 2, 4, 0), (1, 16, 16, 2, 8, 4), (1, 32, 32, 2, 16, 8)])
def test_one_bucket_for_every_pair(cfg):
    """A constant bias: the softmax does not see it, and its gradient is the sum of all dS, zero but for roundings."""
    B, H, W, heads, M, s = cfg
    buckets = torch.zeros((2 * M - 1, 2 * M - 1), dtype=torch.int32)
    inp = draw(B, H, W, heads, M, 1)
    compare(run(inp, M, s, buckets), *relbias.full(inp["q"], inp["k"], inp["v"], inp["table"], M, s, buckets=buckets,
                                                  dout=inp["dout"]))


def places(M):
    """Row and column displacement of every entry of a table without a bucket map."""
    e = torch.arange((2 * M - 1) ** 2)
    return e // (2 * M - 1) - (M - 1), e % (2 * M - 1) - (M - 1)


@pytest.mark.parametrize("cfg", [(1, 16, 16, 1, 16, 0), (1, 32, 32, 1, 16, 8), (1, 32, 32, 1, 32, 0), (1, 64, 64, 1, 64, 0)])
def test_a_small_entry_of_the_table_gradient_beside_large_ones(cfg):
    """Keys to the right of their query get e^-25 of the weight: their entries of dtable are some 1e-9 of the others',
    and as exact by the oracle's bound, which has no part of the others in it."""
    B, H, W, heads, M, s = cfg
    inp = draw(*cfg[:5])
    inp["dout"] = inp["dout"] * 64
    right = places(M)[1] < 0
    inp["table"][:, right] -= 25
    ref, err = relbias.full(inp["q"], inp["k"], inp["v"], inp["table"], M, s, dout=inp["dout"])
    got = run(inp, M, s)["dtable"].double().cpu()
    assert 0 < ref["dtable"][:, right].abs().max() < 1e-6 * ref["dtable"].abs().max()
    assert ((got - ref["dtable"]).abs() <= err["dtable"] * (1 + 1e-3))[:, right].all()


@pytest.mark.parametrize("cfg", [(1, 16, 16, 1, 16, 0), (1, 32, 32, 1, 32, 0), (1, 64, 64, 1, 64, 0)])
def test_a_gradient_that_is_not_finite_reaches_its_own_displacements_only(cfg):
    """The window's first token as query only has displacements that are not positive."""
    B, H, W, heads, M, s = cfg
    inp = draw(*cfg[:5])
    clean = run(inp, M, s)["dtable"]
    inp["dout"][0, 0, 0] = INF
    got = run(inp, M, s)["dtable"]
    di, dj = places(M)
    apart = ((di > 0) | (dj > 0)).cuda()
    assert torch.isnan(got[:, ~apart]).all() and torch.isfinite(got[:, apart]).all()
    # the first token adds nothing to those entries, finite or not
    assert torch.equal(got[:, apart], clean[:, apart])

LOWEST = torch.finfo(torch.bfloat16).min
FAR = [(1, 8, 12, 2, 4, 0), (2, 16, 16, 2, 8, 0), (1, 20, 13, 2, 8, 4), (1, 16, 32, 2, 16, 0), (1, 32, 32, 2, 16, 4),
       (1, 40, 36, 2, 16, 12), (1, 64, 64, 2, 32, 16), (1, 64, 64, 2, 64, 0), (1, 64, 70, 2, 64, 16)]


@pytest.mark.parametrize("cfg", FAR)
def test_lowest_value_for_every_key_of_a_row(cfg):
    """The type's lowest value as a mask.  Head 0: every entry, each row is the uniform one.  Head 1: all but the keys
    of the rows below, so that only the queries of a window's last row have none but masked keys."""
    B, H, W, heads, M, s = cfg
    inp = draw(*cfg[:5])
    inp["table"][0] = LOWEST
    inp["table"][1, places(M)[0] >= 0] = LOWEST
    ref, err = relbias.full(inp["q"], inp["k"], inp["v"], inp["table"], M, s, dout=inp["dout"])
    compare(run(inp, M, s), ref, err, keys=("o", "dq", "dk", "dv", "dtable"))


@pytest.mark.parametrize("cfg", FAR)
@pytest.mark.parametrize("value", [-1e9, 1e9, -3e20])
def test_large_entries_for_every_key_of_a_row(cfg, value):
    """Half a step of fp32 at 1e9 log2(e) is 64, more than any score: as with the lowest value.  The bits are the same,
    but for dq, whose sums at M >= 16 come in any order."""
    B, H, W, heads, M, s = cfg
    inp = draw(*cfg[:5])
    inp["table"][0] = LOWEST
    inp["table"][1, places(M)[1] > 0] = LOWEST
    inp["table"][1, places(M)[1] <= 0] = -INF
    want = run(inp, M, s)
    inp["table"][0] = value
    inp["table"][1, places(M)[1] > 0] = value
    inp["table"][1, places(M)[1] <= 0] = value - 3 * abs(value)
    got = run(inp, M, s)
    assert all(torch.isfinite(got[key]).all() for key in ("o", "dq", "dk", "dv", "dtable"))
    for key in ("o", "dk", "dv"):
        assert torch.equal(got[key][..., 0, :], want[key][..., 0, :]), key
    rows = torch.isfinite(want["lse"][..., 1])  # queries with a key to their left in their region
    assert 0 < rows.sum() < rows.numel() and torch.equal(got["o"][..., 1, :][rows], want["o"][..., 1, :][rows])
    assert torch.equal(got["dtable"][0], want["dtable"][0])
    size = want["dq"].float().abs().max()
    assert (got["dq"].float() - want["dq"].float())[:, :, :, 0].abs().max() <= 2.0 ** -7 * size


@pytest.mark.parametrize("cfg", FAR)
@pytest.mark.parametrize("value", [-9984.0, 9984.0])
def test_a_bias_of_ten_thousand_for_every_key(cfg, value, monkeypatch):
    """A constant: the plain softmax, from scores that fp32 holds to half a step of 2^-10 beside it (base 2), each way
    and in the row's own maximum: less than 2^-9 of a probability."""
    B, H, W, heads, M, s = cfg
    inp = draw(*cfg[:5])
    inp["table"][:] = value
    monkeypatch.setattr(relbias, "EPS_P", 2.0 ** -9)
    ref, err = relbias.full(inp["q"], inp["k"], inp["v"], inp["table"], M, s, dout=inp["dout"])
    compare(run(inp, M, s), ref, err)


# CTAs of a B200 that a forward fills with workers of their own (M >= 16: four a CTA and one CTA an SM, M <= 8: four
# CTAs an SM); the backward has fewer of them.
WORKERS = 4 * 148


@pytest.mark.parametrize("copies,H,W,heads,M,s", [(580, 20, 20, 1, 4, 0), (300, 20, 17, 2, 4, 0), (450, 24, 24, 1, 8, 4),
                                                 (230, 24, 20, 2, 8, 0), (155, 32, 48, 1, 16, 8), (90, 40, 33, 2, 16, 4),
                                                 (230, 32, 32, 1, 16, 0), (60, 64, 64, 1, 32, 16), (120, 33, 64, 2, 32, 0),
                                                 (60, 64, 64, 1, 64, 0), (30, 70, 64, 2, 64, 16)])
def test_many_items_a_worker(copies, H, W, heads, M, s):
    """Every worker walks three items or more, forward and backward.  The images are one image times powers of two, drawn
    for each: q 2^a, k 2^-a, v 2^c, dout 2^e leave P as it is and scale o by 2^c, dv by 2^e, dq by 2^(c+e-a) and dk by
    2^(c+e+a), exactly.  A tile taken from another item than its own shows."""
    tiles = -(-copies * -(-H // M) * -(-W // M) * M * M // 128)
    assert tiles >= 3 * WORKERS // heads
    one = draw(1, H, W, heads, M)
    g = torch.Generator().manual_seed(7)
    a, c, e = (torch.randint(-3, 4, (copies,), generator=g).double() for _ in "ace")
    power = lambda x: torch.exp2(x).view(-1, 1, 1, 1, 1)  # noqa: E731
    scaled = lambda name, x: (one[name].double() * power(x)).to(torch.bfloat16)  # noqa: E731
    many = dict(q=scaled("q", a), k=scaled("k", -a), v=scaled("v", c), dout=scaled("dout", e), table=one["table"])
    ref, err = relbias.full(one["q"], one["k"], one["v"], one["table"], M, s, dout=one["dout"])
    got = run(many, M, s)
    for key, x in (("o", c), ("dq", c + e - a), ("dk", c + e + a), ("dv", e)):
        back = got[key].double().cpu() * power(-x)
        compare({key: back}, {key: ref[key].expand_as(back)}, {key: err[key]}, keys=(key,))
        # (at M = 4 the two windows of a warp add in orders of their own, and dq at M >= 16 as its parts come)
        if M > 4 and (key != "dq" or M == 8):
            assert torch.equal(back, back[:1].expand_as(back)), key
    compare(dict(lse=got["lse"]), dict(lse=ref["lse"].expand_as(got["lse"])), err, keys=("lse",))
    total = float(torch.exp2(c + e).sum())
    compare(dict(dtable=got["dtable"]), dict(dtable=ref["dtable"] * total), dict(dtable=err["dtable"] * total), keys=("dtable",))


@pytest.mark.parametrize("cfg", [(1, 64, 64, 2, 64, 0), (1, 64, 70, 1, 64, 32)])
def test_parity_by_buckets_largest_windows(cfg):
    B, H, W, heads, M, s = cfg
    buckets, n = ops.log_distance_buckets(M, exact=2, device="cpu")
    buckets[0, 0], buckets[-1, -1], buckets[M - 1, 0] = -1, n, 2 ** 31 - 1
    inp = draw(B, H, W, heads, M, n)
    compare(run(inp, M, s, buckets), *relbias.full(inp["q"], inp["k"], inp["v"], inp["table"], M, s, buckets=buckets,
                                                  dout=inp["dout"]))


@pytest.mark.parametrize("copies,H,W,M,s", [(400, 20, 20, 4, 0), (300, 24, 24, 8, 4), (60, 32, 48, 16, 8), (40, 64, 40, 32, 8),
                                            (30, 64, 64, 64, 0)])
def test_one_head_of_large_entries_among_others(copies, H, W, M, s):
    """Many items a worker, the middle head of three masked by the lowest value, captured and replayed: that head is the
    oracle's uniform softmax in every image, the others' bits are those of a table without large entries."""
    one = draw(1, H, W, 3, M)
    many = {k: t if k == "table" else t.expand(copies, *t.shape[1:]).contiguous() for k, t in one.items()}
    clean = run(many, M, s)
    one["table"] = many["table"] = many["table"].clone()
    one["table"][1] = LOWEST
    ref, err = relbias.full(one["q"], one["k"], one["v"], one["table"], M, s, dout=one["dout"])
    eager = run(many, M, s)
    d = {k: t.cuda() for k, t in many.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = ops.winattn_relbias_fwd(d["q"], d["k"], d["v"], d["table"], M, s)
        dq, dk, dv, dt = ops.winattn_relbias_bwd(d["q"], d["k"], d["v"], o, d["dout"], lse, d["table"], M, s)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    replayed = dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv, dtable=dt)
    for got in (eager, replayed):
        for key in ("o", "dq", "dk", "dv"):
            x = got[key].double().cpu()
            compare({key: x}, {key: ref[key].expand_as(x)}, {key: err[key]}, keys=(key,))
        compare(dict(dtable=got["dtable"]), dict(dtable=copies * ref["dtable"]), dict(dtable=copies * err["dtable"]),
                keys=("dtable",))
        for h in (0, 2):
            for key in ("o", "lse", "dk", "dv"):
                assert torch.equal(got[key][:, :, :, h], clean[key][:, :, :, h]), key
            assert torch.equal(got["dtable"][h], clean["dtable"][h])
    for key in ("o", "lse", "dk", "dv", "dtable"):
        assert torch.equal(eager[key], replayed[key]), key


@pytest.mark.parametrize("value", [-1e9, 3e7])
@pytest.mark.parametrize("B,H,M,s", [(8, 128, 4, 0), (8, 128, 8, 4), (8, 128, 16, 8), (8, 128, 32, 0), (4, 128, 64, 32)])
def test_one_key_of_a_large_bias_and_large_scores(B, H, M, s, value):
    """Every query has its own token for its only key, and scores of thousands beside a bias whose steps are 4 or 128 (in
    base 2): whichever way a score is rounded there, P is 1, o = v and dv = dout."""
    inp = draw(B, H, H, 3, M, qk_scale=30.0)
    inp["table"][:] = -INF
    inp["table"][:, (2 * M - 1) ** 2 // 2] = value
    got = run(inp, M, s)
    assert torch.equal(got["o"].cpu(), inp["v"]) and torch.equal(got["dv"].cpu(), inp["dout"])
    # dP - D is a rounding of two equal sums of 32 products of about 1
    for key, size in (("dq", 30.0), ("dk", 30.0)):
        assert got[key].float().abs().max() <= 2.0 ** -10 * size, key


@pytest.mark.parametrize("B,H,W,M,s", [(3, 24, 16, 8, 4), (40, 48, 80, 8, 4), (3, 48, 32, 16, 8), (40, 48, 32, 16, 8),
                                       (2, 96, 64, 32, 16), (1, 128, 64, 64, 32)])
def test_large_entries_that_only_some_windows_feel(B, H, W, M, s):
    """Only keys half a window above or below are without the mask: every query of an ordinary window has one, and no
    query of the last row of windows, which the shift cuts there."""
    inp = draw(1, H, W, 2, M)
    inp["table"][:, places(M)[0].abs() != M // 2] = LOWEST
    ref, err = relbias.full(inp["q"], inp["k"], inp["v"], inp["table"], M, s, dout=inp["dout"])
    far = ref["lse"] < -1e30
    assert 0 < far.sum() < far.numel()
    many = {k: t if k == "table" else t.expand(B, *t.shape[1:]).contiguous() for k, t in inp.items()}
    got = run(many, M, s)
    for key in ("o", "dq", "dk", "dv"):
        x = got[key].double().cpu()
        compare({key: x}, {key: ref[key].expand_as(x)}, {key: err[key]}, keys=(key,))
    compare(dict(dtable=got["dtable"]), dict(dtable=B * ref["dtable"]), dict(dtable=B * err["dtable"]), keys=("dtable",))
