"""Refusals of the layer operators (attention with a relative position bias, residual step, gated feed-forward): calls
that return before they touch a device, by the C entry points and by the Python functions."""
import pytest
import torch

from vision_transformer_windowed_b200 import _lib, ops

PTR = 4096  # an aligned address that no refused call reads


def status_of(call, *args):
    with pytest.raises(_lib.FswinError) as e:
        call(*args)
    return e.value.status


# ------------------------------------------------- attention with a relative position bias
def relbias_fwd(shape, n_buckets=225, buckets=0, **at):
    p = {**dict(q=PTR, k=PTR, v=PTR, table=PTR, buckets=buckets, n=n_buckets, o=PTR, lse=PTR), **at}
    return status_of(_lib.fs_winattn_relbias_fwd, _lib.make_shape(*shape), *p.values(), 0)


def relbias_bwd(shape, n_buckets=225, buckets=0, **at):
    p = {**dict(q=PTR, k=PTR, v=PTR, o=PTR, dout=PTR, lse=PTR, table=PTR, buckets=buckets, n=n_buckets, dq=PTR, dk=PTR,
                dv=PTR, dtable=PTR, ws=PTR, size=1 << 40), **at}
    return status_of(_lib.fs_winattn_relbias_bwd, _lib.make_shape(*shape), *p.values(), 0)


SHAPE = (1, 16, 16, 2, 32, 8, 4)


@pytest.mark.parametrize("shape", [(1, 16, 16, 2, 64, 8, 4), (1, 16, 16, 2, 32, 12, 0), (1, 7, 16, 2, 32, 8, 0),
                                   (1, 16, 16, 0, 32, 8, 0), (1, 16, 16, 2, 32, 8, 8), (-1, 16, 16, 2, 32, 8, 0)])
def test_relbias_shapes(shape):
    assert relbias_fwd(shape) == _lib.FS_ERR_SHAPE and relbias_bwd(shape) == _lib.FS_ERR_SHAPE
    assert _lib.fs_winattn_relbias_bwd_workspace_bytes(_lib.make_shape(*shape)) == 0


@pytest.mark.parametrize("n,buckets", [(224, 0), (226, 0), (0, PTR), (-1, PTR), ((1 << 20) + 1, PTR)])
def test_relbias_buckets(n, buckets):
    assert relbias_fwd(SHAPE, n, buckets) == _lib.FS_ERR_SHAPE and relbias_bwd(SHAPE, n, buckets) == _lib.FS_ERR_SHAPE


def test_relbias_pointers():
    for name in ("q", "k", "v", "table", "o"):
        assert relbias_fwd(SHAPE, **{name: 0}) == _lib.FS_ERR_NULL, name
    for name, at in (("q", 8), ("k", 8), ("v", 2), ("o", 8), ("table", 1), ("lse", 2)):
        assert relbias_fwd(SHAPE, **{name: PTR + at}) == _lib.FS_ERR_ALIGN, name
    assert relbias_fwd(SHAPE, buckets=PTR + 2) == _lib.FS_ERR_ALIGN
    for name in ("q", "k", "v", "o", "dout", "lse", "table", "dq", "dk", "dv", "dtable"):
        assert relbias_bwd(SHAPE, **{name: 0}) == _lib.FS_ERR_NULL, name
    for name, at in (("q", 8), ("dout", 8), ("dq", 8), ("dk", 4), ("dv", 2), ("dtable", 1), ("lse", 1)):
        assert relbias_bwd(SHAPE, **{name: PTR + at}) == _lib.FS_ERR_ALIGN, name


def test_relbias_workspace():
    need = _lib.fs_winattn_relbias_bwd_workspace_bytes(_lib.make_shape(*SHAPE))
    assert need > 0
    assert relbias_bwd(SHAPE, ws=0) == _lib.FS_ERR_WORKSPACE
    assert relbias_bwd(SHAPE, ws=PTR + 16) == _lib.FS_ERR_WORKSPACE
    assert relbias_bwd(SHAPE, size=need - 1) == _lib.FS_ERR_WORKSPACE


# ------------------------------------------------- residual step
def step_shape(samples=2, tokens=5, channels=96, f32=0, pre=1, post=0, eps=1e-5, p=0.0):
    return _lib.ResnormShape(samples, tokens, channels, f32, pre, post, eps, p)


def step_fwd(shape, **at):
    p = {**dict(x=PTR, f=PTR, gate=0, scale=0, post_w=0, post_b=0, pre_w=PTR, pre_b=PTR, rng=0, r=PTR, n=PTR), **at}
    return status_of(_lib.fs_resnorm_fwd, shape, *p.values(), 0)


def step_bwd(shape, **at):
    p = {**dict(dr=PTR, dn=PTR, r=PTR, f=PTR, gate=0, scale=0, post_w=0, post_b=0, pre_w=PTR, pre_b=PTR, rng=0, dx=PTR,
                df=PTR, dgate=0, dscale=0, dpost_w=0, dpost_b=0, dpre_w=PTR, dpre_b=PTR, ws=PTR, size=1 << 40), **at}
    return status_of(_lib.fs_resnorm_bwd, shape, *p.values(), 0)


@pytest.mark.parametrize("kw", [dict(samples=-1), dict(tokens=-1), dict(channels=0), dict(channels=8193), dict(f32=2),
                                dict(pre=3), dict(post=-1), dict(eps=-1.0), dict(eps=float("nan")),
                                dict(eps=float("inf")), dict(p=1.0), dict(p=-0.1), dict(p=float("nan")),
                                dict(samples=1 << 31), dict(samples=1 << 20, tokens=1 << 11)])
def test_step_shapes(kw):
    assert step_fwd(step_shape(**kw)) == _lib.FS_ERR_SHAPE and step_bwd(step_shape(**kw)) == _lib.FS_ERR_SHAPE
    assert _lib.fs_resnorm_bwd_workspace_bytes(step_shape(**kw)) == 0


def test_step_pointers():
    for name in ("x", "f", "r", "n"):
        assert step_fwd(step_shape(), **{name: 0}) == _lib.FS_ERR_NULL, name
    for name in ("r", "f", "dx", "df"):
        assert step_bwd(step_shape(), **{name: 0}) == _lib.FS_ERR_NULL, name
    assert step_fwd(step_shape(p=0.1)) == _lib.FS_ERR_NULL  # no generator
    assert step_bwd(step_shape(p=0.1)) == _lib.FS_ERR_NULL
    assert step_fwd(step_shape(p=0.1), rng=PTR + 4) == _lib.FS_ERR_ALIGN
    for name in ("x", "f", "r", "n", "scale", "pre_w"):
        assert step_fwd(step_shape(), **{name: PTR + 1}) == _lib.FS_ERR_ALIGN, name
    for name in ("x", "r", "gate", "pre_b"):
        assert step_fwd(step_shape(f32=1), **{name: PTR + 2}) == _lib.FS_ERR_ALIGN, name
    # parameters of a norm that is not there
    assert step_fwd(step_shape(post=0), post_w=PTR) == _lib.FS_ERR_SHAPE
    assert step_fwd(step_shape(pre=0)) == _lib.FS_ERR_SHAPE
    need = _lib.fs_resnorm_bwd_workspace_bytes(step_shape())
    for at in (dict(ws=0), dict(ws=PTR + 64), dict(size=need - 1)):
        assert step_bwd(step_shape(), **at) == _lib.FS_ERR_WORKSPACE


# ------------------------------------------------- gated feed-forward
def mlp_fwd(shape, **at):
    p = {**dict(x=PTR, w_gate=PTR, w_up=PTR, w_down=PTR, b_gate=0, b_up=0, b_down=0, y=PTR, ws=PTR, size=1 << 40), **at}
    return status_of(_lib.fs_gated_mlp_fwd, _lib.MlpShape(*shape), *p.values(), 0)


def mlp_bwd(shape, **at):
    p = {**dict(dy=PTR, x=PTR, w_gate=PTR, w_up=PTR, w_down=PTR, b_gate=0, b_up=0, dx=PTR, dw_gate=PTR, dw_up=PTR,
                dw_down=PTR, db_gate=0, db_up=0, db_down=0, ws=PTR, size=1 << 40), **at}
    return status_of(_lib.fs_gated_mlp_bwd, _lib.MlpShape(*shape), *p.values(), 0)


@pytest.mark.parametrize("shape", [(-1, 96, 256, 0), (0x7FFFFF01, 96, 256, 0), (4, 0, 256, 0), (4, 12, 256, 0),
                                   (4, 16392, 256, 0), (4, 96, 4, 0), (4, 96, 260, 0), (4, 96, 65544, 0),
                                   (4, 96, 256, 2), (4, 96, 256, -1)])
def test_mlp_shapes(shape):
    assert mlp_fwd(shape) == _lib.FS_ERR_SHAPE and mlp_bwd(shape) == _lib.FS_ERR_SHAPE
    assert _lib.fs_gated_mlp_fwd_workspace_bytes(_lib.MlpShape(*shape)) == 0
    assert _lib.fs_gated_mlp_bwd_workspace_bytes(_lib.MlpShape(*shape)) == 0


def test_mlp_pointers():
    shape = (4, 96, 256, 1)
    for name in ("x", "w_gate", "w_up", "w_down", "y"):
        assert mlp_fwd(shape, **{name: 0}) == _lib.FS_ERR_NULL, name
    for name in ("dy", "x", "w_gate", "w_up", "w_down", "dx", "dw_gate", "dw_up", "dw_down"):
        assert mlp_bwd(shape, **{name: 0}) == _lib.FS_ERR_NULL, name
    for name in ("x", "w_up", "b_down", "y"):
        assert mlp_fwd(shape, **{name: PTR + 8}) == _lib.FS_ERR_ALIGN, name
    for name in ("dy", "dx", "dw_down", "db_gate"):
        assert mlp_bwd(shape, **{name: PTR + 2}) == _lib.FS_ERR_ALIGN, name
    for call, need in ((mlp_fwd, _lib.fs_gated_mlp_fwd_workspace_bytes(_lib.MlpShape(*shape))),
                       (mlp_bwd, _lib.fs_gated_mlp_bwd_workspace_bytes(_lib.MlpShape(*shape)))):
        assert need > 0
        for at in (dict(ws=0), dict(ws=PTR + 128), dict(size=need - 1)):
            assert call(shape, **at) == _lib.FS_ERR_WORKSPACE


# ------------------------------------------------- Python
def test_host_tensors_are_refused():
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    q = z(1, 16, 16, 2, 32)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        ops.winattn_relbias_fwd(q, q, q, z(2, 225), 8, 0)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        ops.residual_norm_fwd(z(2, 5, 96), z(2, 5, 96))
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        ops.gated_mlp_fwd(z(2, 96), z(256, 96), z(256, 96), z(96, 256))
    with pytest.raises(ValueError, match="None, 'layer' or 'rms'"):
        ops.residual_norm_fwd(z(2, 5, 96), z(2, 5, 96), pre="batch")
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        ops.residual_norm_fwd(z(2, 5, 96).half(), z(2, 5, 96))
    with pytest.raises(ValueError, match="samples"):
        ops.residual_norm_fwd(z(96), z(96))
    with pytest.raises(ValueError, match="act must be"):
        ops.gated_mlp_fwd(z(2, 96), z(256, 96), z(256, 96), z(96, 256), act="relu")


def mlp_bwd_bytes(tokens, channels, hidden):
    return _lib.fs_gated_mlp_bwd_workspace_bytes(_lib.MlpShape(tokens, channels, hidden, 0))


@pytest.mark.parametrize("channels,hidden", [(8, 8), (96, 256), (1024, 4096), (4096, 16384), (16384, 65536)])
def test_mlp_workspace_of_few_tokens(channels, hidden):
    """Up to 384 tokens (a part has four blocks of 64 or more) are summed in one: h and its two gradients, and an fp32 copy of the gradients."""
    for tokens in (1, 64, 384):
        need = 6 * tokens * hidden + 12 * channels * hidden + 8 * (2 * hidden + channels)
        assert need <= mlp_bwd_bytes(tokens, channels, hidden) <= need + 9 * 256


@pytest.mark.parametrize("tokens", [449, 5000, 100000, 1 << 24])
@pytest.mark.parametrize("channels,hidden", [(96, 256), (384, 1024), (1536, 4096), (16384, 65536)])
def test_mlp_workspace_of_more_tokens(tokens, channels, hidden):
    """As many copies as there are parts, 16 at most; with weights that give every SM work, hardly more than one."""
    one = 12 * channels * hidden + 8 * (2 * hidden + channels)
    parts = (mlp_bwd_bytes(tokens, channels, hidden) - 6 * tokens * hidden) / one
    assert 1 <= parts <= (3 if channels * hidden >= 1 << 28 else 16) + 9 * 256 / one
