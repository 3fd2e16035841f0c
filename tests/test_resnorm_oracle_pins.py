"""Pins of the residual step's oracle: torch's own norms, autograd, differences, and the generator's published vectors."""
import pytest
import torch

from oracle import resnorm


def test_philox_known_answers():
    """Known-answer vectors of Philox4x32-10 published with the Random123 library."""
    f = 0xFFFFFFFF
    assert resnorm.philox4x32((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert resnorm.philox4x32((f, f, f, f), (f, f)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert resnorm.philox4x32((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def draw(B, T, C, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    return dict(x=n(B, T, C), f=n(B, T, C), gate=n(B), scale=n(C), post_weight=n(C), post_bias=n(C), pre_weight=n(C),
                pre_bias=n(C)), n(B, T, C), n(B, T, C)


@pytest.mark.parametrize("pre", [None, "layer", "rms"])
@pytest.mark.parametrize("post", [None, "layer", "rms"])
def test_equals_torch_norms_and_autograd(pre, post):
    t, dr, dn = draw(3, 5, 12)
    for k, kind in (("pre", pre), ("post", post)):
        if kind is None:
            t[k + "_weight"] = t[k + "_bias"] = None
    rng = torch.tensor([5, 77])
    got = resnorm.step(**t, pre=pre, post=post, p=0.3, rng=rng, dr=dr, dn=dn if pre else None)
    leaf = {k: v.clone().requires_grad_() for k, v in t.items() if v is not None}

    def norm(v, kind, which):
        w, b = leaf[which + "_weight"], leaf[which + "_bias"]
        if kind == "layer":
            return torch.nn.functional.layer_norm(v, (12,), w, b, 1e-5)
        return torch.nn.functional.rms_norm(v, (12,), w, 1e-5) + b

    y = norm(leaf["f"], post, "post") if post else leaf["f"]
    y = y * resnorm.keep_mask(y.shape, 0.3, 5, 77) / 0.7 * leaf["scale"] * leaf["gate"][:, None, None]
    r = leaf["x"] + y
    n = norm(r, pre, "pre") if pre else None
    assert torch.allclose(got["r"], r, atol=1e-12)
    loss = (r * dr).sum() + ((n * dn).sum() if pre else 0)
    for key, grad in zip(leaf, torch.autograd.grad(loss, list(leaf.values()))):
        assert torch.allclose(got["d" + key], grad, atol=1e-11), key
    if pre:
        assert torch.allclose(got["n"], n, atol=1e-12)


def test_gradients_by_differences():
    t, dr, dn = draw(2, 3, 7, seed=4)
    kw = dict(pre="rms", post="layer", p=0.25, rng=torch.tensor([9, 1]))
    got = resnorm.step(**t, **kw, dr=dr, dn=dn)

    def loss(**over):
        o = resnorm.step(**{**t, **over}, **kw)
        return float((o["r"] * dr).sum() + (o["n"] * dn).sum())

    for key, v in t.items():
        at = tuple(s // 2 for s in v.shape)
        up, down = v.clone(), v.clone()
        up[at] += 1e-6
        down[at] -= 1e-6
        assert abs((loss(**{key: up}) - loss(**{key: down})) / 2e-6 - float(got["d" + key][at])) < 1e-6, key


def test_zero_gate_takes_nothing_from_its_branch():
    t, dr, dn = draw(2, 3, 8)
    t["gate"] = torch.tensor([0.0, 1.0], dtype=torch.float64)
    t["f"][0] = float("nan")
    got = resnorm.step(**t, pre="layer", post="layer", dr=dr, dn=dn)
    assert torch.equal(got["r"][0], t["x"][0]) and (got["df"][0] == 0).all()
    assert torch.isfinite(got["dscale"]).all() and torch.isfinite(got["dpost_weight"]).all()
