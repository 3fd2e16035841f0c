"""Pins of the gated feed-forward oracle: torch's activations, autograd and differences."""
import pytest
import torch

from oracle import mlp

NAMES = ("x", "w_gate", "w_up", "w_down", "b_gate", "b_up", "b_down")


def draw(T, C, F, bias, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    t = dict(x=n(T, C), w_gate=n(F, C) * C ** -0.5, w_up=n(F, C) * C ** -0.5, w_down=n(C, F) * F ** -0.5)
    return dict(t, **({"b_gate": n(F), "b_up": n(F), "b_down": n(C)} if bias else {})), n(T, C)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("bias", [False, True])
def test_equals_torch_and_autograd(act, bias):
    t, dy = draw(9, 16, 24, bias)
    out, err = mlp.full(**t, act=act, dy=dy)
    leaf = {k: v.clone().requires_grad_() for k, v in t.items()}
    L = torch.nn.functional.linear
    f = torch.nn.functional.silu if act == "silu" else torch.nn.functional.gelu
    y = L(f(L(leaf["x"], leaf["w_gate"], leaf.get("b_gate"))) * L(leaf["x"], leaf["w_up"], leaf.get("b_up")),
          leaf["w_down"], leaf.get("b_down"))
    assert torch.allclose(out["y"], y, atol=1e-12)
    for key, grad in zip(leaf, torch.autograd.grad(y, list(leaf.values()), dy)):
        assert torch.allclose(out["d" + key], grad, atol=1e-11), key
        assert (err["d" + key] >= 0).all()
    assert (out["db_gate"] is None) == (not bias)


def test_gradients_by_differences():
    t, dy = draw(4, 8, 8, True, seed=2)
    out, _ = mlp.full(**t, act="gelu", dy=dy)
    for key in NAMES:
        at = tuple(s // 2 for s in t[key].shape)
        f = []
        for sign in (1e-6, -1e-6):
            v = t[key].clone()
            v[at] += sign
            f.append((mlp.full(**{**t, key: v}, act="gelu")[0]["y"] * dy).sum())
        assert abs((f[0] - f[1]) / 2e-6 - out["d" + key][at]) < 1e-6, key
