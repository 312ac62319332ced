"""The 64-bit forms of the learner's operators against central differences of
their own forward, and hand-worked values (CPU)."""

import math

import pytest
import torch

import learner_refs as R


def _central(f, x, i, h=1e-6):
    a, b = x.clone(), x.clone()
    a.view(-1)[i] += h
    b.view(-1)[i] -= h
    return (f(a) - f(b)) / (2 * h)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate_dim", [0, 1, 2])
def test_norm_backward_is_the_forwards_derivative(post, gate_dim):
    g = torch.Generator().manual_seed(3 + post * 5 + gate_dim)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    n, d, scale = 4, 7, 0.6
    t = {"x": r(n, d), "y": r(n, d), "w_pre": r(d), "w_post": r(d) if post else None,
         "gate": None if gate_dim == 0 else r(d) if gate_dim == 1 else r(n, d)}
    cu, ch = r(n, d), r(n, d)

    def objective(**change):
        a = {**t, **change}
        h, _, _ = R.norm_forward(a["x"], a["y"], a["w_pre"], a["w_post"], a["gate"], scale)
        return float((R.norm_out(h, a["w_pre"])[0] * cu).sum() + (h * ch).sum())

    h, _, r_post = R.norm_forward(t["x"], t["y"], t["w_pre"], t["w_post"], t["gate"], scale)
    out, _ = R.norm_backward(cu, ch, h, t["y"], t["w_pre"], R.rms(h, 1e-6), t["w_post"], r_post, t["gate"], scale)
    for name, key in (("x", "dx"), ("y", "dy"), ("w_pre", "dw_pre"), ("w_post", "dw_post"), ("gate", "dgate")):
        if t[name] is None:
            continue
        for i in range(0, t[name].numel(), 3):
            want = _central(lambda v: objective(**{name: v}), t[name], i)
            assert abs(float(out[key].reshape(-1)[i]) - want) < 1e-6 * (1 + abs(want)), (key, i)


@pytest.mark.parametrize("smoothing,z_weight,mean", [(0.0, 0.0, True), (0.1, 0.0, True), (0.2, 0.05, False)])
def test_cross_entropy_gradient_is_the_losss_derivative(smoothing, z_weight, mean):
    g = torch.Generator().manual_seed(9)
    H = torch.randn(5, 6, generator=g, dtype=torch.float64)
    W = torch.randn(11, 6, generator=g, dtype=torch.float64)
    y = torch.tensor([3, -100, 10, 0, 11])
    kw = dict(smoothing=smoothing, z_weight=z_weight, mean=mean)
    out = R.cross_entropy(H, W, y, grad_scale=1.5, **kw)
    for i in range(H.numel()):
        want = 1.5 * _central(lambda v: float(R.cross_entropy(v, W, y, **kw)["loss"]), H, i)
        assert abs(float(out["dH"].view(-1)[i]) - want) < 1e-7
    for i in range(0, W.numel(), 4):
        want = 1.5 * _central(lambda v: float(R.cross_entropy(H, v, y, **kw)["loss"]), W, i)
        assert abs(float(out["dW"].view(-1)[i]) - want) < 1e-7
    assert out["token_loss"][1] == 0 and out["token_loss"][4] == 0


def test_cross_entropy_of_even_logits():
    W = torch.ones(8, 4, dtype=torch.float64)
    out = R.cross_entropy(torch.ones(2, 4, dtype=torch.float64), W, torch.tensor([0, 5]), smoothing=0.3)
    assert abs(float(out["loss"]) - math.log(8)) < 1e-12


def test_adamw_first_step_by_hand():
    """From zero states the first step moves every weight by lr (its sign), beside the decay."""
    w = torch.tensor([1.0, -2.0], dtype=torch.float64)
    g = torch.tensor([0.5, -4.0], dtype=torch.float64)
    z = torch.zeros(2, dtype=torch.float64)
    nw, m, v = R.adamw(w, g, z, z, 1, 0.1, 0.01, (0.9, 0.99), 1e-12)
    assert torch.allclose(nw, w * (1 - 0.001) - 0.1 * torch.sign(g), atol=1e-9)
    assert torch.allclose(m, 0.1 * g) and torch.allclose(v, 0.01 * g * g)
