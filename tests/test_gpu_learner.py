"""The learner's operators together, as one training step runs them: the norms
around the last block make the head's input, the loss (cross entropy, or the
REINFORCE Zero loss on the sampled logprobs) and its gradient go back through
the head and the norms, and one AdamW step updates the weights. Checked against
the same step in 64 bits, eagerly and as a replayed graph; then that a rollout's
FP8 rows come from the same norm.

Tolerance: with fp32 weights and activations each of the three gradients is
within 1e-4 of its norm of the 64-bit one (d + V + n additions of one half step
each, 2^-24, on sums whose terms are at most ten times the result: below 3e-5 at
these sizes); a weight then differs by at most what AdamW's first step makes of
it, which depends on a gradient's sign alone where it is not tiny, so states
are compared, and weights through the states.
"""

import pytest
import torch

import learner_refs as R
from helpers import same_bits

pytestmark = pytest.mark.gpu


def _model(n, d, V, dtype, device, seed=3):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    t = {"x": r(n, d), "y": r(n, d), "w_pre": 1 + 0.1 * r(d), "w_post": 1 + 0.1 * r(d), "gate": 0.5 + 0.1 * r(d),
         "W": 0.05 * r(V, d)}
    t = {k: v.to(dtype).to(device) for k, v in t.items()}
    y = torch.randint(0, V, (n,), generator=g, dtype=torch.int32)
    y[: n // 4] = -100
    return t, y.to(device)


class _Step:
    """One supervised step over the final norms and the head, gradients in place."""

    def __init__(self, itl, t, y, state_bits):
        self.itl, self.t, self.y = itl, t, y
        names = ("W", "w_pre", "w_post", "gate")
        self.grads = {k: torch.zeros(t[k].shape, dtype=torch.float32, device=y.device) for k in names}
        self.plan = itl.adamw_plan([t[k] for k in names], [self.grads[k] for k in names], lr=1e-3, weight_decay=0.01,
                                   state_bits=state_bits)
        self.kw = {"w_post": t["w_post"], "gate": t["gate"], "scale": 0.5}

    def __call__(self):
        itl, t = self.itl, self.t
        h, u, r_pre, r_post = itl.residual_norm(t["x"], t["y"], t["w_pre"], **self.kw)
        loss, _, _, dH, _ = itl.cross_entropy_grad(u, t["W"], self.y, z_weight=1e-4, dW=self.grads["W"])
        dx, dy, dw_pre, dw_post, dgate = itl.residual_norm_backward(dH, None, h, t["y"], t["w_pre"], r_pre,
                                                                    rstd_post=r_post, **self.kw)
        for k, g in (("w_pre", dw_pre), ("w_post", dw_post), ("gate", dgate)):
            self.grads[k].copy_(g)
        norm = itl.adamw_step(self.plan, max_norm=1.0)
        return loss, dx, dy, norm


def _reference(t, y):
    c = {k: R.f64(v) for k, v in t.items()}
    h, _, r_post = R.norm_forward(c["x"], c["y"], c["w_pre"], c["w_post"], c["gate"], 0.5)
    u, r_pre = R.norm_out(h, c["w_pre"])
    ce = R.cross_entropy(u, c["W"], y, z_weight=1e-4)
    out, _ = R.norm_backward(ce["dH"], None, h, c["y"], c["w_pre"], r_pre, c["w_post"], r_post, c["gate"], 0.5)
    grads = {"W": ce["dW"], "w_pre": out["dw_pre"], "w_post": out["dw_post"], "gate": out["dgate"]}
    return float(ce["loss"]), out, grads


def _near(got, want, rel):
    got, want = R.f64(got), want
    assert float((got - want).norm()) <= rel * float(want.norm())


def test_step_against_64_bits(cuda):
    import invariant_token_logprobs_lm_amd as itl

    t, y = _model(300, 192, 2000, torch.float32, cuda)
    loss, out, grads = _reference(t, y)
    before = {k: R.f64(v) for k, v in t.items()}
    step = _Step(itl, t, y, 32)
    got, dx, dy, norm = step()
    assert abs(float(got) - loss) <= 1e-5 * loss
    _near(dx, out["dx"], 1e-4)
    _near(dy, out["dy"], 1e-4)
    for k, g in grads.items():
        _near(step.grads[k].view(g.shape), g, 1e-4)
    want_norm = float(torch.sqrt(sum((g ** 2).sum() for g in grads.values())))
    assert abs(float(norm) - want_norm) <= 1e-4 * want_norm
    clip = min(1.0, 1.0 / (want_norm + 1e-6))
    lr = float(step.plan.lr)
    for i, k in enumerate(("W", "w_pre", "w_post", "gate")):
        n, o = t[k].numel(), step.plan.offsets[i]
        m = step.plan.exp_avg[o:o + n]
        _near(m, 0.1 * clip * grads[k].reshape(-1), 2e-4)
        # the weights follow from the states the step left
        v = R.f64(step.plan.exp_avg_sq[o:o + n])
        w = before[k].reshape(-1) * (1 - lr * 0.01) - lr / 0.1 * R.f64(m) / (torch.sqrt(v) / (1 - 0.999) ** 0.5 + 1e-8)
        assert bool(((R.f64(t[k]).reshape(-1) - w).abs() <= 64 * R.EPS24 * (before[k].reshape(-1).abs() + lr * 4)).all())


@pytest.mark.parametrize("dtype,bits", [(torch.float32, 32), (torch.bfloat16, 32), (torch.bfloat16, 8)])
def test_captured_step_replays_like_the_eager_one(cuda, dtype, bits):
    import invariant_token_logprobs_lm_amd as itl

    (te, y), (tc, _) = _model(200, 128, 1500, dtype, cuda), _model(200, 128, 1500, dtype, cuda)
    eager, captured = _Step(itl, te, y, bits), _Step(itl, tc, y, bits)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = captured()
    for rep in range(4):
        want = eager()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, out):
            assert torch.equal(a, b), rep
        for k in ("W", "w_pre", "w_post", "gate"):
            assert torch.equal(te[k], tc[k]), (rep, k)
    assert int(captured.plan.step) == 4
    assert float(out[0]) == float(want[0])


def test_reinforce_gradient_through_the_norm(cuda):
    """The sampled logprobs' loss goes back through head and norm as the supervised one does."""
    import invariant_token_logprobs_lm_amd as itl

    n, d, V = 96, 128, 700
    t, y = _model(n, d, V, torch.float32, cuda)
    y = torch.where(y < 0, torch.zeros_like(y), y)
    h, u, r_pre, _ = itl.residual_norm(t["x"], t["y"], t["w_pre"])
    lp, lse = itl.lmhead_logprob(u, t["W"], y)
    offsets = torch.tensor([0, 40, n], dtype=torch.int64, device=cuda)
    adv = torch.tensor([1.0, -0.5], device=cuda)
    _, _, coef = itl.reinforce_zero_loss(lp, lp, adv, offsets)
    dH, dW = itl.reinforce_zero_backward(u, t["W"], y, lse, coef)
    dx, dy, dw, _, _ = itl.residual_norm_backward(dH, None, h, t["y"], t["w_pre"], r_pre)
    c = {k: R.f64(v) for k, v in t.items()}
    h64, _, _ = R.norm_forward(c["x"], c["y"], c["w_pre"])
    u64, r64 = R.norm_out(h64, c["w_pre"])
    p = torch.softmax(u64 @ c["W"].t(), 1)
    G = R.f64(coef)[:, None] * (torch.nn.functional.one_hot(y.cpu().long(), V) - p)
    out, _ = R.norm_backward(G @ c["W"], None, h64, c["y"], c["w_pre"], r64)
    _near(dx, out["dx"], 1e-4)
    _near(dy, out["dy"], 1e-4)
    _near(dw, out["dw_pre"], 1e-4)


def test_fp8_rows_for_the_rollout(cuda):
    """The FP8 head on the norm's codes: within the format's error of the full-precision logprob, and a
    row's logprob does not depend on its batch through both calls."""
    import invariant_token_logprobs_lm_amd as itl

    n, d, V = 150, 256, 3000
    t, y = _model(n, d, V, torch.bfloat16, cuda)
    y = torch.where(y < 0, torch.zeros_like(y), y)
    Wq, ws = itl.quantize_rows_fp8(t["W"])
    _, Uq, us, _, _ = itl.residual_norm_fp8(t["x"], t["y"], t["w_pre"])
    lp, _ = itl.lmhead_logprob_fp8(Uq, us, Wq, ws, y)
    _, u, _, _ = itl.residual_norm(t["x"], t["y"], t["w_pre"])
    full, _ = itl.lmhead_logprob(u, t["W"], y)
    # a logit of d products, each off by at most 2 * 2^-4 of itself with independent signs: 6 standard deviations
    sigma = 2.0 ** -4 * (R.f64(u) ** 2 @ (R.f64(t["W"]) ** 2).t()).sqrt().amax(1)
    assert bool(((R.f64(lp) - R.f64(full)).abs() <= 12 * sigma).all())
    one = slice(77, 78)
    _, Uq1, us1, _, _ = itl.residual_norm_fp8(t["x"][one], t["y"][one], t["w_pre"])
    lp1, _ = itl.lmhead_logprob_fp8(Uq1, us1, Wq, ws, y[one])
    assert torch.equal(Uq1, Uq[one]) and same_bits(us1, us[one]) and same_bits(lp1, lp[one])
