"""The cross entropy's gradient where a trained model has it: targets of
probability 0.9 to 0.9999, whose entries of G (p - 1) are small beside the
parts they are made of. Every type of gradient, few tokens and many.

Bounds, from the arithmetic, per token, in units of u = grad_scale / N (EPS is
half a step of fp32, a = 1 + 2 lam lse, c = e / V):
* logits off by at most dz = (d / 16 + 8) EPS max_v sum |H W| move a probability
  by at most 2 dz p (1 - p) (first order; 2.1 below covers the rest);
* p itself is off by r = (3 (|z| + |lse|) + V / 256 + 96) EPS of itself: z and
  lse in units of log 2, their difference and lse's own rounding, and one step
  per tile or partial of the sum of exponentials once it is near its value;
* G's entries of a bf16 head are held to half a step of bf16, 2^-8 (calls of
  at most 128 tokens: two such rows, 2^-16); with fp32 gradients the target's
  to a few steps of fp32, as the documentation has it;
* the contractions add half a step of fp32 per addition, the results half a
  step of their type.

The last case is more than one chunk of tokens.
"""

import pytest
import torch

import learner_refs as R
from helpers import say

pytestmark = pytest.mark.gpu


def trained(n, d, V, dtype, seed):
    """A head that is sure of most targets, by margins spread over the tokens."""
    g = torch.Generator().manual_seed(seed)
    W = (0.1 * torch.randn(V, d, generator=g)).to(dtype)
    y = torch.randint(0, V, (n,), generator=g, dtype=torch.int32)
    gain = torch.linspace(11.0, 18.5, n)[torch.randperm(n, generator=g)] / (0.01 * d)
    H = (W[y.long()].float() * gain[:, None] + 0.5 * torch.randn(n, d, generator=g)).to(dtype)
    y[5::97] = -100
    return H, W, y


def bounds(H, W, y, dtype, grad_dtype, smoothing=0.0, z_weight=0.0):
    """(want, {"dH", "dW"} bounds), in 64 bits."""
    n, d, V = len(H), H.shape[1], len(W)
    h, w, t = R.f64(H), R.f64(W), y.long()
    want = R.cross_entropy(h, w, y, smoothing=smoothing, z_weight=z_weight)
    live = t >= 0
    rows, at = torch.arange(n), t.clamp(min=0)
    z = h @ w.t()
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    a = 1 + 2 * z_weight * lse
    dz = 2.1 * (d / 16 + 8) * R.EPS24 * want["mag_z"]
    r = (3 * (z.abs().amax(1) + lse.abs()) + V / 256 + 96) * R.EPS24
    off = (a[:, None] * p) * (dz[:, None] * (1 - p) + r[:, None])
    G = a[:, None] * p - smoothing / V
    G[rows, at] -= 1 - smoothing
    held = 0.0 if dtype == torch.float32 else 2.0 ** -16 if n <= 128 else R.half_step(dtype)
    held = torch.full_like(G, held)
    if grad_dtype == torch.float32:
        held[rows, at] = 0.0
    off = off + (held + 8 * R.EPS24) * G.abs()
    off, G = off * live[:, None] / int(live.sum()), G * live[:, None] / int(live.sum())
    bound = {"dH": off @ w.abs() + V * R.EPS24 * (G.abs() @ w.abs()),
             "dW": off.t() @ h.abs() + (n + 64) * R.EPS24 * (G.abs().t() @ h.abs())}
    return want, {k: b + R.half_step(grad_dtype) * want[k].abs() for k, b in bound.items()}, p[rows, at], G[rows, at]


CASES = [(80, 256, 4000), (129, 128, 700), (400, 256, 4000), (1500, 256, 4000), (1500, 64, 300), (16684, 64, 300)]
TYPES = [(torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32)]


@pytest.mark.parametrize("kw", [{}, {"smoothing": 0.05, "z_weight": 1e-4}])
@pytest.mark.parametrize("dtype,grad", TYPES)
@pytest.mark.parametrize("n,d,V", CASES)
def test_confident_targets(cuda, n, d, V, dtype, grad, kw):
    import invariant_token_logprobs_lm_amd as itl

    say("confident", n, d, V, dtype, grad, kw)
    H, W, y = trained(n, d, V, dtype, n + V)
    want, bound, _, _ = bounds(H, W, y, dtype, grad, **kw)
    _, _, _, dH, dW = itl.cross_entropy_grad(H.to(cuda), W.to(cuda), y.to(cuda), grad_dtype=grad,
                                             label_smoothing=kw.get("smoothing", 0.0), z_weight=kw.get("z_weight", 0.0))
    for name, got in (("dH", dH), ("dW", dW)):
        assert bool(((R.f64(got) - want[name]).abs() <= bound[name]).all()), name
