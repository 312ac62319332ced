"""The bounds of the confident tokens' gradients tell a wrong target entry
from a right one (CPU, 64 bits): G with its target's entry left out, or
rounded before the -1 is taken off it, passes them for hardly any token."""

import pytest
import torch

import learner_refs as R
from test_gpu_confident_tokens import CASES, bounds, trained


@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,d,V", CASES)
def test_bounds_see_the_targets_entry(n, d, V, grad):
    H, W, y = trained(n, d, V, torch.bfloat16, n + V)
    want, bound, p, G = bounds(H, W, y, torch.bfloat16, grad)
    live = y >= 0
    assert float((p[live] > 1 - 2.0 ** -8).float().mean()) > 0.35
    lost = (G.abs()[:, None] * R.f64(W).abs()[y.long().clamp(min=0)] > bound["dH"]).any(1)
    assert bool(lost[live & (p < 1 - 1e-4)].all())
    if n > 128:  # (two rows lose less than fp32's own roundings do)
        early = (p.float().bfloat16().double() - p).abs() / int(live.sum())  # p rounded, then the exact -1
        seen = (early[:, None] * R.f64(W).abs()[y.long().clamp(min=0)] > bound["dH"]).any(1)
        assert float(seen[live].float().mean()) > 0.5
