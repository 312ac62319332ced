"""Calls of more rows or tokens than a launch of one workgroup (or wavefront) per
row has threads for in one dimension: 2^32."""

import pytest
import torch

from helpers import same_bits, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [1, 8])
def test_norm_of_rows_past_one_dimension(cuda, d):
    """A wavefront per row: 2^26 rows are 2^32 threads."""
    import invariant_token_logprobs_lm_amd as itl

    n = (1 << 26) + 5
    say("norm", n, d)
    x = torch.randn(n, d, device=cuda).bfloat16()
    w = torch.ones(d, dtype=torch.bfloat16, device=cuda)
    y = x.flip(0).contiguous()
    u = torch.full_like(x, float("nan"))
    h, u, r, _ = itl.residual_norm(x, y, w, u=u)
    for rows in (slice(0, 1000), slice((1 << 25) - 7, (1 << 25) + 900), slice(n - 1003, n)):
        h1, u1, r1, _ = itl.residual_norm(x[rows], y[rows], w)
        assert torch.equal(h[rows], h1) and torch.equal(u[rows], u1) and same_bits(r[rows], r1)
    assert bool(u.isfinite().all()) and bool(r.isfinite().all())
