"""Calls of more rows or tokens than a launch of one workgroup (or wavefront) per
row has threads for in one dimension: 2^32. Rows are compared with those of
small calls, whose bits they share."""

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


@pytest.mark.parametrize("smoothing", [0.0, 0.1])
def test_loss_of_tokens_past_one_dimension(cuda, smoothing):
    """A workgroup per token gathers the counted rows (2^24 tokens are 2^32
    threads), a wavefront per token makes its loss with smoothing."""
    import invariant_token_logprobs_lm_amd as itl

    n, d, V = (1 << 24) + 700, 64, 300
    say("loss", n, smoothing)
    g = torch.Generator(device=cuda).manual_seed(5)
    H = torch.randn(n, d, generator=g, device=cuda, dtype=torch.bfloat16)
    W = (torch.randn(V, d, generator=g, device=cuda) * 0.1).bfloat16()
    y = torch.randint(-30, V, (n,), generator=g, device=cuda, dtype=torch.int32)
    loss, token, lse = itl.cross_entropy(H, W, y, label_smoothing=smoothing)
    for rows in (slice(0, 900), slice((1 << 23) - 400, (1 << 23) + 500), slice(n - 900, n)):
        _, t1, l1 = itl.cross_entropy(H[rows], W, y[rows], label_smoothing=smoothing)
        assert same_bits(token[rows], t1) and same_bits(lse[rows], l1)
    live = (y >= 0).sum()
    want = token.double().sum() / live
    assert abs(float(loss) - float(want)) <= 2.0 ** -23 * float(want)


def test_gradient_of_tokens_past_one_dimension(cuda):
    """dH's rows of tokens that do not count are cleared for every token of the call."""
    import invariant_token_logprobs_lm_amd as itl

    n, d, V = (1 << 24) + 700, 64, 300
    say("loss and gradient", n)
    g = torch.Generator(device=cuda).manual_seed(6)
    H = torch.randn(n, d, generator=g, device=cuda, dtype=torch.bfloat16)
    W = (torch.randn(V, d, generator=g, device=cuda) * 0.1).bfloat16()
    y = torch.full((n,), -100, dtype=torch.int32, device=cuda)
    few = torch.cat([torch.arange(0, 500), torch.arange((1 << 23) - 200, (1 << 23) + 200), torch.arange(n - 500, n)]).to(cuda)
    y[few] = torch.randint(0, V, (len(few),), generator=g, device=cuda, dtype=torch.int32)
    dH = torch.full((n, d), float("nan"), dtype=torch.bfloat16, device=cuda)
    _, token, _, _, dW = itl.cross_entropy_grad(H, W, y, reduction="sum", grad_dtype=torch.bfloat16, dH=dH)
    _, t1, _, dH1, dW1 = itl.cross_entropy_grad(H[few], W, y[few], reduction="sum", grad_dtype=torch.bfloat16)
    assert same_bits(token[few], t1)
    # the same products; the K splits and the tiles' sums go by the call's size
    assert float((dH[few].float() - dH1.float()).abs().max()) <= 2.0 ** -6 * float(dH1.float().abs().max())
    assert float((dW.float() - dW1.float()).abs().max()) <= 2.0 ** -6 * float(dW1.float().abs().max())
    y_out = torch.ones(n, dtype=torch.bool, device=cuda)
    y_out[few] = False
    assert not bool(dH[y_out].any())
