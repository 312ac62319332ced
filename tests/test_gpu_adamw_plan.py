"""What an AdamW plan holds and what may be done to it between steps: the
learning rate and the count by assignment, everything else fixed; tensors that
have moved; autograd's view of updated weights; states that share memory."""

import pytest
import torch

from helpers import same_bits

pytestmark = pytest.mark.gpu


def _itl():
    import invariant_token_logprobs_lm_amd as itl

    return itl


def _tensors(device, seed=3, sizes=(5000, 300), dtypes=(torch.bfloat16, torch.float32)):
    g = torch.Generator().manual_seed(seed)
    p = [(torch.randn(n, generator=g) * 0.1).to(t).to(device) for n, t in zip(sizes, dtypes)]
    return p, [torch.randn(n, generator=g).to(device) for n in sizes]


@pytest.mark.parametrize("default", [torch.bfloat16, torch.float16, torch.float64])
def test_rate_is_fp32_whatever_the_default_type(cuda, default):
    itl = _itl()
    p, g = _tensors(cuda)
    q, h = _tensors(cuda)
    want = itl.adamw_plan(q, h, lr=3e-4)
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        plan = itl.adamw_plan(p, g, lr=3e-4)
        assert plan.lr.dtype == torch.float32 and same_bits(plan.lr, want.lr)
        norm = itl.adamw_step(plan, max_norm=1.0)
    finally:
        torch.set_default_dtype(before)
    assert same_bits(norm, itl.adamw_step(want, max_norm=1.0))
    assert torch.equal(p[0], q[0]) and same_bits(p[1], q[1])
