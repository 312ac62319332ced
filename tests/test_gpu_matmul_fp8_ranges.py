"""The block-scaled product where its scales' product is at the ends of fp32's range,
for each of its kernels.

Tolerances. The scales' product s is rounded to fp32: by half a step of itself (within the
chain's bound, as in test_gpu_matmul_fp8.py) from 2^-126 on, below by at most 2^-150; a
block's sum is at most 128 448^2 < 2^25, so that is 2^-125 of C a block. A multiply-add
whose result is subnormal rounds by at most 2^-150, one a block; bf16 results that are
subnormal by half of bf16's least step, 2^-134.
"""

import pytest
import torch

import block_refs as B
import learner_refs as R
from helpers import say

pytestmark = pytest.mark.gpu

# few tiles whose wavefronts share the blocks; 64 x 64 tiles; bf16 256 x 256, fp32 128 x 128; fp32 256 x 256
SIZES = [(16, 300, 1024), (300, 1001, 1024), (2100, 4100, 384), (4096, 4096, 384)]


@pytest.fixture(scope="module")
def itl():
    import invariant_token_logprobs_lm_amd as itl

    return itl


def _codes(n, k, g, top):
    """Codes of either sign below `top`."""
    return (torch.randint(0, top, (n, k), generator=g) + 128 * torch.randint(0, 2, (n, k), generator=g)).to(torch.uint8)


def _scales(shape, g, low):
    return (low * (1 + torch.rand(shape, generator=g, dtype=torch.float64))).float()


def _off(itl, cuda, m, n, k, dtype, low_a, low_b, top):
    g = torch.Generator().manual_seed(m + n + k)
    ops = (_codes(m, k, g, top), _scales((k // 128, m), g, low_a), _codes(n, k, g, top), _scales((-(-n // 128), k // 128), g, low_b))
    got = itl.matmul_fp8_blocks(*(t.to(cuda) for t in ops), out_dtype=dtype)
    want, mag = B.product(*ops)
    blocks = k // 128
    bound = (256 + blocks + 3) * R.EPS24 * mag + blocks * 2.0 ** -150
    if dtype == torch.bfloat16:
        bound += R.half_step(dtype) * want.abs() + 7 * 2.0 ** -13 * mag + 2.0 ** -134
    return got, (R.f64(got) - want).abs(), bound


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_scales_whose_product_is_just_normal(cuda, itl, m, n, k, dtype):
    say("normal", m, n, k, dtype)
    _, off, bound = _off(itl, cuda, m, n, k, dtype, 2.0 ** -100, 2.0 ** -26, 0x7F)
    assert bool((off <= bound).all())
    # and just below the largest number, with codes of at most 2^-6
    got, off, bound = _off(itl, cuda, m, n, k, dtype, 2.0 ** 99, 2.0 ** 26, 0x08)
    assert bool(torch.isfinite(got).all()) and bool((off <= bound).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("low_a,low_b", [(2.0 ** -125, 2.0 ** -15), (2.0 ** -126, 2.0 ** -30), (2.0 ** -100, 2.0 ** -27)])
def test_scales_whose_product_is_subnormal(cuda, itl, m, n, k, dtype, low_a, low_b):
    say("subnormal", m, n, k, dtype, low_a, low_b)
    got, off, bound = _off(itl, cuda, m, n, k, dtype, low_a, low_b, 0x7F)
    assert bool((off <= bound + k // 128 * 2.0 ** -125).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_have_one_value_where_the_product_is_subnormal(cuda, itl, dtype):
    g = torch.Generator().manual_seed(1)
    m, n, k = 2100, 4100, 384
    a, sa, b, sb = (t.to(cuda) for t in (_codes(m, k, g, 0x7F), _scales((k // 128, m), g, 2.0 ** -125),
                                         _codes(n, k, g, 0x7F), _scales((-(-n // 128), k // 128), g, 2.0 ** -15)))
    whole = itl.matmul_fp8_blocks(a, sa, b, sb, out_dtype=dtype)
    for i, some in ((0, 1), (40, 16), (77, 100), (1000, 700)):
        got = itl.matmul_fp8_blocks(a[i:i + some].contiguous(), sa[:, i:i + some].contiguous(), b, sb, out_dtype=dtype)
        assert torch.equal(got, whole[i:i + some]), i
