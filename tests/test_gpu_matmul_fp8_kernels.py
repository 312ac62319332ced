"""Each kernel of the block-scaled product over more steps than its slots, rounds and
registers hold at once: some rows and columns against 64 bits, others against smaller
calls' bits; codes of NaN; operands and results past 2^31 elements.

Tolerances as in test_gpu_matmul_fp8.py.
"""

import pytest
import torch

import block_refs as B
import learner_refs as R
from helpers import say

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]

LONG = [
    (16, 70000, 1024), (33, 60001, 640), (64, 50000, 8448),  # 128 x 64 tiles through three slots: 8, 5 and 66 steps
    (16, 4096, 16640), (16, 8000, 8448), (30, 8000, 8448),   # blocks shared by wavefronts: 3, 3 and 5 rounds
    (16, 9000, 4224), (5, 16384, 16640),                     # the same, 64 columns: 3 and 9 rounds
    (512, 2048, 8448), (1024, 2560, 8448),                   # 64 x 64 tiles, two steps per barrier and one
    (1024, 4000, 8448),                                      # 64 x 128 tiles (bf16)
    (128, 40000, 8448), (2048, 4096, 8448),                  # 128 x 128 tiles (bf16; fp32)
    (4096, 4096, 8448),                                      # 256 x 256 tiles
]


@pytest.fixture(scope="module")
def itl():
    import invariant_token_logprobs_lm_amd as itl

    return itl


def _bits(t):
    return t.contiguous().view(torch.uint8)


def _codes(n, k, seed, device):
    """Codes of either sign, none of them NaN (the lowest bit of the exponent is 0)."""
    g = torch.Generator(device=device).manual_seed(seed)
    return torch.randint(0, 256, (n, k), generator=g, device=device, dtype=torch.uint8).bitwise_and_(0xF7)


def _operands(m, n, k, device):
    g = torch.Generator(device=device).manual_seed(m + n + k)
    scale = lambda *s: torch.rand(*s, generator=g, device=device) + 0.5
    return _codes(m, k, m, device), scale(k // 128, m), _codes(n, k, n + 1, device), scale(-(-n // 128), k // 128)


def _check_some(out, ops, rows):
    """Those rows at the columns of the first, the middle and the last of B's tiles, against 64 bits."""
    a, sa, b, sb = ops
    n, tiles = b.shape[0], sb.shape[0]
    some = sorted({0, tiles // 2, tiles - 1})
    cols = torch.cat([torch.arange(t * 128, min(n, t * 128 + 128)) for t in some]).to(b.device)
    rows = torch.tensor(rows, device=b.device)
    want, mag = B.product(a[rows], sa[:, rows].contiguous(), b[cols], sb[torch.tensor(some, device=b.device)])
    off = (R.f64(out[rows][:, cols]) - want).abs()
    bound = (256 + sa.shape[0] + 3) * R.EPS24 * mag
    if out.dtype == torch.bfloat16:
        bound += R.half_step(torch.bfloat16) * want.abs() + 7 * 2.0 ** -13 * mag
        assert float(off.norm()) <= 2.0 ** -8 * float(want.norm())
    assert bool((off <= bound).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", LONG)
def test_long_contractions(cuda, itl, m, n, k, dtype):
    say("long", m, n, k, dtype)
    a, sa, b, sb = ops = _operands(m, n, k, cuda)
    out = itl.matmul_fp8_blocks(*ops, out_dtype=dtype)
    _check_some(out, ops, sorted({0, m // 3, m // 2, m - 1}))
    for i, some in ((0, 1), (m // 2, min(20, m - m // 2)), (m - 1, 1)):
        got = itl.matmul_fp8_blocks(a[i:i + some], sa[:, i:i + some].contiguous(), b, sb, out_dtype=dtype)
        assert torch.equal(_bits(got), _bits(out[i:i + some])), i
    for t, some in ((0, 1), (n // 256, 5), ((n - 1) // 128, 1)):
        got = itl.matmul_fp8_blocks(a, sa, b[128 * t:128 * (t + some)], sb[t:t + some], out_dtype=dtype)
        assert torch.equal(_bits(got), _bits(out[:, 128 * t:128 * (t + some)])), t


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [(20, 130, 256), (16, 9000, 384), (300, 1001, 256), (33, 60001, 384), (128, 40000, 256),
                                   (900, 5000, 256), (2100, 4100, 384), (4096, 4096, 384)])
def test_codes_of_nan_stay_in_their_row_and_column(cuda, itl, m, n, k, dtype):
    say("nan", m, n, k, dtype)
    a, sa, b, sb = _operands(m, n, k, cuda)
    want = itl.matmul_fp8_blocks(a, sa, b, sb, out_dtype=dtype)
    rows, cols = sorted({0, m // 2 + 1, m - 1}), sorted({1, n // 2, n - 1})
    hit = torch.zeros(m, n, dtype=torch.bool, device=cuda)
    for at, i in enumerate(rows):
        a[i, (at * 131) % k] = 0x7F if at % 2 else 0xFF
        hit[i] = True
    for at, j in enumerate(cols):
        b[j, (at * 77 + 5) % k] = 0xFF if at % 2 else 0x7F
        hit[:, j] = True
    got = itl.matmul_fp8_blocks(a, sa, b, sb, out_dtype=dtype)
    assert torch.equal(torch.isnan(got), hit)
    assert torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k", [128, 384])
@pytest.mark.parametrize("long_rows", [True, False])
def test_more_than_2_to_the_31_elements(cuda, itl, k, long_rows, dtype):
    """An operand and C both past 2^31 elements (and 2^32 bytes), along either of C's sides."""
    far = (1 << 24) + 1000
    m, n = (far, 130) if long_rows else (130, far)
    say("large", m, n, k, dtype)
    a, sa, b, sb = ops = _operands(m, n, k, cuda)
    out = itl.matmul_fp8_blocks(*ops, out_dtype=dtype)
    _check_some(out, ops, [0, 1, m // 2, m - 2, m - 1])
    # (along C's rows: where the operand's and C's offsets pass 31 and 32 bits)
    ends = [(1 << 31) // k, (1 << 32) // k, (1 << 31) // 130, (1 << 32) // (130 * out.element_size()), far]
    for end in (e for e in ends if e <= far):
        i = max(0, end - 400) // 128 * 128
        some = min(600, far - i)
        if long_rows:
            got = itl.matmul_fp8_blocks(a[i:i + some], sa[:, i:i + some].contiguous(), b, sb, out_dtype=dtype)
            assert torch.equal(_bits(got), _bits(out[i:i + some])), i
        else:
            got = itl.matmul_fp8_blocks(a, sa, b[i:i + some], sb[i // 128:i // 128 - (-some // 128)], out_dtype=dtype)
            assert torch.equal(_bits(got), _bits(out[:, i:i + some])), i
