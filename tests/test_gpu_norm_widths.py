"""The norms' forward at every count of groups that a thread holds (a width of
512 k columns per wavefront, 2048 k per workgroup of four), vectors and single
columns, at both ends of each."""

import pytest
import torch

import test_gpu_norm as N

pytestmark = pytest.mark.gpu

ONE = [512 * k for k in range(1, 9)]
FOUR = [2048 * k for k in range(3, 9)]
WIDTHS = sorted({w for b in ONE + FOUR for w in (b - 511, b - 504, b - 8, b - 1)} - {1}) + FOUR + [16385]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", WIDTHS)
def test_forward(cuda, d, dtype):
    N.test_forward(cuda, 5, d, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", FOUR + [b - k for b in ONE + FOUR for k in (384, 128)])
def test_forward_fp8(cuda, d, dtype):
    N.test_forward_fp8(cuda, 5, d, dtype)


@pytest.mark.parametrize("d", FOUR + [b - 8 for b in ONE])
def test_rows_do_not_depend_on_the_batch(cuda, d):
    N.test_rows_do_not_depend_on_the_batch(cuda, d)
