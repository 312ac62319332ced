"""Calls whose kernels would need 2^32 threads in one grid dimension, where a
launch wraps without an error, are refused before anything is launched (CPU)."""

import ctypes

import pytest

UNSUPPORTED = 2
MB = 1 << 20
v = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    import invariant_token_logprobs_lm_amd as itl

    return itl.lib


def _refused(lib, status):
    return status == UNSUPPORTED and "too large" in lib.itl_last_error().decode()


# a workgroup of 512 threads (MXFP4: 256) per 256 tokens and slice group, and 16
# threads per token to merge the slices
@pytest.mark.parametrize("n,vocab", [(1 << 28, 200), (1 << 24, 151936)])
def test_forwards(lib, n, vocab):
    huge, p = 1 << 62, [v((i + 1) * MB) for i in range(9)]
    assert _refused(lib, lib.itl_lmhead_logprob(p[0], p[1], 0, n, 64, vocab, p[2], p[3], None, p[4], huge, None))
    assert _refused(lib, lib.itl_lmhead_logprob_keep_logits(p[0], p[1], 0, n, 64, vocab, p[2], p[3], None, p[5], 1 << 20, p[4],
                                                            huge, None))
    assert _refused(lib, lib.itl_lmhead_logprob_fp8(p[0], p[1], p[2], p[3], n, 128, vocab, p[4], p[5], None, p[6], huge, None))
    n *= 2 if vocab > 200 else 1
    assert _refused(lib, lib.itl_lmhead_logprob_mxfp4(p[0], p[1], p[2], p[3], n, 128, vocab, p[4], p[5], None, p[6], huge, None))


def test_quantized_rows(lib):
    p = [v((i + 1) * MB) for i in range(3)]
    assert lib.itl_quantize_rows_fp8(p[0], 0, 1 << 26, 128, p[1], p[2], None) == UNSUPPORTED
    assert lib.itl_quantize_rows_mxfp4(p[0], 0, 1 << 30, 128, p[1], p[2], None) == UNSUPPORTED
