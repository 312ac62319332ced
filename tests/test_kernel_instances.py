"""The cross entropy's compiled kernels are those that its calls launch: one
instance per case of dtype and mode that exists, read from the library's own
symbols (CPU)."""

import re
import shutil
import subprocess

import pytest

# <dtype, ...>: 0 bf16, 1 fp32. Modes of dW: 0 rounded to bf16, 1 written in
# fp32, 2 added to fp32, 3 partial sums.
INSTANCES = {
    "ce_partial_kernel": {"0, false, false", "0, false, true", "0, true, false", "0, true, true"},
    "ce_partial_narrow_kernel": {"0, false, 64", "0, true, 64"},
    "ce_lse_f32_kernel": {"false", "true"},
    "ce_colsum_kernel": {"0", "1"},
    "ce_token_loss_kernel": {"0", "1"},
    "ce_grad_logits_kernel": {"0", "1"},
    "ce_dh_kernel": {"0", "1"},
    "ce_dh_finish_kernel": {"0", "1"},
    # bf16: 16-bit results, fp32 sums over several chunks, fp32 results on the targets' rests
    "ce_dw_kernel": {"0, 0", "0, 1", "0, 2", "0, 3", "1, 1", "1, 2", "1, 3"},
    # (calls of few tokens are one chunk)
    "ce_dw_few_kernel": {"0", "2"},
    "ce_dw_finish_kernel": {"0", "1", "2"},
}


@pytest.mark.skipif(shutil.which("nm") is None, reason="needs nm")
def test_no_instance_without_a_call():
    from invariant_token_logprobs_lm_amd import LIB_PATH

    out = subprocess.run(["nm", "-C", LIB_PATH], capture_output=True, text=True, check=True).stdout
    seen = {}
    for name, args in re.findall(r"__device_stub__(ce_\w+)<([^>]*)>\(", out):
        seen.setdefault(name, set()).add(args)
    assert seen == INSTANCES
