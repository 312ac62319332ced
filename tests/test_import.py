"""What the package needs of torch to be imported and asked for sizes (CPU)."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_getCurrent")]:
    delattr(torch._C, name)
import invariant_token_logprobs_lm_amd as itl
assert itl.lmhead_workspace_bytes(4, 1000) > 0 and itl.cross_entropy_workspace_bytes(4, 64, 1000) > 0
assert "gfx950" in itl.build_info()
x = torch.zeros(4, 64)
try:
    itl.residual_norm(x, None, x[0])
except ValueError as e:
    print(e)
"""


def test_import_without_torchs_private_stream_query():
    """A torch built without it still serves the host-side entry points and checks."""
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True, timeout=110)
    assert r.returncode == 0, r.stderr
    assert "must be on a HIP device" in r.stdout
