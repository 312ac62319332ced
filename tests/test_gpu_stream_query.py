"""Calls go to the caller's current stream, with torch's quick query of it and without."""

import pytest
import torch

from helpers import same_bits

pytestmark = pytest.mark.gpu


def test_both_queries_name_the_current_stream(cuda):
    import invariant_token_logprobs_lm_amd as itl

    side = torch.cuda.Stream(device=cuda)
    for stream in (torch.cuda.current_stream(cuda), side):
        with torch.cuda.stream(stream):
            assert itl._raw_stream(cuda.index) == itl._stream_handle(cuda.index) == stream.cuda_stream


def test_results_without_the_quick_query(cuda, monkeypatch):
    import invariant_token_logprobs_lm_amd as itl

    g = torch.Generator().manual_seed(1)
    H, W = torch.randn(70, 128, generator=g).to(cuda), torch.randn(500, 128, generator=g).to(cuda)
    y = torch.randint(0, 500, (70,), generator=g, dtype=torch.int32).to(cuda)
    w = torch.ones(128, device=cuda)
    call = lambda: itl.cross_entropy_grad(itl.residual_norm(H, None, w)[1], W, y) + itl.lmhead_logprob(H, W, y)
    want = call()
    monkeypatch.setattr(itl, "_raw_stream", itl._stream_handle)
    side = torch.cuda.Stream(device=cuda)
    side.wait_stream(torch.cuda.current_stream(cuda))
    with torch.cuda.stream(side):
        got = call()
    side.synchronize()
    for a, b in zip(want, got):
        assert same_bits(a, b)
