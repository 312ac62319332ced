"""The AdamW step's refusals on the host (no GPU, nothing launched)."""

import ctypes

import pytest

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
MB = 1 << 20
v = ctypes.c_void_p


@pytest.fixture(scope="module")
def itl():
    import invariant_token_logprobs_lm_amd as itl

    return itl


def _step(itl, pieces=64, bits=8, eps=1e-8, betas=(0.9, 0.95), **over):
    names = ("plan", "m", "v", "m_scale", "v_scale", "master", "lr", "step", "norm", "ws")
    p = {k: v(over.get(k, (n + 1) * MB)) for n, k in enumerate(names)}
    return itl.lib.itl_adamw_step(p["plan"], 40 * pieces, bits, p["m"], p["v"], p["m_scale"], p["v_scale"], p["master"], p["lr"],
                                  p["step"], *betas, eps, 1.0, p["norm"], p["ws"], MB, None)


def test_shared_states_are_refused(itl):
    at = lambda n: (n + 1) * MB
    shared = [dict(v=at(1)), dict(m=at(0)), dict(v=at(1) + 64 * 256 - 16), dict(m_scale=at(1)), dict(v_scale=at(3) + 252),
              dict(master=at(1)), dict(master=at(5), v=at(5) + 64 * 1024 - 16), dict(lr=at(5) + 4), dict(step=at(2)),
              dict(lr=at(7) + 4), dict(norm=at(6)), dict(norm=at(9)), dict(ws=at(0)), dict(plan=at(5))]
    for over in shared:
        if over == dict(v=at(1)):
            assert _step(itl, bits=32, **over) == INVALID and "share" in itl.lib.itl_last_error().decode()
        assert _step(itl, **over) == INVALID and "share" in itl.lib.itl_last_error().decode(), over
    assert _step(itl, bits=32, v=at(1) + 64 * 1024 - 16) == INVALID


def test_eps_that_vanishes_in_fp32_is_refused(itl):
    """The kernel adds eps in fp32: where it is 0 a weight without a gradient becomes 0 / 0."""
    for eps in (1e-46, 1e-300, 0.0, float("nan")):
        assert _step(itl, eps=eps) == INVALID and "eps" in itl.lib.itl_last_error().decode(), eps
    assert _step(itl, eps=1e-44, ws=0) == WORKSPACE  # (a subnormal eps is one: the next check answers)


def test_more_pieces_than_a_launch_has_threads_for_are_refused(itl):
    """A workgroup of 256 threads per piece: 2^24 pieces are a grid dimension's 2^32
    threads, and the launch would wrap without an error."""
    def sizes(n):
        t = itl._AdamWTensor(MB, 1 << 50, n, 0, 0, 0.0)
        nb, el = ctypes.c_int64(), ctypes.c_int64()
        return itl.lib.itl_adamw_plan_sizes(ctypes.byref(t), 1, ctypes.byref(nb), ctypes.byref(el)), nb.value

    most = (1 << 24) - 1
    assert sizes(most * 2048) == (OK, most * 40)
    assert sizes(most * 2048 + 1)[0] == UNSUPPORTED
    assert _step(itl, pieces=most + 1) == UNSUPPORTED
