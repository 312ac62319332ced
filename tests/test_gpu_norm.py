"""The norms around a block against their 64-bit forms: both types, both
column walks (widths of a multiple of 8 and others), one row and many, gates
of both shapes, with and without the post norm; then invariance, aliasing,
other streams and replayed graphs.

Tolerances, from the arithmetic: the row sums add d / 64 values or more per
lane and then log2 of the lanes: K = d / 32 + 64 half steps of fp32 relative
to the sum of magnitudes covers every order the kernels use; each stored value
adds half a step of its own type.
"""

import pytest
import torch

import learner_refs as R
from helpers import same_bits, say

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 8), (3, 7), (2, 64), (5, 100), (7, 200), (1, 2560), (33, 1001), (130, 512), (65, 1536), (9, 4096),
          (4, 5000), (3, 7168), (2, 8200), (3, 16384), (2, 20008), (1000, 128)]


def _itl():
    import invariant_token_logprobs_lm_amd as itl

    return itl


def _operands(n, d, dtype, post, gate, seed, device):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    t = {"x": r(n, d), "y": 0.7 * r(n, d), "w_pre": 1 + 0.1 * r(d), "w_post": 0.8 + 0.1 * r(d) if post else None,
         "gate": None if gate == 0 else 0.5 + 0.3 * (r(d) if gate == 1 else r(n, d))}
    return {k: None if v is None else v.to(dtype).to(device) for k, v in t.items()}


def _kw(t, scale=0.5):
    return {"w_post": t["w_post"], "gate": t["gate"], "scale": scale}


def _k(d):
    return (d / 32 + 64) * R.EPS24


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,d", SHAPES)
def test_forward(cuda, n, d, dtype):
    itl = _itl()
    for post, gate in ((False, 0), (True, 1), (True, 2), (False, 2)):
        say("norm forward", n, d, dtype, post, gate)
        t = _operands(n, d, dtype, post, gate, n * 7 + d, cuda)
        h, u, r_pre, r_post = itl.residual_norm(t["x"], t["y"], t["w_pre"], **_kw(t))
        c = {k: R.f64(v) for k, v in t.items()}
        want, mag, rp = R.norm_forward(c["x"], c["y"], c["w_pre"], c["w_post"], c["gate"], 0.5)
        assert bool(((R.f64(h) - want).abs() <= (R.half_step(dtype) + _k(d)) * mag).all())
        wu, wr = R.norm_out(R.f64(h), c["w_pre"])  # the norm is the kept h's
        assert bool(((R.f64(u) - wu).abs() <= (R.half_step(dtype) + _k(d)) * wu.abs()).all())
        assert bool(((R.f64(r_pre) - wr).abs() <= _k(d) * wr).all())
        if post:
            assert bool(((R.f64(r_post) - rp).abs() <= _k(d) * rp).all())
        else:
            assert r_post is None


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,d", [(1, 128), (3, 1536), (70, 2560), (5, 4096), (2, 7168), (2, 16512)])
def test_forward_fp8(cuda, n, d, dtype):
    itl = _itl()
    t = _operands(n, d, dtype, True, 1, d, cuda)
    t["y"][0] = 0
    t["x"][0] = 0  # a row of zeros: scale 1, codes 0
    h, Uq, s, r_pre, _ = itl.residual_norm_fp8(t["x"], t["y"], t["w_pre"], **_kw(t))
    h2, u2, r2, _ = itl.residual_norm(t["x"], t["y"], t["w_pre"], **_kw(t))
    assert torch.equal(h.view(torch.uint8), h2.view(torch.uint8)) and same_bits(r_pre, r2)
    assert float(s[0]) == 1.0 and not bool(Uq[0].any())
    # in fp32 the two-step path rounds nothing in between: the same codes and scales
    if dtype == torch.float32:
        q, qs = itl.quantize_rows_fp8(u2)
        assert torch.equal(q, Uq) and same_bits(qs, s)
        assert torch.equal((u2 / s[:, None]).cpu().to(torch.float8_e4m3fn).view(torch.uint8), Uq.cpu())
    wu, _ = R.norm_out(R.f64(h), R.f64(t["w_pre"]))
    amax = wu.abs().amax(1)
    assert bool(((R.f64(s)[1:] - amax[1:] / 448).abs() <= (_k(d) + 2 * R.EPS24) * amax[1:] / 448).all())
    got = Uq.cpu().view(torch.float8_e4m3fn).double() * R.f64(s)[:, None]
    # half a step: 2^-4 of the value, or of the subnormals' step 2^-9
    bound = torch.maximum(wu.abs() * 2.0 ** -4, R.f64(s)[:, None] * 2.0 ** -10) + 2 * _k(d) * wu.abs()
    assert bool(((got - wu).abs() <= bound).all())


@pytest.mark.parametrize("dtype,grad", [(torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16),
                                        (torch.float32, torch.float32)])
@pytest.mark.parametrize("n,d", SHAPES)
def test_backward(cuda, n, d, dtype, grad):
    itl = _itl()
    for post, gate, with_dh in ((False, 0, True), (True, 1, True), (True, 2, False), (False, 1, True)):
        say("norm backward", n, d, dtype, grad, post, gate, with_dh)
        t = _operands(n, d, dtype, post, gate, n * 5 + d, cuda)
        h, _, r_pre, r_post = itl.residual_norm(t["x"], t["y"], t["w_pre"], **_kw(t))
        g = torch.Generator().manual_seed(n + d)
        du = torch.randn(n, d, generator=g).to(grad).to(cuda)
        dh = torch.randn(n, d, generator=g).to(dtype).to(cuda) if with_dh else None
        dx, dy, dw_pre, dw_post, dgate = itl.residual_norm_backward(du, dh, h, t["y"], t["w_pre"], r_pre,
                                                                    rstd_post=r_post, **_kw(t))
        got = {"dx": dx, "dy": dy, "dw_pre": dw_pre, "dw_post": dw_post, "dgate": dgate}
        want, mag = R.norm_backward(R.f64(du), R.f64(dh), R.f64(h), R.f64(t["y"]), R.f64(t["w_pre"]), R.f64(r_pre),
                                    R.f64(t["w_post"]), R.f64(r_post), R.f64(t["gate"]), 0.5)
        for k, v in got.items():
            if k not in want:
                assert v is None, k
                continue
            column = v.dim() == 1
            # a column's sum over n rows: at most n additions on top of its terms' own error
            tol = (2 * _k(d) + (n * R.EPS24 if column else 0.0)) * mag[k]
            if v.dtype != torch.float32:
                tol = tol + R.half_step(v.dtype) * (want[k].abs() + tol)
            else:
                tol = tol + R.EPS24 * want[k].abs()
            assert bool(((R.f64(v) - want[k]).abs() <= tol).all()), k


def test_without_a_block(cuda):
    """y None: the norm of x alone, the same bits as norming a stored h."""
    itl = _itl()
    for d in (1001, 2560):
        t = _operands(40, d, torch.bfloat16, True, 1, d, cuda)
        h, u, r, _ = itl.residual_norm(t["x"], t["y"], t["w_pre"], **_kw(t))
        h2, u2, r2, none = itl.residual_norm(h, None, t["w_pre"])
        assert h2 is h and none is None and torch.equal(u, u2) and same_bits(r, r2)
        dx, dy, dw, dp, dg = itl.residual_norm_backward(u, None, h, None, t["w_pre"], r)
        want, mag = R.norm_backward(R.f64(u), None, R.f64(h), None, R.f64(t["w_pre"]), R.f64(r))
        assert dy is None and dp is None and dg is None
        tol = 2 * _k(d) * mag["dx"]
        assert bool(((R.f64(dx) - want["dx"]).abs() <= tol + 2.0 ** -8 * (want["dx"].abs() + tol)).all())


@pytest.mark.parametrize("d", [1001, 2560, 7168])
def test_rows_do_not_depend_on_the_batch(cuda, d):
    itl = _itl()
    t = _operands(300, d, torch.bfloat16, True, 2, d, cuda)
    du = torch.randn(300, d, device=cuda)
    h, u, r, rp = itl.residual_norm(t["x"], t["y"], t["w_pre"], **_kw(t))
    dx, dy, *_ = itl.residual_norm_backward(du, h, h, t["y"], t["w_pre"], r, rstd_post=rp, **_kw(t))
    for rows in ([0], [17], [299], list(range(250, 300)), [5, 4, 3, 100]):
        i = torch.tensor(rows, device=cuda)
        kw = {"w_post": t["w_post"], "gate": t["gate"][i].contiguous(), "scale": 0.5}
        h1, u1, r1, rp1 = itl.residual_norm(t["x"][i], t["y"][i], t["w_pre"], **kw)
        assert torch.equal(h1, h[i]) and torch.equal(u1, u[i]) and same_bits(r1, r[i]) and same_bits(rp1, rp[i])
        dx1, dy1, *_ = itl.residual_norm_backward(du[i], h1, h1, t["y"][i], t["w_pre"], r1, rstd_post=rp1, **kw)
        assert torch.equal(dx1, dx[i]) and torch.equal(dy1, dy[i])


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 4096), (torch.float32, 2048), (torch.bfloat16, 8192)])
def test_rows_of_a_large_call(cuda, dtype, d):
    """Results past the caches' size take another store: the same bits as the rows alone."""
    itl = _itl()
    n = (80 << 20) // (d * (2 if dtype == torch.bfloat16 else 4))
    x = torch.randn(n, d, device=cuda).to(dtype)
    y = torch.randn(n, d, device=cuda).to(dtype)
    w = torch.randn(d, device=cuda).to(dtype)
    h, u, r, _ = itl.residual_norm(x, y, w)
    for i in (slice(0, 3), slice(n // 2, n // 2 + 50), slice(n - 1, n)):
        h1, u1, r1, _ = itl.residual_norm(x[i], y[i], w)
        assert torch.equal(h1, h[i]) and torch.equal(u1, u[i]) and same_bits(r1, r[i])


@pytest.mark.parametrize("n,d", [(700, 2560), (64, 1001), (5000, 96), (257, 9000)])
def test_column_sums_are_deterministic(cuda, n, d):
    itl = _itl()
    t = _operands(n, d, torch.bfloat16, True, 1, d, cuda)
    du = torch.randn(n, d, device=cuda)
    h, u, r, rp = itl.residual_norm(t["x"], t["y"], t["w_pre"], **_kw(t))
    first = itl.residual_norm_backward(du, None, h, t["y"], t["w_pre"], r, rstd_post=rp, **_kw(t))
    again = itl.residual_norm_backward(du, None, h, t["y"], t["w_pre"], r, rstd_post=rp, **_kw(t))
    for a, b in zip(first[2:], again[2:]):
        assert same_bits(a, b)


@pytest.mark.parametrize("d", [1001, 2560, 5001, 7168, 9000, 16392])
def test_in_place(cuda, d):
    """h may be x, and dx may be dh."""
    itl = _itl()
    t = _operands(50, d, torch.float32, True, 1, 4, cuda)
    h, u, r, rp = itl.residual_norm(t["x"], t["y"], t["w_pre"], **_kw(t))
    x = t["x"].clone()
    h2, u2, *_ = itl.residual_norm(x, t["y"], t["w_pre"], h=x, **_kw(t))
    assert h2 is x and same_bits(x, h) and same_bits(u, u2)
    dh = torch.randn(50, d, device=cuda)
    want = itl.residual_norm_backward(u, dh, h, t["y"], t["w_pre"], r, rstd_post=rp, **_kw(t))
    got = itl.residual_norm_backward(u, dh, h, t["y"], t["w_pre"], r, rstd_post=rp, dx=dh, **_kw(t))
    assert got[0] is dh
    for a, b in zip(want, got):
        assert same_bits(a, b)


def test_nothing_and_bad_values(cuda):
    itl = _itl()
    e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device=cuda)
    h, u, r, rp = itl.residual_norm(e(0, 64), e(0, 64), e(64), w_post=e(64))
    assert u.shape == (0, 64) and r.numel() == 0
    dx, dy, dw, dwp, dg = itl.residual_norm_backward(e(0, 64), None, h, e(0, 64), e(64), r, w_post=e(64), rstd_post=rp,
                                                     gate=e(64))
    for s in (dw, dwp, dg):
        assert not bool(s.any())
    # a NaN stays in its row
    t = _operands(6, 2560, torch.bfloat16, True, 1, 1, cuda)
    want = itl.residual_norm(t["x"], t["y"], t["w_pre"], **_kw(t))
    t["y"][2, 5] = float("nan")
    t["x"][4, 9] = float("inf")
    got = itl.residual_norm(t["x"], t["y"], t["w_pre"], **_kw(t))
    keep = torch.tensor([0, 1, 3, 5], device=cuda)
    assert torch.equal(got[1][keep], want[1][keep])
    assert bool(got[1][2].isnan().all()) and bool(got[1][4, 9].isnan())


def test_refusals(cuda):
    itl = _itl()
    t = _operands(4, 64, torch.bfloat16, True, 1, 1, cuda)
    x, y, w = t["x"], t["y"], t["w_pre"]
    bad = [
        (ValueError, lambda: itl.residual_norm(x, y.float(), w)),
        (ValueError, lambda: itl.residual_norm(x, y[:3], w)),
        (ValueError, lambda: itl.residual_norm(x.t(), y.t(), w)),
        (ValueError, lambda: itl.residual_norm(x, y, w[:32])),
        (ValueError, lambda: itl.residual_norm(x, None, w, gate=w)),
        (ValueError, lambda: itl.residual_norm(x, y, w, gate=w[:1])),
        (itl.ItlError, lambda: itl.residual_norm(x, y, w, eps=0.0)),
        (itl.ItlError, lambda: itl.residual_norm(x, y, w, scale=float("nan"))),
        (itl.ItlError, lambda: itl.residual_norm_fp8(x, y, w)),  # 64 is no multiple of 128
        (ValueError, lambda: itl.residual_norm(x, y, w, u=torch.empty(4, 65, dtype=x.dtype, device=cuda))),
        (ValueError, lambda: itl.residual_norm_backward(x, x, x, y, w, torch.ones(4, device=cuda), w_post=w)),
        (ValueError, lambda: itl.residual_norm_backward(x, x, x, y, w, torch.ones(3, device=cuda))),
        (itl.ItlError, lambda: itl.residual_norm(torch.empty(257, dtype=x.dtype, device=cuda)[1:].view(4, 64), y, w)),
    ]
    for error, call in bad:
        with pytest.raises(error):
            call()


@pytest.mark.parametrize("d", [1001, 2560])
def test_side_stream_and_replay(cuda, d):
    itl = _itl()
    t = _operands(200, d, torch.bfloat16, True, 1, 8, cuda)
    du = torch.randn(200, d, device=cuda)
    ws = torch.empty(itl.residual_norm_backward_workspace_bytes(200, d), dtype=torch.uint8, device=cuda)

    def step():
        h, u, r, rp = itl.residual_norm(t["x"], t["y"], t["w_pre"], **_kw(t))
        return (h, u) + itl.residual_norm_backward(du, h, h, t["y"], t["w_pre"], r, rstd_post=rp, workspace=ws, **_kw(t))

    want = [a.clone() for a in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream(device=cuda)
    side.wait_stream(torch.cuda.current_stream(cuda))
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream(cuda).wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for o in out:
            o.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, out):
            assert torch.equal(a, b)
        step()
        torch.cuda.synchronize()


@pytest.mark.parametrize("d", [256, 7168, 16512])
def test_fp8_rows_that_nearly_vanish(cuda, d):
    """Rows whose amax / 448 would leave fp32's normal range: the scale is at
    least 2^-126. A code is off by half a step of E4M3, 2^-4 of its value or
    2^-10 of the scale; u by a few roundings (2^-20 of it, 2^-148 below the
    normal range)."""
    itl = _itl()
    g = torch.Generator().manual_seed(5)
    x = torch.randn(12, d, generator=g).to(cuda)
    for e in (-110, -122, -128, -134, -140, -149):
        w = torch.full((d,), 2.0 ** e, dtype=torch.float64).to(torch.float32).to(cuda)
        w[::3] = 0.0
        h, q, s, r, _ = itl.residual_norm_fp8(x, None, w)
        assert bool((s >= 2.0 ** -126).all()), e
        got = q.view(torch.float8_e4m3fn).double() * s.double()[:, None]
        u = x.double() * r.double()[:, None] * w.double()
        tol = u.abs() * (2.0 ** -4 + 2.0 ** -20) + s.double()[:, None] * 2.0 ** -10 + 2.0 ** -148
        assert bool(((got - u).abs() <= tol).all()), e
