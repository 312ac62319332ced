"""Dropout and the norms with it against their 64-bit forms: the generator's
bits, both types, widths read in whole vectors and others, one row to many,
far rows, all and none dropped; the norms' forward (own type and block codes)
and backward, the gradient against differences; pieces, other streams, replayed
graphs, values that are not finite where they are dropped.

Tolerances, from the arithmetic: the keep factor is one fp32 rounding and its
product another; the rest as the norms' without dropout (test_gpu_norm.py).
"""

import pytest
import torch

import block_refs as B
import learner_refs as R
from helpers import same_bits, say

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 8), (3, 7), (2, 64), (5, 100), (130, 136), (7, 513), (1, 2560), (33, 1001), (700, 24), (9, 4096),
          (4, 5000), (3, 5001), (3, 7168), (2, 8200), (2, 16384), (2, 20008), (2, 20011)]
DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def itl():
    import invariant_token_logprobs_lm_amd as itl

    return itl


def _drop(itl, device, p=0.3, seed=0x1234567890ABCDEF, site=5, first_row=0):
    return itl.Dropout(p, torch.tensor([seed], dtype=torch.int64, device=device), site, first_row)


def _factors(n, d, drop):
    return B.keep_factors(n, d, drop.p, int(drop.seed) & (2 ** 64 - 1), drop.site, drop.first_row)


def _bits(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", SHAPES)
def test_dropout(cuda, itl, n, d, dtype):
    x = torch.randn(n, d, generator=torch.Generator().manual_seed(n + d)).to(dtype).to(cuda)
    for kw in ({}, {"p": 0.0}, {"p": 1.0}, {"p": 1e-6}, {"p": 0.5, "seed": -3, "site": 2 ** 32 - 1, "first_row": 2 ** 40 - 1}):
        say("dropout", n, d, dtype, kw)
        drop = _drop(itl, cuda, **kw)
        f = _factors(n, d, drop)
        want = R.f64(x) * f
        got = R.f64(itl.dropout(x, drop))
        assert torch.equal(got == 0, (f == 0) | (R.f64(x) == 0))
        assert bool(((got - want).abs() <= (R.half_step(dtype) + 2 * R.EPS24) * want.abs()).all())
    y = x.clone()
    assert itl.dropout(y, drop, y=y) is y and torch.equal(_bits(y), _bits(itl.dropout(x, drop)))


def test_share_dropped(cuda, itl):
    """Of 2^22 values p are dropped, within five standard deviations; columns, rows, sites and seeds differ."""
    x = torch.ones(2048, 2048, device=cuda)
    first = itl.dropout(x, _drop(itl, cuda, 0.1)) == 0
    sd = (0.1 * 0.9 / x.numel()) ** 0.5
    assert abs(float(first.double().mean()) - 6554 / 65536) < 5 * sd
    for other in (_drop(itl, cuda, 0.1, site=6), _drop(itl, cuda, 0.1, seed=7), _drop(itl, cuda, 0.1, first_row=2048)):
        both = float((first & (itl.dropout(x, other) == 0)).double().mean())
        assert abs(both - 0.01) < 5 * (0.01 * 0.99 / x.numel()) ** 0.5
    for cols in (first[:, ::2], first[:, 1::2], first[:, 7::8]):
        assert abs(float(cols.double().mean()) - 0.1) < 5 * (0.09 / cols.numel()) ** 0.5


@pytest.mark.parametrize("d", [64, 100, 1001])
def test_pieces_have_the_bits_of_the_whole(cuda, itl, d):
    n = 37
    x = torch.randn(n, d, device=cuda)
    base = 2 ** 32 - 20  # the rows' numbers pass 32 bits
    whole = itl.dropout(x, _drop(itl, cuda, first_row=base))
    for a, b in ((0, 1), (5, 30), (36, 37)):
        assert same_bits(itl.dropout(x[a:b].contiguous(), _drop(itl, cuda, first_row=base + a)), whole[a:b])
    # and of any width
    wide = itl.dropout(torch.ones(n, 1024, device=cuda), _drop(itl, cuda)) != 0
    assert torch.equal(itl.dropout(torch.ones(n, d, device=cuda), _drop(itl, cuda)) != 0, wide[:, :d] if d < 1024 else wide)


def test_nothing_beyond_the_rows_is_written(cuda, itl):
    for n, d, dtype in ((3, 7, torch.float32), (5, 72, torch.bfloat16), (1, 513, torch.bfloat16)):
        flat = torch.full((n * d + 64,), 7.0, dtype=dtype, device=cuda)
        y = flat[32:32 + n * d].view(n, d)
        itl.dropout(torch.randn(n, d, device=cuda).to(dtype), _drop(itl, cuda), y=y)
        assert bool((flat[:32] == 7).all()) and bool((flat[32 + n * d:] == 7).all())


def test_more_rows_than_a_part_of_the_grid_holds(cuda, itl):
    """Rows of two groups: 2^31 groups and more, in two parts (19 GB, in place)."""
    n, d, k = (1 << 30) + 1000, 9, 1 << 16
    x = torch.ones(n, d, dtype=torch.bfloat16, device=cuda)
    itl.dropout(x, _drop(itl, cuda), y=x)
    for a in (0, n - k):  # (the second part begins at row 2^30 - 1)
        assert torch.equal(x[a:a + k].cpu() == 0, _factors(k, d, _drop(itl, cuda, first_row=a)) == 0), a


def test_dropped_values_are_zero_whatever_they_are(cuda, itl):
    for d in (64, 65):
        x = torch.randn(4, d, device=cuda)
        drop = _drop(itl, cuda, 0.5)
        dropped = itl.dropout(x, drop) == 0
        for bad in (float("nan"), float("inf"), -float("inf")):
            y = torch.where(dropped, torch.full_like(x, bad), x)
            assert same_bits(itl.dropout(y, drop), itl.dropout(x, drop))
            w = torch.ones(d, device=cuda)
            h, u, _, _ = itl.residual_norm(x, y, w, dropout=drop)
            h2, u2, r, _ = itl.residual_norm(x, x, w, dropout=drop)
            assert same_bits(h, h2) and same_bits(u, u2)
            gate = torch.ones_like(x)
            a = itl.residual_norm_backward(x, None, h, y, w, r, gate=gate, dropout=drop)
            b = itl.residual_norm_backward(x, None, h, x, w, r, gate=gate, dropout=drop)
            assert all(same_bits(p, q) for p, q in zip(a, b) if p is not None)
            a = itl.residual_norm_backward(x, None, h, y, w, r, gate=w, dropout=drop)
            b = itl.residual_norm_backward(x, None, h, x, w, r, gate=w, dropout=drop)
            assert all(same_bits(p, q) for p, q in zip(a, b) if p is not None)


# ------------------------------------------------------------------ the norms

def _operands(n, d, dtype, post, gate, seed, device):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    t = {"x": r(n, d), "y": 0.7 * r(n, d), "w_pre": 1 + 0.1 * r(d), "w_post": 0.8 + 0.1 * r(d) if post else None,
         "gate": None if gate == 0 else 0.5 + 0.3 * (r(d) if gate == 1 else r(n, d))}
    return {k: None if v is None else v.to(dtype).to(device) for k, v in t.items()}


def _kw(t, scale=0.5):
    return {"w_post": t["w_post"], "gate": t["gate"], "scale": scale}


def _k(d):
    return (d / 32 + 66) * R.EPS24


def _gate(c, f):
    return f if c["gate"] is None else c["gate"] * f


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", SHAPES)
def test_norm_forward(cuda, itl, n, d, dtype):
    for post, gate in ((False, 0), (True, 1), (True, 2), (False, 2)):
        say("norm forward", n, d, dtype, post, gate)
        t, drop = _operands(n, d, dtype, post, gate, n * 7 + d, cuda), _drop(itl, cuda, 0.2, first_row=3)
        h, u, r_pre, r_post = itl.residual_norm(t["x"], t["y"], t["w_pre"], dropout=drop, **_kw(t))
        c = {k: R.f64(v) for k, v in t.items()}
        want, mag, rp = R.norm_forward(c["x"], c["y"], c["w_pre"], c["w_post"], _gate(c, _factors(n, d, drop)), 0.5)
        assert bool(((R.f64(h) - want).abs() <= (R.half_step(dtype) + _k(d)) * mag).all())
        wu, wr = R.norm_out(R.f64(h), c["w_pre"])
        assert bool(((R.f64(u) - wu).abs() <= (R.half_step(dtype) + _k(d)) * wu.abs()).all())
        assert bool(((R.f64(r_pre) - wr).abs() <= _k(d) * wr).all())
        if post:
            assert bool(((R.f64(r_post) - rp).abs() <= _k(d) * rp).all())
        # p 0 is no dropout, bit for bit
        a = itl.residual_norm(t["x"], t["y"], t["w_pre"], dropout=_drop(itl, cuda, 0.0), **_kw(t))
        b = itl.residual_norm(t["x"], t["y"], t["w_pre"], **_kw(t))
        assert all(torch.equal(_bits(p), _bits(q)) for p, q in zip(a, b) if p is not None)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", [(1, 128), (3, 1536), (70, 2560), (5, 4096), (2, 7168), (3, 16384), (2, 16512)])
def test_norm_to_block_codes(cuda, itl, n, d, dtype):
    t = _operands(n, d, dtype, True, 1, d, cuda)
    t["y"][0] = 0
    t["x"][0] = 0
    for drop in (None, _drop(itl, cuda, 0.2)):
        h, Uq, s, r_pre, r_post = itl.residual_norm_blocks_fp8(t["x"], t["y"], t["w_pre"], dropout=drop, **_kw(t))
        h2, u2, r2, p2 = itl.residual_norm(t["x"], t["y"], t["w_pre"], dropout=drop, **_kw(t))
        assert s.shape == (d // 128, n) and float(s[:, 0].min()) == 1.0 and not bool(Uq[0].any())
        assert torch.equal(_bits(h), _bits(h2)) and same_bits(r_post, p2)
        if d <= 16384:
            assert same_bits(r_pre, r2)
        if dtype == torch.float32 and d <= 16384:  # nothing is rounded in between: the quantiser's codes
            q, qs, _, _ = itl.quantize_blocks_fp8(u2)
            assert torch.equal(q, Uq) and same_bits(qs, s)
        c = {k: R.f64(v) for k, v in t.items()}
        wu, _ = R.norm_out(R.f64(h), c["w_pre"])
        top = wu.view(n, d // 128, 128).abs().amax(2).t() / 448
        assert bool(((R.f64(s) - torch.where(top > 0, top, torch.ones_like(top))).abs() <= (_k(d) + R.EPS24) * torch.where(top > 0, top, torch.ones_like(top))).all())
        back = (B.values(Uq).view(n, d // 128, 128) * R.f64(s).t()[:, :, None]).view(n, d)
        # half a step of E4M3: 2^-4 of a value, 2^-10 of the scale's unit below the normal range
        unit = R.f64(s).t().repeat_interleave(128, 1) * 2.0 ** -10
        assert bool(((back - wu).abs() <= (2.0 ** -4 + 2 * _k(d)) * wu.abs() + unit).all())
    # without y: the stored rows' norm
    h, Uq, s, _, _ = itl.residual_norm_blocks_fp8(t["x"], None, t["w_pre"])
    assert h is t["x"]
    if dtype == torch.float32 and d <= 16384:
        q, qs, _, _ = itl.quantize_blocks_fp8(itl.residual_norm(t["x"], None, t["w_pre"])[1])
        assert torch.equal(q, Uq) and same_bits(qs, s)


@pytest.mark.parametrize("dtype,grad", [(torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32)])
@pytest.mark.parametrize("n,d", SHAPES)
def test_norm_backward(cuda, itl, n, d, dtype, grad):
    g = torch.Generator().manual_seed(n + 3 * d)
    for post, gate, with_dh in ((False, 0, True), (True, 1, True), (True, 2, False), (False, 2, True), (False, 1, True)):
        say("norm backward", n, d, dtype, grad, post, gate)
        t, drop = _operands(n, d, dtype, post, gate, n * 7 + d, cuda), _drop(itl, cuda, 0.2, first_row=2 ** 32 - 1)
        h, _, r_pre, r_post = itl.residual_norm(t["x"], t["y"], t["w_pre"], dropout=drop, **_kw(t))
        du = torch.randn(n, d, generator=g).to(grad).to(cuda)
        dh = torch.randn(n, d, generator=g).to(dtype).to(cuda) if with_dh else None
        got = itl.residual_norm_backward(du, dh, h, t["y"], t["w_pre"], r_pre, rstd_post=r_post, dropout=drop, **_kw(t))
        c = {k: R.f64(v) for k, v in t.items()}
        f = _factors(n, d, drop)
        want, mag = R.norm_backward(R.f64(du), R.f64(dh), R.f64(h), c["y"], c["w_pre"], R.f64(r_pre), c["w_post"],
                                    R.f64(r_post), _gate(c, f), 0.5)
        if gate:  # of the gate itself, not of gate times keep factor
            q = c["y"] if not post else c["y"] * R.f64(r_post)[:, None] * c["w_post"]
            dg, mg = 0.5 * q * f * want["dx"], (0.5 * q * f).abs() * mag["dx"]
            want["dgate"], mag["dgate"] = (dg.sum(0), mg.sum(0)) if gate == 1 else (dg, mg)
        else:
            want.pop("dgate")
        tol = _k(d) + (n + 8) * R.EPS24
        for name, v in zip(("dx", "dy", "dw_pre", "dw_post", "dgate"), got):
            if name not in want:
                assert v is None, name
                continue
            own = R.half_step(dtype) if v.dtype == dtype else R.EPS24
            off = (R.f64(v) - want[name]).abs()
            assert bool((off <= own * want[name].abs() + 4 * tol * mag[name] + 1e-300).all()), (name, post, gate)


def test_norm_gradient_against_differences(cuda, itl):
    """Of sum(h a + u b) in fp32, along random directions: differences of the
    64-bit form, whose truncation at a step of 1e-5 is below 1e-8 of the slope."""
    n, d = 5, 136
    t, drop = _operands(n, d, torch.float32, True, 1, 1, cuda), _drop(itl, cuda, 0.3)
    g = torch.Generator().manual_seed(9)
    a, b = torch.randn(n, d, generator=g), torch.randn(n, d, generator=g)
    h, _, r_pre, r_post = itl.residual_norm(t["x"], t["y"], t["w_pre"], dropout=drop, **_kw(t))
    got = itl.residual_norm_backward(b.to(cuda), a.to(cuda), h, t["y"], t["w_pre"], r_pre, rstd_post=r_post, dropout=drop, **_kw(t))
    c, f = {k: R.f64(v) for k, v in t.items()}, _factors(n, d, drop)

    def value(c):
        h, _, _ = R.norm_forward(c["x"], c["y"], c["w_pre"], c["w_post"], c["gate"] * f, 0.5)
        return float((h * a.double() + R.norm_out(h, c["w_pre"])[0] * b.double()).sum())

    for name, grad in zip(("x", "y", "w_pre", "w_post", "gate"), got):
        way = torch.randn(c[name].shape, generator=g).double()
        e = 1e-5
        slope = (value({**c, name: c[name] + e * way}) - value({**c, name: c[name] - e * way})) / (2 * e)
        along = float((R.f64(grad) * way).sum())
        bound = float((R.f64(grad).abs() * way.abs()).sum())
        assert abs(along - slope) <= 1e-5 * bound, name


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 65, 5000, 5001, 8200])
def test_dropped_gradients_are_zero_whatever_they_meet(cuda, itl, d, dtype):
    """Gates, post norm weights and a gradient of h that are not finite where the value is
    dropped: the bits of a call with ordinary numbers there (dx holds dh itself)."""
    for n, post, gate in ((6, False, 2), (6, True, 2), (1, False, 1), (1, True, 1)):
        say("dropped gradients", n, d, dtype, post, gate)
        t, drop = _operands(n, d, dtype, post, gate, d, cuda), _drop(itl, cuda, 0.5)
        out = (_factors(n, d, drop) == 0).to(cuda)
        g = torch.Generator().manual_seed(d)
        du, dh = torch.randn(n, d, generator=g).to(cuda), torch.randn(n, d, generator=g).to(dtype).to(cuda)
        forward = itl.residual_norm(t["x"], t["y"], t["w_pre"], dropout=drop, **_kw(t))
        h, _, r_pre, r_post = forward

        def grads(t, dh=dh):
            return itl.residual_norm_backward(du, dh, h, t["y"], t["w_pre"], r_pre, rstd_post=r_post, dropout=drop, **_kw(t))

        def same(a, b):
            return all(torch.equal(_bits(p), _bits(q)) for p, q in zip(a, b) if p is not None)

        want = grads(t)
        for bad in (float("nan"), float("inf"), -float("inf")):
            spoilt = lambda v: torch.where(out if v.dim() == 2 else out[0], torch.full_like(v, bad), v)
            with_gate = {**t, "gate": spoilt(t["gate"])}
            assert same(itl.residual_norm(t["x"], t["y"], t["w_pre"], dropout=drop, **_kw(with_gate)), forward), bad
            assert same(grads(with_gate), want), ("gate", bad)
            if post and n == 1:
                assert same(grads({**t, "w_post": spoilt(t["w_post"])}), want), ("w_post", bad)
            got = grads(t, spoilt(dh))
            assert same(got[1:], want[1:]) and torch.equal(got[0][~out], want[0][~out]), ("dh", bad)


def test_norm_rows_do_not_depend_on_their_batch(cuda, itl):
    for d in (2560, 1001):
        t, drop = _operands(50, d, torch.bfloat16, True, 2, 3, cuda), _drop(itl, cuda, 0.2)
        whole = itl.residual_norm(t["x"], t["y"], t["w_pre"], dropout=drop, **_kw(t))
        part = {k: v if v is None or v.dim() == 1 else v[20:23].contiguous() for k, v in t.items()}
        some = itl.residual_norm(part["x"], part["y"], part["w_pre"], dropout=drop._replace(first_row=20), **_kw(part))
        assert all(torch.equal(_bits(p[20:23]), _bits(q)) for p, q in zip(whole, some))


@pytest.mark.parametrize("d", [256, 1001])
def test_replays_take_the_seed_as_it_is(cuda, itl, d):
    t, seed = _operands(64, d, torch.bfloat16, True, 1, 3, cuda), torch.tensor([5], dtype=torch.int64, device=cuda)
    drop = itl.Dropout(0.2, seed)

    def step():
        seed.add_(1)
        h, u, r_pre, r_post = itl.residual_norm(t["x"], t["y"], t["w_pre"], dropout=drop, **_kw(t))
        return (itl.dropout(u, drop), h, *itl.residual_norm_backward(u, None, h, t["y"], t["w_pre"], r_pre, rstd_post=r_post,
                                                                  dropout=drop, **_kw(t)))

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    seen = set()
    for _ in range(4):
        before = int(seed)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        assert int(seed) == before + 1
        seed.fill_(before)
        want = step()
        assert all(torch.equal(_bits(a), _bits(b)) for a, b in zip(got, want))
        seen.add(int((got[0] == 0).sum()))
    assert len(seen) > 1


def test_other_streams(cuda, itl):
    x, drop = torch.randn(300, 1001, device=cuda), _drop(itl, cuda)
    want = itl.dropout(x, drop)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(itl.dropout(x, drop))
    torch.cuda.synchronize()
    assert all(same_bits(g, want) for g in got)


def test_refusals(cuda, itl):
    x, w = torch.randn(4, 64, device=cuda), torch.ones(64, device=cuda)
    drop = _drop(itl, cuda)
    for bad in (drop._replace(seed=drop.seed.cpu()), drop._replace(seed=drop.seed.int()), drop._replace(site=-1),
                drop._replace(site=2 ** 32), drop._replace(first_row=-1), drop._replace(seed=drop.seed.expand(2).contiguous())):
        with pytest.raises(ValueError):
            itl.dropout(x, bad)
    for bad in (drop._replace(p=1.5), drop._replace(p=float("nan"))):
        with pytest.raises(itl.ItlError):
            itl.dropout(x, bad)
    with pytest.raises(TypeError):
        itl.dropout(x, (0.1, drop.seed))
    with pytest.raises(ValueError):
        itl.dropout(x.t(), drop)
    with pytest.raises(ValueError):
        itl.dropout(x, drop, y=torch.empty(4, 63, device=cuda))
    with pytest.raises(itl.ItlError):  # y over part of x
        flat = torch.zeros(5 * 64, device=cuda)
        itl.dropout(flat[:256].view(4, 64), drop, y=flat[64:].view(4, 64))
    with pytest.raises(itl.ItlError):  # nothing to drop
        itl.residual_norm(x, None, w, dropout=drop)
    with pytest.raises(itl.ItlError):
        itl.residual_norm_blocks_fp8(x, None, w)
    assert itl.dropout(x[:0], drop).shape == (0, 64)
    assert itl.residual_norm(x[:0], x[:0], w, dropout=drop)[1].shape == (0, 64)
    grads = itl.residual_norm_backward(x[:0], None, x[:0], x[:0], w, w[:0], dropout=drop)
    assert not bool(grads[2].any())
