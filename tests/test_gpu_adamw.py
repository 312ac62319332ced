"""The AdamW step over many tensors against its 64-bit form: every mix of
weight and gradient types, 32- and 8-bit states, sizes of 1 to a few pieces,
misaligned views, clipping; then the 8-bit codes, skipped steps, replayed
graphs and dirty memory.

Tolerances, from the arithmetic (each operation rounds to fp32 once, half a
step of 2^-24): m takes three roundings, v four, the clip factor four more (in
v twice); the weight's quotient takes those of m, v and the root and eight of
its own, beside two of the weight itself; a 16-bit weight half a step of its
type.
"""

import pytest
import torch

import learner_refs as R
from helpers import same_bits, say

pytestmark = pytest.mark.gpu

SIZES = [1, 7, 255, 256, 257, 4095, 4096, 4097, 10000, 0, 64]
BETAS, EPS = (0.9, 0.95), 1e-8


def _itl():
    import invariant_token_logprobs_lm_amd as itl

    return itl


def _tensors(sizes, dtypes, device, seed, scale=1.0, shift=0):
    """Tensors of these sizes, the types taken in turn; `shift`: start that many elements into an allocation."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = (torch.randn(n + shift, generator=g) * scale).to(dtypes[i % len(dtypes)]).to(device)
        out.append(t[shift:])
    return out


def _pieces(flat, plan, i):
    n = plan.params[i].numel()
    return flat[plan.offsets[i]:plan.offsets[i] + n]


def _clip(grads, max_norm):
    norm = float(torch.sqrt(sum((R.f64(g) ** 2).sum() for g in grads)))
    return norm, min(1.0, max_norm / (norm + 1e-6)) if max_norm else 1.0


MIXES = [([torch.float32], [torch.float32]), ([torch.bfloat16], [torch.bfloat16]),
         ([torch.bfloat16, torch.float32], [torch.float32, torch.bfloat16, torch.float32])]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("mix", range(3))
@pytest.mark.parametrize("shift", [0, 3])
def test_three_steps(cuda, bits, mix, shift):
    itl = _itl()
    pd, gd = MIXES[mix]
    for master, max_norm in ((None, None), (False, 0.5)):
        say("adamw", bits, mix, shift, master, max_norm)
        params = _tensors(SIZES, pd, cuda, 1, 0.05, shift)
        grads = _tensors(SIZES, gd, cuda, 2, 0.01, shift)
        decay = [0.1 if i % 2 else 0.0 for i in range(len(SIZES))]
        plan = itl.adamw_plan(params, grads, lr=1e-2, weight_decay=decay, state_bits=bits, master=master)
        lr = float(plan.lr)
        for t in range(1, 4):
            for i, g in enumerate(_tensors(SIZES, gd, cuda, 10 + t, 0.01, shift)):
                grads[i].copy_(g)
            if bits == 32:
                m0, v0 = R.f64(plan.exp_avg), R.f64(plan.exp_avg_sq)
            else:
                m0 = R.e4m3_values(plan.exp_avg, plan.exp_avg_scale, 256)
                v0 = R.e4m3_values(plan.exp_avg_sq, plan.exp_avg_sq_scale, 256) ** 2
            before = [R.f64(_pieces(plan.master, plan, i)) if plan.master is not None and p.dtype == torch.bfloat16
                      else R.f64(p) for i, p in enumerate(params)]
            norm = itl.adamw_step(plan, betas=BETAS, eps=EPS, max_norm=max_norm)
            want_norm, clip = _clip(grads, max_norm)
            assert (norm is None) == (max_norm is None)
            if max_norm:
                assert abs(float(norm) - want_norm) <= 4 * R.EPS24 * want_norm
            assert int(plan.step) == t
            for i, p in enumerate(params):
                if p.numel() == 0:
                    continue
                w, m, v = R.adamw(before[i], R.f64(grads[i]), _pieces(m0, plan, i), _pieces(v0, plan, i), t, lr,
                                  decay[i], BETAS, EPS, clip)
                b1, b2 = BETAS
                g = R.f64(grads[i]) * clip
                mag_m = (b1 * _pieces(m0, plan, i)).abs() + (1 - b1) * g.abs()
                tm, tv = 12 * R.EPS24 * mag_m, 24 * R.EPS24 * v
                if bits == 32:
                    assert bool(((R.f64(_pieces(plan.exp_avg, plan, i)) - m).abs() <= tm).all())
                    assert bool(((R.f64(_pieces(plan.exp_avg_sq, plan, i)) - v).abs() <= tv + 1e-45).all())
                rate = lr / (1 - b1 ** t)
                root = torch.sqrt(v) / (1 - b2 ** t) ** 0.5 + EPS
                tw = 3 * R.EPS24 * before[i].abs() + rate / root * (tm + 40 * R.EPS24 * m.abs()) + R.EPS24 * w.abs()
                held = plan.master is not None and p.dtype == torch.bfloat16
                if held:
                    kept = _pieces(plan.master, plan, i)
                    assert bool(((R.f64(kept) - w).abs() <= tw).all())
                    assert torch.equal(p, kept.to(torch.bfloat16))
                else:
                    half = 0.0 if p.dtype == torch.float32 else R.half_step(p.dtype)
                    assert bool(((R.f64(p) - w).abs() <= tw + half * (w.abs() + tw)).all())
                if bits == 8:
                    _check_codes(plan, i, m, v, tm, tv)


def _check_codes(plan, i, m, v, tm, tv):
    n = m.numel()
    o = plan.offsets[i]
    r, tr = torch.sqrt(v), tv / (2 * torch.sqrt(v).clamp(min=1e-300))
    for codes, scale, want, tol in ((plan.exp_avg, plan.exp_avg_scale, m, tm),
                                    (plan.exp_avg_sq, plan.exp_avg_sq_scale, r, tr)):
        nb = -(-n // 256)
        s = scale[o // 256:o // 256 + nb].cpu()
        c = codes[o:o + nb * 256]
        assert not bool(c[n:].any())  # nothing behind the tensor
        pad = torch.zeros(nb * 256, dtype=torch.float64)
        pad[:n] = want.abs()
        amax = pad.view(nb, 256).amax(1)
        ws = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
        assert bool(((s.double() - ws).abs() <= 32 * R.EPS24 * ws).all())
        got = R.e4m3_values(c, s, 256)[:n]
        step = s.double().repeat_interleave(256)[:n]
        # half a step of the code, or of the subnormals' step; a root below the smallest code is raised to it
        lift = 2.0 ** -9 if want is r else 2.0 ** -10
        assert bool(((got - want).abs() <= torch.maximum(2.0 ** -4 * want.abs(), lift * step) + tol + 64 * R.EPS24 * want.abs()).all())
        if want is r:
            assert not bool(((c[:n].cpu() == 0) & (want > 1e-38)).any())


def test_step_count_and_learning_rate_of_the_replay(cuda):
    """A captured step takes the count, the rate and the gradients of the time it is replayed."""
    itl = _itl()
    for bits in (32, 8):
        def make():
            p = _tensors([5000, 300], [torch.bfloat16], cuda, 3, 0.1)
            g = _tensors([5000, 300], [torch.float32], cuda, 4, 0.1)
            return p, g, itl.adamw_plan(p, g, lr=1e-2, weight_decay=0.1, state_bits=bits)

        (pe, ge, eager), (pc, gc, captured) = make(), make()
        norm_c = torch.empty(1, device=cuda)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            itl.adamw_step(captured, max_norm=1.0, grad_norm=norm_c)
        for rep in range(4):
            new = _tensors([5000, 300], [torch.float32], cuda, 20 + rep, 0.1)
            for a, b, c in zip(ge, gc, new):
                a.copy_(c)
                b.copy_(c)
            for plan in (eager, captured):
                plan.lr.fill_(1e-2 / (rep + 1))
            norm_e = itl.adamw_step(eager, max_norm=1.0)
            graph.replay()
            torch.cuda.synchronize()
            assert same_bits(norm_e, norm_c) and int(captured.step) == rep + 1
            for a, b in zip(pe, pc):
                assert torch.equal(a, b)
            assert torch.equal(eager.exp_avg, captured.exp_avg) and torch.equal(eager.exp_avg_sq, captured.exp_avg_sq)
            assert same_bits(eager.master, captured.master)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("bits", [32, 8])
def test_norm_that_is_not_finite_skips(cuda, bad, bits):
    itl = _itl()
    p = _tensors([9000, 20], [torch.float32, torch.bfloat16], cuda, 5, 0.1)
    g = _tensors([9000, 20], [torch.float32], cuda, 6, 0.1)
    plan = itl.adamw_plan(p, g, lr=1e-2, state_bits=bits)
    itl.adamw_step(plan, max_norm=1.0)
    kept = [t.clone() for t in (*p, plan.exp_avg, plan.exp_avg_sq, plan.master, plan.step)]
    g[0][8999] = bad
    norm = itl.adamw_step(plan, max_norm=1.0)
    assert not bool(norm.isfinite())
    for a, b in zip(kept, (*p, plan.exp_avg, plan.exp_avg_sq, plan.master, plan.step)):
        assert torch.equal(a, b)
    g[0][8999] = 1e25  # its square alone passes fp32's range: the norm does not
    norm = itl.adamw_step(plan, max_norm=1.0)
    assert abs(float(norm) / 1e25 - 1) < 1e-6 and int(plan.step) == 2
    assert bool(p[0].isfinite().all())


def test_clip_is_over_all_tensors(cuda):
    """Splitting the tensors otherwise gives the same weights: the norm is theirs together."""
    itl = _itl()
    g = torch.Generator().manual_seed(1)
    w = (torch.randn(8192, generator=g) * 0.1).to(cuda)
    gr = torch.randn(8192, generator=g).to(cuda)
    a, b = w.clone(), w.clone()
    one = itl.adamw_plan([a], [gr], lr=0.1)
    two = itl.adamw_plan([b[:4096], b[4096:]], [gr[:4096], gr[4096:]], lr=0.1)
    na, nb = itl.adamw_step(one, max_norm=0.3), itl.adamw_step(two, max_norm=0.3)
    assert same_bits(na, nb) and same_bits(a, b)
    # a generous bound leaves the step as without one
    c = w.clone()
    three = itl.adamw_plan([c], [gr], lr=0.1)
    d = w.clone()
    four = itl.adamw_plan([d], [gr], lr=0.1)
    itl.adamw_step(three, max_norm=1e30)
    itl.adamw_step(four)
    assert same_bits(c, d)


def test_neighbours_are_left_as_they_were(cuda):
    """Views inside a larger allocation: nothing outside them changes, nor between the states."""
    itl = _itl()
    whole = torch.full((3000,), 3.5, device=cuda)
    gr = torch.ones(3000, device=cuda)
    for bits in (32, 8):
        pad = torch.zeros(512 + 1792, dtype=torch.float32 if bits == 32 else torch.uint8, device=cuda)
        plan = itl.adamw_plan([whole[5:305], whole[1000:2601]], [gr[5:305], gr[1000:2601]], lr=0.1, state_bits=bits,
                              exp_avg=pad)
        itl.adamw_step(plan, max_norm=1.0)
        outside = torch.ones(3000, dtype=torch.bool, device=cuda)
        outside[5:305] = False
        outside[1000:2601] = False
        assert bool((whole[outside] == 3.5).all()) and not bool((whole[~outside] == 3.5).any())
        assert not bool(pad[300:512].any()) and not bool(pad[512 + 1601:].any())


def test_many_small_tensors(cuda):
    itl = _itl()
    sizes = [1 + (37 * i) % 700 for i in range(500)]
    p = _tensors(sizes, [torch.float32], cuda, 8, 0.1)
    g = _tensors(sizes, [torch.float32], cuda, 9, 0.1)
    flat = torch.cat([t.clone() for t in p])
    ref = itl.adamw_plan([flat], [torch.cat(g)], lr=1e-3, weight_decay=0.1)
    plan = itl.adamw_plan(p, g, lr=1e-3, weight_decay=0.1)
    itl.adamw_step(ref)
    itl.adamw_step(plan)
    assert same_bits(torch.cat(p), flat)


def test_refusals(cuda):
    itl = _itl()
    p, g = torch.zeros(100, device=cuda), torch.zeros(100, device=cuda)
    plan = itl.adamw_plan([p], [g], lr=0.1)
    bad = [
        (ValueError, lambda: itl.adamw_plan([], [], lr=0.1)),
        (ValueError, lambda: itl.adamw_plan([p], [g[:99]], lr=0.1)),
        (ValueError, lambda: itl.adamw_plan([p], [g, g], lr=0.1)),
        (ValueError, lambda: itl.adamw_plan([p.half()], [g], lr=0.1)),
        (ValueError, lambda: itl.adamw_plan([p.cpu()], [g], lr=0.1)),
        (ValueError, lambda: itl.adamw_plan([p], [g], lr=0.1, state_bits=16)),
        (ValueError, lambda: itl.adamw_plan([p], [g], lr=0.1, exp_avg=torch.zeros(100, device=cuda))),
        (ValueError, lambda: itl.adamw_plan([p], [g], lr=0.1, weight_decay=[0.1, 0.1])),
        (itl.ItlError, lambda: itl.adamw_plan([p], [g], lr=0.1, weight_decay=-1.0)),
        (itl.ItlError, lambda: itl.adamw_plan([p, p], [g, g], lr=0.1)),
        (itl.ItlError, lambda: itl.adamw_plan([p[:60], p[50:]], [g[:60], g[50:]], lr=0.1)),
        (TypeError, lambda: itl.adamw_step([p])),
        (itl.ItlError, lambda: itl.adamw_step(plan, betas=(1.0, 0.9))),
        (itl.ItlError, lambda: itl.adamw_step(plan, eps=0.0)),
        (itl.ItlError, lambda: itl.adamw_step(plan, max_norm=0.0)),
        (ValueError, lambda: itl.adamw_step(plan, grad_norm=torch.zeros(2, device=cuda))),
    ]
    for error, call in bad:
        with pytest.raises(error):
            call()


def test_eight_bit_states_fade_away(cuda):
    """Gradients that stay zero: m shrinks by beta1 a step until a block's
    amax / 448 would leave fp32's normal range (2^-126); codes, scales and
    weights stay finite, and what never had a gradient never moves."""
    itl = _itl()
    g = torch.Generator().manual_seed(31)
    p = torch.randn(600, generator=g).to(cuda)
    grad = (torch.randn(600, generator=g) * 1e-3).to(cuda)
    grad[::2] = 0.0
    start = p.clone()
    plan = itl.adamw_plan([p], [grad], lr=1e-3, state_bits=8)
    itl.adamw_step(plan)
    grad.zero_()
    for _ in range(1100):  # 0.9^1100 = 5e-51, below fp32's smallest number
        itl.adamw_step(plan)
    assert bool(p.isfinite().all())
    assert same_bits(p[::2].contiguous(), start[::2].contiguous())
    for codes, scale in ((plan.exp_avg, plan.exp_avg_scale), (plan.exp_avg_sq, plan.exp_avg_sq_scale)):
        assert not bool(((codes & 0x7F) == 0x7F).any())
        assert bool((scale >= 2.0 ** -126).all())
