"""The training loop as the README writes it: one plan over gradients that every
step's backward writes into, with no copies; outputs that have no operand are
refused rather than left unwritten."""

import pytest
import torch

from helpers import same_bits

pytestmark = pytest.mark.gpu


def _model(device, n=200, d=128, V=1500, dtype=torch.bfloat16, rows=False):
    g = torch.Generator().manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=g)
    t = {"w_pre": 1 + 0.1 * r(d), "w_post": 1 + 0.1 * r(d), "gate": 0.5 + 0.1 * (r(n, d) if rows else r(d)), "W": 0.05 * r(V, d)}
    t = {k: v.to(dtype).to(device) for k, v in t.items()}
    batches = [(r(n, d).to(dtype).to(device), r(n, d).to(dtype).to(device),
                torch.randint(-20, V, (n,), generator=g, dtype=torch.int32).to(device)) for _ in range(3)]
    return t, batches


@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
def test_loop_without_copies(cuda, bits, rows):
    import invariant_token_logprobs_lm_amd as itl

    names = ("W", "w_pre", "w_post", "gate")
    weights = []
    for written in (True, False):
        t, batches = _model(cuda, rows=rows)
        grads = {k: torch.full(t[k].shape, float("nan"), dtype=torch.bfloat16 if k == "gate" and rows else torch.float32,
                               device=cuda) for k in names}
        plan = itl.adamw_plan([t[k] for k in names], [grads[k] for k in names], lr=1e-3, state_bits=bits)
        for x, y, targets in batches:
            h, u, r_pre, r_post = itl.residual_norm(x, y, t["w_pre"], w_post=t["w_post"], gate=t["gate"], scale=0.5)
            _, _, _, dH, _ = itl.cross_entropy_grad(u, t["W"], targets, dW=grads["W"])
            out = {k: grads[k] for k in ("w_pre", "w_post", "gate")} if written else {}
            got = itl.residual_norm_backward(dH, None, h, y, t["w_pre"], r_pre, w_post=t["w_post"], rstd_post=r_post,
                                             gate=t["gate"], scale=0.5, **{"d" + k: v for k, v in out.items()})
            for k, v in zip(("w_pre", "w_post", "gate"), got[2:]):
                if written:
                    assert v is grads[k]
                else:
                    grads[k].copy_(v)
            itl.adamw_step(plan, max_norm=1.0)
        weights.append([t[k] for k in names] + [plan.master])
    for a, b in zip(*weights):
        assert torch.equal(a, b) and bool(a.isfinite().all())


def test_column_gradients_given(cuda):
    import invariant_token_logprobs_lm_amd as itl

    t, batches = _model(cuda)
    x, y, _ = batches[0]
    h, u, r_pre, r_post = itl.residual_norm(x, y, t["w_pre"], w_post=t["w_post"], gate=t["gate"])
    du = torch.randn(200, 128, device=cuda)
    call = lambda **kw: itl.residual_norm_backward(du, None, h, y, t["w_pre"], r_pre, w_post=t["w_post"], rstd_post=r_post,
                                                   gate=t["gate"], **kw)
    f = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device=cuda)
    for bad in (dict(dw_pre=f(127)), dict(dw_pre=f(128, dt=torch.bfloat16)), dict(dw_post=f(1, 128)),
                dict(dgate=f(200, 128, dt=torch.bfloat16)), dict(dgate=f(128, dt=torch.bfloat16))):
        with pytest.raises(ValueError):
            call(**bad)
    one = f(128)
    with pytest.raises(itl.ItlError):
        call(dw_pre=one, dw_post=one)
    want = call()
    got = call(dw_pre=f(128), dw_post=f(128), dgate=f(128))
    for a, b in zip(want, got):
        assert torch.equal(a, b)
def test_outputs_without_their_operand_are_refused(cuda):
    import invariant_token_logprobs_lm_amd as itl

    t, batches = _model(cuda)
    x = batches[0][0]
    f = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device=cuda)
    b = f(200, 128, dt=torch.bfloat16)
    with pytest.raises(ValueError, match="h needs y"):
        itl.residual_norm(x, None, t["w_pre"], h=b)
    with pytest.raises(ValueError, match="h needs y"):
        itl.residual_norm_fp8(x, None, t["w_pre"], h=b)
    h, u, r_pre, _ = itl.residual_norm(x, None, t["w_pre"], h=x)  # (h is x either way)
    for kw in (dict(dy=b), dict(dw_post=f(128)), dict(dgate=f(128))):
        with pytest.raises(ValueError, match="needs"):
            itl.residual_norm_backward(b, None, h, None, t["w_pre"], r_pre, **kw)
