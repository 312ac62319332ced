"""What an AdamW plan holds and what may be done to it between steps: the
learning rate and the count by assignment, everything else fixed; tensors that
have moved; autograd's view of updated weights; states that share memory."""

import copy
import pickle

import pytest
import torch

from helpers import same_bits

pytestmark = pytest.mark.gpu


def _itl():
    import invariant_token_logprobs_lm_amd as itl

    return itl


def _tensors(device, seed=3, sizes=(5000, 300), dtypes=(torch.bfloat16, torch.float32)):
    g = torch.Generator().manual_seed(seed)
    p = [(torch.randn(n, generator=g) * 0.1).to(t).to(device) for n, t in zip(sizes, dtypes)]
    return p, [torch.randn(n, generator=g).to(device) for n in sizes]


@pytest.mark.parametrize("default", [torch.bfloat16, torch.float16, torch.float64])
def test_rate_is_fp32_whatever_the_default_type(cuda, default):
    itl = _itl()
    p, g = _tensors(cuda)
    q, h = _tensors(cuda)
    want = itl.adamw_plan(q, h, lr=3e-4)
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        plan = itl.adamw_plan(p, g, lr=3e-4)
        assert plan.lr.dtype == torch.float32 and same_bits(plan.lr, want.lr)
        norm = itl.adamw_step(plan, max_norm=1.0)
    finally:
        torch.set_default_dtype(before)
    assert same_bits(norm, itl.adamw_step(want, max_norm=1.0))
    assert torch.equal(p[0], q[0]) and same_bits(p[1], q[1])


@pytest.mark.parametrize("bits", [32, 8])
def test_rate_and_count_are_assigned_into_the_plans_tensors(cuda, bits):
    itl = _itl()
    p, g = _tensors(cuda)
    q, h = _tensors(cuda)
    plan = itl.adamw_plan(p, g, lr=1e-2, state_bits=bits)
    lr, step = plan.lr, plan.step
    plan.lr = 5e-6
    assert plan.lr is lr and float(lr) == float(torch.tensor(5e-6))
    plan.lr = torch.tensor(2e-3, device=cuda, dtype=torch.float64)
    assert plan.lr is lr and lr.dtype == torch.float32 and float(lr) == float(torch.tensor(2e-3))
    plan.lr *= 0.5
    plan.step = 7
    plan.step += 2
    assert plan.lr is lr and plan.step is step and int(step) == 9
    for bad in (torch.zeros(2, device=cuda), [0.1, 0.2], "rate", None):
        with pytest.raises((TypeError, ValueError)):
            plan.lr = bad
    other = itl.adamw_plan(q, h, lr=lr.clone(), step=step.clone(), state_bits=bits)
    itl.adamw_step(plan)
    itl.adamw_step(other)
    assert int(plan.step) == 10 and torch.equal(p[0], q[0]) and same_bits(p[1], q[1])


@pytest.mark.parametrize("bits", [32, 8])
def test_the_rest_of_a_plan_is_fixed(cuda, bits):
    itl = _itl()
    p, g = _tensors(cuda)
    plan = itl.adamw_plan(p, g, lr=1e-2, state_bits=bits)
    names = [n for n in type(plan).__slots__ if n not in ("lr", "step")]
    for name in names:
        held = getattr(plan, name)
        with pytest.raises(AttributeError):
            setattr(plan, name, held.clone() if isinstance(held, torch.Tensor) else 0)
        assert getattr(plan, name) is held
    for name in names + ["lr", "step"]:
        with pytest.raises(AttributeError):
            delattr(plan, name)
    for seq in (plan.params, plan.grads, plan.offsets):
        with pytest.raises(TypeError):
            seq[0] = seq[1]
    plan.exp_avg *= 0  # (in place: the same tensor)
    for make in (copy.copy, copy.deepcopy, pickle.dumps):
        with pytest.raises(TypeError):
            make(plan)
    itl.adamw_step(plan)


@pytest.mark.parametrize("which", ["params", "grads", "exp_avg", "exp_avg_sq", "master", "lr", "step"])
def test_a_tensor_that_moved_is_refused(cuda, which):
    itl = _itl()
    p, g = _tensors(cuda)
    plan = itl.adamw_plan(p, g, lr=1e-2)
    t = getattr(plan, which)
    t = t[1] if isinstance(t, tuple) else t
    kept, before = t.data, [x.clone() for x in (*p, plan.exp_avg, plan.step)]
    t.data = kept.clone()
    with pytest.raises(ValueError, match=which):
        itl.adamw_step(plan)
    t.data = kept
    for a, b in zip((*p, plan.exp_avg, plan.step), before):
        assert torch.equal(a, b)
    itl.adamw_step(plan)
    assert int(plan.step) == 1


def test_freed_storage_is_refused(cuda):
    itl = _itl()
    p, g = _tensors(cuda)
    plan = itl.adamw_plan(p, g, lr=1e-2)
    g[0].untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="grads"):
        itl.adamw_step(plan)


def test_autograd_sees_that_the_weights_changed(cuda):
    itl = _itl()
    p, g = _tensors(cuda)
    w = p[1].requires_grad_()
    plan = itl.adamw_plan(p, g, lr=1e-2)
    x = torch.ones_like(w, requires_grad=True)
    y = (x * w).sum()  # saves w
    version = p[0]._version, w._version
    itl.adamw_step(plan)
    assert p[0]._version > version[0] and w._version > version[1]
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    (x * w).sum().backward()
    assert same_bits(x.grad, w.detach())


def test_states_that_share_memory_are_refused(cuda):
    itl = _itl()
    p, g = _tensors(cuda, dtypes=(torch.bfloat16, torch.bfloat16))
    total = 5120 + 512
    f32 = lambda n=total: torch.zeros(n, device=cuda)
    u8 = lambda n=total: torch.zeros(n, dtype=torch.uint8, device=cuda)
    s, long = f32(), f32(2 * total)
    scales = f32(2 * total // 256)
    w32 = f32()
    bad = [
        dict(exp_avg=s, exp_avg_sq=s), dict(exp_avg=s, master=s), dict(exp_avg_sq=long[:total], master=long[256:256 + total]),
        dict(exp_avg=s, lr=s[5:6]), dict(exp_avg=s, step=s.view(torch.int64)[9:10]),
        dict(state_bits=8, exp_avg=u8(), exp_avg_scale=scales[:total // 256], exp_avg_sq_scale=scales[8:8 + total // 256]),
        dict(state_bits=8, exp_avg=s.view(torch.uint8)[:total], exp_avg_sq=s.view(torch.uint8)[1024:1024 + total]),
    ]
    for kw in bad:
        with pytest.raises(ValueError, match="share"):
            itl.adamw_plan(p, g, **{"lr": 0.1, **kw})
    with pytest.raises(ValueError, match="share"):  # a state over the weights, or over a gradient
        itl.adamw_plan([w32[:5000]], [g[0]], lr=0.1, exp_avg=w32[:5120])
    with pytest.raises(ValueError, match="share"):
        itl.adamw_plan([p[0]], [w32[:5000]], lr=0.1, exp_avg_sq=w32[:5120])
    plan = itl.adamw_plan(p, g, lr=0.1, exp_avg=long[:total], exp_avg_sq=long[total:], master=s)  # neighbours do not
    itl.adamw_step(plan)
    assert bool(s[:5000].any())
