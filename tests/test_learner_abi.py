"""Host-side tests of the learner's entry points (no GPU, nothing launched):
argument checks before any device work, workspace sizes, the optimizer's plan
(a host-side layout), and compiled kernels without scratch."""

import ctypes
import os
import struct

import pytest

from test_device_code import _compile, needs_hipcc
from invariant_token_logprobs_lm_amd import build

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
SIZE_MAX = ctypes.c_size_t(-1).value
v = ctypes.c_void_p


@pytest.fixture(scope="module")
def itl():
    import invariant_token_logprobs_lm_amd as itl

    return itl


def test_norm_arguments(itl):
    def f(x=256, y=256, gate=0, stride=0, wpost=0, wpre=256, dt=0, n=4, d=64, scale=1.0, eps=1e-6, h=256, u=256):
        return itl.lib.itl_residual_norm(v(x), v(y), v(gate), stride, v(wpost), v(wpre), dt, n, d, scale, eps, v(h), v(u),
                                         None, None, None)

    assert f(n=0, x=0, y=0, wpre=0, h=0, u=0) == OK
    assert f(n=-1) == INVALID and f(d=0) == INVALID
    assert f(dt=5) == UNSUPPORTED and f(n=1 << 31) == UNSUPPORTED and f(d=(1 << 24) + 1) == UNSUPPORTED
    assert f(eps=0.0) == INVALID and f(eps=float("nan")) == INVALID and f(scale=float("inf")) == INVALID
    assert f(gate=256, stride=32) == INVALID
    assert f(y=0, gate=256) == INVALID and f(y=0, wpost=256) == INVALID
    for name in ("x", "wpre", "h", "u"):
        assert f(**{name: 0}) == INVALID, name
    for name in ("x", "y", "wpre", "h", "u"):
        assert f(**{name: 264}) == INVALID, name       # 8 bytes off where whole vectors are moved
        assert f(**{name: 257}, d=63) == INVALID, name  # no element starts there
    q = itl.lib.itl_residual_norm_fp8
    assert q(v(256), None, None, 0, None, v(256), 0, 4, 64, 1.0, 1e-6, None, v(256), v(256), None, None, None) == UNSUPPORTED
    assert q(v(256), None, None, 0, None, v(256), 0, 4, 128, 1.0, 1e-6, None, v(257), v(256), None, None, None) == INVALID
    assert q(v(256), None, None, 0, None, v(256), 0, 4, 128, 1.0, 1e-6, None, v(256), None, None, None, None) == INVALID


def test_norm_backward_arguments(itl):
    def f(du=256, dud=1, dh=0, h=256, y=256, gate=0, stride=0, wpost=0, rpost=0, dt=0, n=4, d=64, dx=256, dy=256, dg=0,
          dwpre=256, dwpost=0, ws=256, wsb=1 << 30):
        return itl.lib.itl_residual_norm_backward(v(du), dud, v(dh), v(h), v(y), v(gate), stride, v(wpost), v(256), v(256),
                                                  v(rpost), dt, n, d, 1.0, v(dx), v(dy), v(dg), v(dwpre), v(dwpost), v(ws),
                                                  wsb, None)

    assert f(n=-1) == INVALID and f(dt=3) == UNSUPPORTED
    assert f(dud=0, dt=1) == UNSUPPORTED  # bf16 gradients of an fp32 norm
    for name in ("du", "h", "dx", "dy", "dwpre"):
        assert f(**{name: 0}) == INVALID, name
    assert f(gate=256) == INVALID and f(wpost=256, rpost=256) == INVALID  # their gradients' outputs are missing
    assert f(wpost=256, dwpost=256) == INVALID                            # rstd_post is
    assert f(du=260) == INVALID and f(dy=264) == INVALID
    assert f(ws=0) == WORKSPACE and f(wsb=16) == WORKSPACE and f(ws=257) == WORKSPACE
    w = itl.lib.itl_residual_norm_backward_workspace_bytes
    assert w(-1, 64) == SIZE_MAX and w(4, 0) == SIZE_MAX and 0 < w(4, 64) <= w(100000, 64) < 1 << 30


def test_cross_entropy_arguments(itl):
    def f(H=256, W=256, dt=0, n=4, d=64, V=10, y=256, eps=0.0, lam=0.0, red=1, scale=1.0, gd=0, loss=256, tok=256, dH=256,
          dW=256, ws=256, wsb=1 << 40):
        grad = itl.lib.itl_cross_entropy_grad(v(H), v(W), dt, n, d, V, v(y), eps, lam, red, scale, gd, v(loss), v(tok),
                                              None, v(dH), v(dW), v(ws), wsb, None)
        if dH == 256 and dW == 256 and scale == 1.0 and gd == 0 and dt != 1:
            assert itl.lib.itl_cross_entropy(v(H), v(W), dt, n, d, V, v(y), eps, lam, red, v(loss), v(tok), None, v(ws),
                                             wsb, None) == grad
        return grad

    assert f(n=-1) == INVALID and f(d=96) == UNSUPPORTED and f(dt=9) == UNSUPPORTED
    assert f(eps=1.0) == INVALID and f(eps=-0.1) == INVALID and f(eps=float("nan")) == INVALID
    assert f(lam=-1.0) == INVALID and f(lam=float("inf")) == INVALID
    assert f(red=2) == INVALID and f(scale=float("nan")) == INVALID
    assert f(dt=1, gd=0) == UNSUPPORTED and f(gd=4) == UNSUPPORTED
    for name in ("H", "W", "y", "loss", "tok", "dH", "dW"):
        assert f(**{name: 0}) == INVALID, name
    for name in ("H", "W", "dH", "dW"):
        assert f(**{name: 264}) == INVALID, name
    assert f(ws=0) == WORKSPACE and f(wsb=16) == WORKSPACE and f(ws=255) == WORKSPACE
    w = itl.lib.itl_cross_entropy_workspace_bytes
    assert w(0, 64, 10, 0, 1, 0) == 0
    assert w(-1, 64, 10, 0, 0, 0) == SIZE_MAX and w(4, 63, 10, 0, 0, 0) == SIZE_MAX and w(4, 64, 10, 1, 1, 0) == SIZE_MAX
    assert w(4, 64, 10, 0, 0, 0) < w(4, 64, 10, 0, 1, 0) < 1 << 30
    # the logits of one chunk only, whatever the number of tokens
    one, ten = w(16384, 128, 50000, 0, 1, 0), w(163840, 128, 50000, 0, 1, 0)
    assert 16384 * 50000 * 4 < one < ten < one + 163840 * 64 + 50000 * 128 * 4 + (1 << 20)


def _refused_as_shared(itl, status):
    return status == INVALID and "share" in itl.lib.itl_last_error().decode()


def test_shared_memory_is_refused(itl):
    """Outputs over inputs or other outputs (but h over x, dx over dh, row for row)."""
    MB = 1 << 20

    def norm(**over):
        a = dict(x=1, y=2, gate=3, w_post=4, w_pre=5, h=6, u=7, r=8, rp=9)
        at = {k: over.get(k, n * MB) for k, n in a.items()}
        return itl.lib.itl_residual_norm(v(at["x"]), v(at["y"]), v(at["gate"]), 64, v(at["w_post"]), v(at["w_pre"]), 0, 4, 64,
                                         1.0, 1e-6, v(at["h"]), v(at["u"]), v(at["r"]), v(at["rp"]), None)

    for over in (dict(u=MB), dict(u=2 * MB), dict(u=6 * MB), dict(u=3 * MB + 496), dict(u=5 * MB), dict(h=2 * MB),
                 dict(h=MB + 16), dict(r=7 * MB), dict(rp=8 * MB + 12), dict(h=MB, u=MB), dict(h=MB, x=MB, y=MB)):
        assert _refused_as_shared(itl, norm(**over)), over

    def backward(d=64, **over):
        names = ("du", "dh", "h", "y", "gate", "w_post", "w_pre", "r", "rp", "dx", "dy", "dgate", "dw_pre", "dw_post", "ws")
        p = {k: v(over.get(k, (16 + n) * 16 * MB)) for n, k in enumerate(names)}
        return itl.lib.itl_residual_norm_backward(p["du"], 0, p["dh"], p["h"], p["y"], p["gate"], d, p["w_post"], p["w_pre"],
                                                  p["r"], p["rp"], 0, 4, d, 1.0, p["dx"], p["dy"], p["dgate"], p["dw_pre"],
                                                  p["dw_post"], p["ws"], 1 << 30, None)

    at = lambda n: (16 + n) * 16 * MB
    for d in (64, 16384):
        for over in (dict(dx=at(0)), dict(dx=at(2)), dict(dx=at(3)), dict(dy=at(1)), dict(dy=at(3)), dict(dy=at(9)),
                     dict(dx=at(1) + 16), dict(dgate=at(4)), dict(dw_pre=at(6)), dict(dw_post=at(12)), dict(ws=at(0)),
                     dict(dx=at(1), dy=at(1))):
            assert _refused_as_shared(itl, backward(d, **over)), (d, over)

    def entropy(**over):
        names = ("H", "W", "y", "loss", "tok", "lse", "dH", "dW", "ws")
        p = {k: v(over.get(k, (n + 1) * 16 * MB)) for n, k in enumerate(names)}
        return itl.lib.itl_cross_entropy_grad(p["H"], p["W"], 0, 4, 64, 300, p["y"], 0.0, 0.0, 1, 1.0, 0, p["loss"], p["tok"],
                                              p["lse"], p["dH"], p["dW"], p["ws"], 1 << 40, None)

    at = lambda n: (n + 1) * 16 * MB
    for over in (dict(dH=at(0)), dict(dW=at(1)), dict(dW=at(6)), dict(tok=at(2)), dict(lse=at(4)), dict(loss=at(4) + 12),
                 dict(dH=at(1) + 256), dict(ws=at(0))):
        assert _refused_as_shared(itl, entropy(**over)), over

    P, G = 1 << 20, 1 << 30
    for g in (P, P + 198, P - 2, (1 << 22) + 64):
        st = _plan(itl, [(P, G, 100, 0, 0, 0.0), (1 << 22, g, 100, 0, 0, 0.0)])[0]
        assert _refused_as_shared(itl, st), g
    for g in (P + 200, P - 200, (1 << 22) - 200):
        assert _plan(itl, [(P, G, 100, 0, 0, 0.0), (1 << 22, g, 100, 0, 0, 0.0)])[0] == OK


def _plan(itl, tensors):
    T = itl._AdamWTensor
    table = (T * max(1, len(tensors)))(*[T(*t) for t in tensors])
    nb, el = ctypes.c_int64(), ctypes.c_int64()
    st = itl.lib.itl_adamw_plan_sizes(table, len(tensors), ctypes.byref(nb), ctypes.byref(el))
    if st != OK:
        return st, None, None, None
    buf = ctypes.create_string_buffer(max(1, nb.value))
    st = itl.lib.itl_adamw_plan(table, len(tensors), buf, nb.value)
    return st, nb.value, el.value, buf.raw


def test_adamw_plan_layout(itl):
    P, G = 1 << 20, 1 << 30
    st, nb, el, raw = _plan(itl, [(P, G, 10000, 0, 1, 0.5), (1 << 22, G, 0, 0, 0, 0.0), ((1 << 23) + 2, G, 300, 0, 0, 0.0)])
    assert st == OK and nb == 6 * 40 and el == 10240 + 512
    rows = [struct.unpack_from("<QQqiIfi", raw, 40 * i) for i in range(6)]
    assert [r[:4] for r in rows] == [(P + 4096 * i, G + 8192 * i, 2048 * i, 2048 if i < 4 else 1808) for i in range(5)] + [
        ((1 << 23) + 2, G, 10240, 300)]
    assert [r[4] for r in rows] == 5 * [2 | 4] + [0]  # fp32 gradients, whole vectors; the last is misaligned
    assert [r[5] for r in rows] == 5 * [0.5] + [0.0]


def test_adamw_plan_refusals(itl):
    P, G = 1 << 20, 1 << 30
    assert _plan(itl, [])[0] == OK
    for bad, want in (((P, G, -1, 0, 0, 0.0), INVALID), ((0, G, 4, 0, 0, 0.0), INVALID), ((P, 0, 4, 0, 0, 0.0), INVALID),
                      ((P, G, 4, 7, 0, 0.0), UNSUPPORTED), ((P, G, 4, 0, 0, -1.0), INVALID),
                      ((P, G, 4, 0, 0, float("nan")), INVALID), ((P + 1, G, 4, 0, 0, 0.0), INVALID),
                      ((P, G + 2, 4, 0, 1, 0.0), INVALID)):
        assert _plan(itl, [bad])[0] == want, bad
    assert _plan(itl, [(P, G, 100, 0, 0, 0.0), (P + 198, G, 100, 0, 0, 0.0)])[0] == INVALID  # one weight shared
    assert _plan(itl, [(P, G, 100, 0, 0, 0.0), (P + 200, G, 100, 0, 0, 0.0)])[0] == OK       # gradients may be
    assert "share" not in itl.lib.itl_last_error().decode()


def test_adamw_step_arguments(itl):
    def f(plan=256, nb=40, bits=32, m=256, sq=256, ms=0, vs=0, master=0, lr=256, step=256, b1=0.9, b2=0.9, eps=1e-8, mx=1.0,
          ws=256, wsb=1 << 20):
        return itl.lib.itl_adamw_step(v(plan), nb, bits, v(m), v(sq), v(ms), v(vs), v(master), v(lr), v(step), b1, b2, eps, mx,
                                      None, v(ws), wsb, None)

    assert f(nb=41) == INVALID and f(bits=16) == UNSUPPORTED
    assert f(b1=1.0) == INVALID and f(b2=-0.1) == INVALID and f(b1=float("nan")) == INVALID
    assert f(eps=0.0) == INVALID and f(mx=0.0) == INVALID and f(mx=float("nan")) == INVALID
    for name in ("plan", "m", "sq", "lr", "step"):
        assert f(**{name: 0}) == INVALID, name
    assert f(bits=8) == INVALID  # scales missing
    assert f(m=260) == INVALID and f(master=8) == INVALID and f(plan=260) == INVALID
    assert f(ws=0) == WORKSPACE and f(wsb=16) == WORKSPACE and f(ws=255) == WORKSPACE


def test_bindings_refuse_host_tensors(itl):
    import torch

    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        itl.residual_norm(x, x, x[0])
    with pytest.raises(ValueError):
        itl.cross_entropy(x, x, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        itl.adamw_plan([x], [x], lr=0.1)
    with pytest.raises(TypeError):
        itl.residual_norm([1.0], None, x[0])


@needs_hipcc
@pytest.mark.parametrize("src,kernels", [
    ("cross_entropy.hip", ["ce_partial_kernelILi0E", "ce_partial_narrow_kernel", "ce_logits_f32_kernel", "ce_dh_kernelILi0E",
                           "ce_dh_kernelILi1E", "ce_dw_kernelILi0E", "ce_dw_kernelILi1E", "ce_dw_few_kernel"]),
    ("norm.hip", ["norm_"]),
    ("adamw.hip", ["adamw_"]),
])
def test_kernels_have_no_scratch(tmp_path, src, kernels):
    import re

    r = _compile(os.path.join(build.CSRC, src), str(tmp_path),
                 ("-c", "-o", str(tmp_path / "x.o"), "-Rpass-analysis=kernel-resource-usage"))
    seen, current = set(), None
    for line in r.stderr.splitlines():
        m = re.search(r"Function Name: (\S+)", line)
        if m:
            current = m.group(1)
        m = re.search(r"ScratchSize \[bytes/lane\]: (\d+)", line)
        if m and current:
            for k in kernels:
                if k in current:
                    assert int(m.group(1)) == 0, (current, line)
                    seen.add(k)
    assert seen == set(kernels)


@needs_hipcc
def test_inline_asm_loads_write_lds_only(tmp_path):
    import test_device_code

    test_device_code.test_inline_asm_loads_write_lds_only(tmp_path, "cross_entropy.hip")
