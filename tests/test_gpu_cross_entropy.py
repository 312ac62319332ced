"""The vocabulary cross entropy and its gradient against the 64-bit form:
both head types and gradient types, one token to several row blocks, tiny and
ragged vocabularies, masks that leave some, one or no token, smoothing and
z-loss; then invariance, repeated targets, chunks and replayed graphs.

Tolerances, from the arithmetic: a logit's error is at most
dz = (d / 16 + 8) half steps of fp32 of sum |H W| (d products, added in runs
of 16 or more by the matrix cores); the losses inherit at most 2 dz plus a
few steps of their size. A gradient's entry G is off by at most
half_step(head type) + 2 dz + 8 steps of its terms; the contractions add one
step per addition, and a 16-bit result half a step of its own.
"""

import pytest
import torch

import learner_refs as R
from helpers import same_bits, say

pytestmark = pytest.mark.gpu


def _itl():
    import invariant_token_logprobs_lm_amd as itl

    return itl


def _head(n, d, V, dtype, seed, device, mask="some"):
    g = torch.Generator().manual_seed(seed)
    H = torch.randn(n, d, generator=g).to(dtype)
    W = (torch.randn(V, d, generator=g) * 0.1).to(dtype)
    y = torch.randint(0, V, (n,), generator=g, dtype=torch.int32)
    if mask == "some":
        y[torch.rand(n, generator=g) < 0.3] = -100
    elif mask == "none left":
        y[:] = -100
    elif mask == "one left":
        y[: n - 1] = V  # ids past the vocabulary do not count either
    return H.to(device), W.to(device), y.to(device)


def _check(got, H, W, y, grad_dtype, **kw):
    loss, token, lse, dH, dW = got
    n, d = H.shape
    V = W.shape[0]
    want = R.cross_entropy(R.f64(H), R.f64(W), y, **kw)
    dz = (d / 16 + 8) * R.EPS24 * want["mag_z"]
    lam = kw.get("z_weight", 0.0)
    live = want["lse"] != 0
    size = 1 + want["lse"].abs() + want["mag_z"] * 2.0 ** -10
    tol = (2 * dz * (1 + 2 * lam * want["lse"].abs()) + 32 * R.EPS24 * size * (1 + lam * want["lse"].abs())) * live
    assert bool(((R.f64(token) - want["token_loss"]).abs() <= tol).all())
    assert bool(((R.f64(lse) - want["lse"]).abs() <= 2 * tol).all())
    N = max(1, int(live.sum())) if kw.get("mean", True) else 1
    assert abs(float(loss) - float(want["loss"])) <= float(tol.sum()) / N + 2 * R.EPS24 * abs(float(want["loss"]))
    if dH is None:
        return
    entry = R.half_step(H.dtype) + 2 * float(dz.max()) + 16 * R.EPS24
    for name, t, adds in (("dH", dH, V), ("dW", dW, n)):
        assert t.dtype == grad_dtype
        # with a 16-bit head the one-hot entry p - (1 - e) may cancel against nothing larger than 1 + p:
        # its terms are within 3 times its unit, which every magnitude below holds once per token
        bound = (entry + adds * R.EPS24) * (want["mag_" + name] + _terms(name, H, W, y, want, kw))
        bound = bound + R.half_step(grad_dtype) * want[name].abs()
        assert bool(((R.f64(t) - want[name]).abs() <= bound).all()), name


def _terms(name, H, W, y, want, kw):
    """Magnitude of the parts of G at the targets: (p + 1) units of the row of W, or of H."""
    V = W.shape[0]
    t = y.cpu().long()
    live = (t >= 0) & (t < V)
    N = max(1, int(live.sum())) if kw.get("mean", True) else 1
    unit = abs(kw.get("grad_scale", 1.0)) / N * (2 + 2 * kw.get("z_weight", 0.0) * want["lse"].abs())
    t = t.clamp(0, V - 1)
    if name == "dH":
        return (unit * live)[:, None] * R.f64(W).abs()[t]
    out = torch.zeros(V, H.shape[1], dtype=torch.float64)
    return out.index_add_(0, t, (unit * live)[:, None] * R.f64(H).abs())


CASES = [  # n, d, V, mask
    (1, 64, 1, "all"), (1, 64, 300, "all"), (2, 128, 255, "some"), (63, 64, 256, "some"), (64, 192, 257, "all"),
    (65, 64, 1000, "one left"), (129, 128, 511, "some"), (256, 64, 4099, "some"), (300, 320, 3000, "none left"),
    (700, 256, 70000, "some"), (513, 512, 2049, "some"),
]


@pytest.mark.parametrize("dtype,grad", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                        (torch.float32, torch.float32)])
@pytest.mark.parametrize("n,d,V,mask", CASES)
def test_loss_and_gradient(cuda, n, d, V, mask, dtype, grad):
    itl = _itl()
    for kw in ({}, {"smoothing": 0.1, "z_weight": 1e-3, "mean": False, "grad_scale": -0.5}):
        say("cross entropy", n, d, V, mask, dtype, grad, kw)
        H, W, y = _head(n, d, V, dtype, n + d + V, cuda, mask)
        args = dict(label_smoothing=kw.get("smoothing", 0.0), z_weight=kw.get("z_weight", 0.0),
                    reduction="mean" if kw.get("mean", True) else "sum")
        got = itl.cross_entropy_grad(H, W, y, grad_scale=kw.get("grad_scale", 1.0), grad_dtype=grad, **args)
        _check(got, H, W, y, grad, **kw)
        alone = itl.cross_entropy(H, W, y, **args)
        _check(alone + (None, None), H, W, y, grad, **kw)
        for a, b in zip(alone, got):  # the loss has the same bits with and without its gradient
            assert same_bits(a, b)


# dW's tiles by the number of tokens and tiles: whole (walks of one and of
# two), its tokens split (one token left: most splits are empty), and dH's
# vocabulary over as many workgroups as one block of tokens takes
SIZES = [
    (1100, 1024, 17000, "some"), (1100, 2048, 70000, "all"), (4030, 256, 1330, "some"), (2100, 320, 300, "one left"),
    (1025, 64, 700, "all"), (3, 192, 70000, "some"), (200, 128, 40000, "some"),
]


@pytest.mark.parametrize("dtype,grad", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                        (torch.float32, torch.float32)])
@pytest.mark.parametrize("n,d,V,mask", SIZES)
def test_how_the_gradients_are_split(cuda, n, d, V, mask, dtype, grad):
    itl = _itl()
    say("cross entropy", n, d, V, mask, dtype, grad)
    H, W, y = _head(n, d, V, dtype, n + d + V, cuda, mask)
    H *= 0.25  # (logits that leave several ids some probability at these widths)
    got = itl.cross_entropy_grad(H, W, y, grad_dtype=grad, label_smoothing=0.1)
    _check(got, H, W, y, grad, smoothing=0.1)
    again = itl.cross_entropy_grad(H, W, y, grad_dtype=grad, label_smoothing=0.1)
    for a, b in zip(got, again):
        assert same_bits(a, b)


def test_agrees_with_the_logprob(cuda):
    """Without smoothing and z-loss a token's loss is minus its logprob, bit for bit."""
    itl = _itl()
    for n in (1, 64, 100, 700):
        H, W, y = _head(n, 256, 5000, torch.bfloat16, n, cuda, "all")
        _, token, lse = itl.cross_entropy(H, W, y)
        lp, ls = itl.lmhead_logprob(H, W, y)
        assert same_bits(token, -lp) and same_bits(lse, ls)


def test_tokens_do_not_depend_on_the_batch(cuda):
    itl = _itl()
    H, W, y = _head(600, 192, 3001, torch.bfloat16, 5, cuda, "some")
    _, token, lse = itl.cross_entropy(H, W, y, label_smoothing=0.1, z_weight=1e-3)
    for rows in ([3], list(range(40, 140)), list(range(599, 300, -1))):
        i = torch.tensor(rows, device=cuda)
        _, t1, l1 = itl.cross_entropy(H[i], W, y[i], label_smoothing=0.1, z_weight=1e-3)
        assert same_bits(t1, token[i]) and same_bits(l1, lse[i])


@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
def test_every_token_the_same_target(cuda, grad):
    """One row of dW takes every token's one-hot term."""
    itl = _itl()
    H, W, _ = _head(400, 128, 600, torch.bfloat16, 2, cuda, "all")
    y = torch.full((400,), 599, dtype=torch.int32, device=cuda)
    _check(itl.cross_entropy_grad(H, W, y, grad_dtype=grad), H, W, y, grad)


@pytest.mark.parametrize("dtype,grad", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                        (torch.float32, torch.float32)])
def test_several_chunks(cuda, dtype, grad):
    """More tokens than one chunk of the workspace; the mask puts every
    counted token in the first, or spreads them."""
    itl = _itl()
    n = 16384 + 300
    for mask in ("spread", "few"):
        H, W, y = _head(n, 64, 700, dtype, 1, cuda, "some")
        if mask == "few":
            y[50:] = -1
        _check(itl.cross_entropy_grad(H, W, y, grad_dtype=grad), H, W, y, grad)


def test_sharp_and_flat_logits(cuda):
    """Logits of hundreds: a probability of one, others of zero; and a flat row."""
    itl = _itl()
    H, W, y = _head(80, 64, 900, torch.bfloat16, 6, cuda, "all")
    H[:40] *= 200.0
    H[40] = 0
    _check(itl.cross_entropy_grad(H, W, y, grad_dtype=torch.float32), H, W, y, torch.float32)


def test_bad_rows_stay_their_own(cuda):
    """A NaN row that does not count changes nothing; one that counts spoils its own loss."""
    itl = _itl()
    H, W, y = _head(300, 64, 500, torch.bfloat16, 8, cuda, "all")
    y[7] = -100
    H[7] = 0
    want = itl.cross_entropy_grad(H, W, y)
    H[7] = float("nan")
    got = itl.cross_entropy_grad(H, W, y)
    for a, b in zip(want, got):
        assert same_bits(a, b)
    H[9] = float("nan")
    _, token, _ = itl.cross_entropy(H, W, y)
    keep = torch.arange(300, device=cuda) != 9
    assert same_bits(token[keep], want[1][keep]) and bool(token[9].isnan())


def test_run_to_run_and_dirty_memory(cuda):
    """Results do not depend on what the workspace and the outputs held."""
    itl = _itl()
    H, W, y = _head(777, 256, 9001, torch.bfloat16, 3, cuda, "some")
    for grad in (torch.bfloat16, torch.float32):
        need = itl.cross_entropy_workspace_bytes(777, 256, 9001, torch.bfloat16, grad)
        got = []
        for fill in (0, 255, 127):
            ws = torch.full((need,), fill, dtype=torch.uint8, device=cuda)
            dH = torch.full((777, 256), float("nan"), dtype=grad, device=cuda)
            dW = torch.full((9001, 256), float("nan"), dtype=grad, device=cuda)
            got.append(itl.cross_entropy_grad(H, W, y, grad_dtype=grad, label_smoothing=0.1, dH=dH, dW=dW, workspace=ws))
        for other in got[1:]:
            for a, b in zip(got[0], other):
                assert torch.equal(a, b)


def test_nothing_and_refusals(cuda):
    itl = _itl()
    H, W, y = _head(4, 64, 100, torch.bfloat16, 1, cuda, "all")
    loss, token, lse, dH, dW = itl.cross_entropy_grad(H[:0], W, y[:0])
    assert float(loss) == 0.0 and token.numel() == 0 and not bool(dW.any())
    bad = [
        (ValueError, lambda: itl.cross_entropy(H, W.float(), y)),
        (ValueError, lambda: itl.cross_entropy(H, W, y.long())),
        (ValueError, lambda: itl.cross_entropy(H, W, y[:3])),
        (ValueError, lambda: itl.cross_entropy(H, W, y, reduction="none")),
        (ValueError, lambda: itl.cross_entropy_grad(H.float(), W.float(), y, grad_dtype=torch.bfloat16)),
        (ValueError, lambda: itl.cross_entropy_grad(H, W, y, dW=torch.empty(99, 64, device=cuda))),
        (itl.ItlError, lambda: itl.cross_entropy(H, W, y, label_smoothing=1.0)),
        (itl.ItlError, lambda: itl.cross_entropy(H, W, y, z_weight=-1.0)),
        (itl.ItlError, lambda: itl.cross_entropy_grad(H, W, y, grad_scale=float("inf"))),
        (itl.ItlError, lambda: itl.cross_entropy(H[:, :32].contiguous(), W[:, :32].contiguous(), y)),
        (itl.ItlError, lambda: itl.cross_entropy(H, W, y, workspace=torch.empty(16, dtype=torch.uint8, device=cuda))),
    ]
    for error, call in bad:
        with pytest.raises(error):
            call()


@pytest.mark.parametrize("n,dtype,grad", [(500, torch.bfloat16, torch.bfloat16), (500, torch.bfloat16, torch.float32),
                                          (70, torch.bfloat16, torch.bfloat16), (300, torch.float32, torch.float32),
                                          (2500, torch.bfloat16, torch.bfloat16), (2500, torch.bfloat16, torch.float32),
                                          (2500, torch.float32, torch.float32)])
def test_replay(cuda, n, dtype, grad):
    """Another mask at each replay: how many tokens count is not fixed at the capture."""
    itl = _itl()
    H, W, y = _head(n, 128, 3000, dtype, 4, cuda, "some")
    other = y.flip(0).contiguous()
    other[: n // 2] = -100
    ids = y.clone()
    ws = torch.empty(itl.cross_entropy_workspace_bytes(n, 128, 3000, dtype, grad), dtype=torch.uint8, device=cuda)
    call = lambda t: itl.cross_entropy_grad(H, W, t, grad_dtype=grad, label_smoothing=0.1, workspace=ws)
    want = [[a.clone() for a in call(t)] for t in (y, other)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(ids)
    for rep in range(4):
        ids.copy_((y, other)[rep % 2])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want[rep % 2], out):
            assert torch.equal(a, b), rep
        call(other)
        torch.cuda.synchronize()


def test_two_calls_at_once(cuda):
    """Calls on two streams, each with its own workspace, while neither has ended."""
    itl = _itl()
    calls = []
    for n, V, dtype in ((2500, 3000, torch.bfloat16), (40, 60000, torch.bfloat16), (500, 2000, torch.float32)):
        H, W, y = _head(n, 256, V, dtype, n, cuda, "some")
        calls.append(lambda H=H, W=W, y=y: itl.cross_entropy_grad(H, W, y, grad_dtype=H.dtype, label_smoothing=0.1))
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(device=cuda) for _ in calls]
    got = []
    for _ in range(3):
        for s, c in zip(streams, calls):
            with torch.cuda.stream(s):
                got.append(c())
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        for a, b in zip(want[i % len(calls)], out):
            assert same_bits(a, b)
