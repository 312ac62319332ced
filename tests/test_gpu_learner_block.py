"""The learner's block operators together, as a training step runs them: a
block's output projection in 8 bits, dropout, gate, residual and norms, the head's
loss and gradient, the way back through all of it with both of the projection's
gradients, and one AdamW step. Against the same step in 64 bits on the same codes,
then eagerly and as a replayed graph, whole and in pieces.

Tolerance: with fp32 weights and activations each result is within 1e-4 of its
norm of the 64-bit one (d + f + V + n additions of one half step each, 2^-24, on sums
whose terms are at most ten times the result: below 3e-5 at these sizes).
"""

import pytest
import torch

import block_refs as B
import learner_refs as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def itl():
    import invariant_token_logprobs_lm_amd as itl

    return itl


def _model(n, d, f, V, dtype, device, seed=3):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    t = {"act": r(n, f), "x": r(n, d), "P": f ** -0.5 * r(d, f), "w_pre": 1 + 0.1 * r(d), "w_post": 1 + 0.1 * r(d),
         "gate": 0.5 + 0.1 * r(d), "W": 0.05 * r(V, d)}
    t = {k: v.to(dtype).to(device) for k, v in t.items()}
    y = torch.randint(0, V, (n,), generator=g, dtype=torch.int32)
    y[: n // 4] = -100
    return t, y.to(device)


class _Step:
    """One step over the projection P, the norms and the head W; the seed is raised first."""

    def __init__(self, itl, t, y):
        self.itl, self.t, self.y = itl, t, y
        names = ("P", "W", "w_pre", "w_post", "gate")
        self.grads = {k: torch.zeros(t[k].shape, dtype=torch.float32, device=y.device) for k in names}
        self.plan = itl.adamw_plan([t[k] for k in names], list(self.grads.values()), lr=1e-3, weight_decay=0.01)
        self.seed = torch.tensor([41], dtype=torch.int64, device=y.device)
        self.kw = {"w_post": t["w_post"], "gate": t["gate"], "scale": 0.5, "dropout": itl.Dropout(0.2, self.seed, site=1)}

    def forward(self, act, x, kw):
        itl, t = self.itl, self.t
        q, s, _, _ = itl.quantize_blocks_fp8(act)
        pq, ps, pt, pts = itl.quantize_tiles_fp8(t["P"], columns=True)
        y = itl.matmul_fp8_blocks(q, s, pq, ps, out_dtype=x.dtype)
        return (y, *itl.residual_norm(x, y, t["w_pre"], **kw)), (pt, pts)

    def __call__(self):
        itl, t, g = self.itl, self.t, self.grads
        self.seed.add_(1)
        (y, h, u, r_pre, r_post), (pt, pts) = self.forward(t["act"], t["x"], self.kw)
        loss, _, _, dH, _ = itl.cross_entropy_grad(u, t["W"], self.y, z_weight=1e-4, dW=g["W"])
        dx, dy, *_ = itl.residual_norm_backward(dH, None, h, y, t["w_pre"], r_pre, rstd_post=r_post, dw_pre=g["w_pre"],
                                                dw_post=g["w_post"], dgate=g["gate"], **self.kw)
        dq, ds, dt, dts = itl.quantize_blocks_fp8(dy, columns=True)
        _, _, at, ats = itl.quantize_tiles_fp8(t["act"], rows=False, columns=True)
        dact = itl.matmul_fp8_blocks(dq, ds, pt, pts, out_dtype=t["act"].dtype)
        itl.matmul_fp8_blocks(dt, dts, at, ats, out_dtype=torch.float32, out=g["P"])
        norm = itl.adamw_step(self.plan, max_norm=1.0)
        return {"loss": loss, "y": y, "h": h, "u": u, "dx": dx, "dy": dy, "dact": dact, "norm": norm}


def _near(got, want, rel=1e-4):
    got = R.f64(got)
    assert got.shape == want.shape and float((got - want).norm()) <= rel * float(want.norm())


def test_step_against_64_bits(cuda, itl):
    n, d, f = 300, 192, 700
    t, y = _model(n, d, f, 2000, torch.float32, cuda)
    c = {k: R.f64(v) for k, v in t.items()}
    act, P = t["act"].cpu(), t["P"].cpu()
    step = _Step(itl, t, y)
    got = step()
    Y, _ = B.product(*B.blocks(act), *B.tiles(P))
    keep = B.keep_factors(n, d, 0.2, 42, site=1)
    h, _, r_post = R.norm_forward(c["x"], Y, c["w_pre"], c["w_post"], c["gate"] * keep, 0.5)
    u, r_pre = R.norm_out(h, c["w_pre"])
    ce = R.cross_entropy(u, c["W"], y, z_weight=1e-4)
    out, _ = R.norm_backward(ce["dH"], None, h, Y, c["w_pre"], r_pre, c["w_post"], r_post, c["gate"] * keep, 0.5)
    _near(got["y"], Y)
    _near(got["h"], h)
    _near(got["u"], u)
    assert abs(float(got["loss"]) - float(ce["loss"])) <= 1e-5 * float(ce["loss"])
    _near(got["dx"], out["dx"])
    _near(got["dy"], out["dy"])
    _near(step.grads["W"], ce["dW"])
    _near(step.grads["w_pre"], out["dw_pre"])
    _near(step.grads["w_post"], out["dw_post"])
    dgate = 0.5 * (Y * r_post[:, None] * c["w_post"]) * keep * out["dx"]
    _near(step.grads["gate"], dgate.sum(0))
    # the projection's gradients, from the codes of the gradient that arrived
    dy = got["dy"].cpu()
    _near(got["dact"], B.product(*B.blocks(dy), *B.tiles(P.t().contiguous()))[0])
    _near(step.grads["P"], B.product(*B.blocks(dy.t().contiguous()), *B.tiles(act.t().contiguous()))[0])
    want = float(torch.sqrt(sum((R.f64(g) ** 2).sum() for g in step.grads.values())))
    assert abs(float(got["norm"]) - want) <= 1e-4 * want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_captured_step_replays_like_the_eager_one(cuda, itl, dtype):
    (te, y), (tc, _) = _model(200, 128, 384, 1500, dtype, cuda), _model(200, 128, 384, 1500, dtype, cuda)
    eager, captured = _Step(itl, te, y), _Step(itl, tc, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = captured()
    masks = set()
    for rep in range(4):
        want = eager()
        graph.replay()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(out[k], want[k]), (rep, k)
        for k in eager.grads:
            assert torch.equal(te[k], tc[k]), (rep, k)
        masks.add(int((out["h"] == tc["x"]).sum()))  # (what is dropped leaves the stream as it was)
    assert int(captured.seed) == 45 and len(masks) > 1


def test_forward_in_pieces_has_the_bits_of_the_whole(cuda, itl):
    t, y = _model(301, 256, 640, 1500, torch.bfloat16, cuda)
    step = _Step(itl, t, y)
    whole, _ = step.forward(t["act"], t["x"], step.kw)
    for a, b in ((0, 1), (1, 40), (40, 301)):
        kw = {**step.kw, "dropout": step.kw["dropout"]._replace(first_row=a)}
        piece, _ = step.forward(t["act"][a:b].contiguous(), t["x"][a:b].contiguous(), kw)
        for p, w in zip(piece, whole):
            assert torch.equal(p, w[a:b])


def test_rows_from_the_norm_feed_the_product(cuda, itl):
    """residual_norm_blocks_fp8's codes and the quantiser's of the fp32 u: one product."""
    t, _ = _model(77, 256, 640, 10, torch.float32, cuda)
    y = torch.randn(77, 256, device=cuda)
    drop = itl.Dropout(0.1, torch.tensor([7], dtype=torch.int64, device=cuda))
    h, q, s, _, _ = itl.residual_norm_blocks_fp8(t["x"], y, t["w_pre"], dropout=drop)
    _, u, _, _ = itl.residual_norm(t["x"], y, t["w_pre"], dropout=drop)
    q2, s2, _, _ = itl.quantize_blocks_fp8(u)
    pq, ps, _, _ = itl.quantize_tiles_fp8(t["P"].t().contiguous())
    a = itl.matmul_fp8_blocks(q, s, pq, ps, out_dtype=torch.float32)
    assert torch.equal(a, itl.matmul_fp8_blocks(q2, s2, pq, ps, out_dtype=torch.float32))
    _near(a, R.f64(u) @ R.f64(t["P"]), 0.05)  # (codes: 2.6 % of each operand)
