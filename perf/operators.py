"""The learner's operators around the LM head, as measured cases.

Three families, used together in one training step: the norms around a block
with its gate and residual scale (they make the head's input and take its
gradient back), the cross entropy over the vocabulary with its gradient, and
the AdamW step over many tensors. Each case runs either in its plain form
(elementary torch operations in float32) or, with ``own`` set, through the
package's entry points.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
RESIDUAL_SCALE = 0.5
BETAS = (0.9, 0.95)
ADAM_EPS = 1e-8
WEIGHT_DECAY = 0.1
MAX_NORM = 1.0
LR = 1e-5
BLOCK = 256  # flat state layout: every tensor starts at a multiple of this; one scale per block of 8-bit state

_DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token of a decode step entering the head: latency
        _norm("norm, one decode token", "forward", 1, 2560, "bf16", False, "none"),
        # a prompt batch through a sandwich-norm block with a layer scale
        _norm("norm, prompt batch", "forward", 16384, 2560, "bf16", True, "vector"),
        # rows for an FP8 head
        _norm("norm, rows for the FP8 head", "forward_fp8", 4096, 7168, "bf16", False, "none"),
        # the backward of the last block's norms, fed with the head's fp32 dH
        _norm("norm, backward", "backward", 16384, 2560, "bf16", True, "vector"),
        # a small fp32 model of odd width with a gate for each token
        _norm("norm, odd fp32 backward", "backward", 777, 1001, "fp32", True, "rows"),
        # the smallest head: fp32 training of a toy model
        _loss("loss, tiny fp32 head", True, 177, 128, 1024, "fp32", 0.25, 0.0, 0.0),
        # scoring a few tokens (a validation batch of one short answer)
        _loss("loss, scoring 64 tokens", False, 64, 1536, 151936, "bf16", 0.0, 0.0, 0.0),
        # supervised warm start with masked prompts and a z-loss
        _loss("loss and gradient, 4B head", True, 4096, 2560, 151936, "bf16", 0.25, 0.0, 1e-4),
        # the same on the widest head, with label smoothing
        _loss("loss and gradient, MoE head", True, 2500, 7168, 129280, "bf16", 0.125, 0.1, 0.0),
        # the tiny head's weights and two gains: launches count
        _step("step, tiny fp32 model", 3, 131072, "fp32", "fp32", 32, False),
        # all blocks of a small model, bf16 weights with fp32 masters, clipped
        _step("step, many tensors", 96, 1536 * 8960, "bf16", "bf16", 32, True),
        # the 4B head's weights alone, states in 8 bits, gradient as the head's backward gives it
        _step("step, 4B head, 8-bit states", 1, 151936 * 2560, "bf16", "fp32", 8, True),
    ]


def draw(rng):
    kind = rng.choice(["norm", "loss", "step"])
    if kind == "norm":
        what = rng.choice(["forward", "forward_fp8", "backward"])
        width = 128 * rng.randint(1, 56) if what == "forward_fp8" else rng.choice([64 * rng.randint(1, 112), rng.randint(48, 4000)])
        rows = min(_log(rng, 1, 16384), 16384 * 2560 // width)
        return _norm(None, what, rows, width, rng.choice(["bf16", "bf16", "fp32"]), rng.random() < 0.5,
                     rng.choice(["none", "vector", "rows"]))
    if kind == "loss":
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        width, vocab = 64 * rng.randint(1, 80), _log(rng, 300, 151936)
        most = 4096 * 2560 * 151936 // (4 if dtype == "fp32" else 1)
        tokens = max(1, min(_log(rng, 1, 5000), most // (width * vocab)))
        return _loss(None, rng.random() < 0.7, tokens, width, vocab, dtype, rng.choice([0.0, 0.25, 0.5]),
                     rng.choice([0.0, 0.0, 0.1]), rng.choice([0.0, 1e-4]))
    largest = _log(rng, 500, 30_000_000)
    tensors = max(1, min(_log(rng, 1, 200), 300_000_000 // largest))
    param = rng.choice(["bf16", "fp32"])
    return _step(None, tensors, largest, param, rng.choice(["fp32", param]), rng.choice([32, 8]), rng.random() < 0.5)


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _named(name, case):
    return case if name is None else {"name": name, **case}


def _norm(name, what, rows, width, dtype, post, gate):
    return _named(name, {"operator": "norm", "pass": what, "rows": rows, "width": width, "dtype": dtype, "post": post, "gate": gate})


def _loss(name, gradient, tokens, width, vocab, dtype, masked, smoothing, z_weight):
    return _named(name, {"operator": "loss", "gradient": gradient, "tokens": tokens, "width": width, "vocab": vocab,
                         "dtype": dtype, "masked": masked, "smoothing": smoothing, "z_weight": z_weight})


def _step(name, tensors, largest, param, grad, state_bits, clip):
    return _named(name, {"operator": "step", "tensors": tensors, "largest": largest, "param": param, "grad": grad,
                         "state_bits": state_bits, "clip": clip})


def _prompts(case):
    """(period, prompt): of every `period` tokens the first `prompt` are not counted."""
    period = min(512, case["tokens"])
    return period, int(period * case["masked"])


def _counted(case):
    period, prompt = _prompts(case)
    full, rest = divmod(case["tokens"], period)
    return full * (period - prompt) + max(0, rest - prompt)


def _sizes(case):
    """Matrices and vectors of falling sizes, ragged."""
    return [max(1, (case["largest"] >> (2 * (i % 7))) - (37 * i) % 101) for i in range(case["tensors"])]


def _layout(case):
    sizes, at, offsets = _sizes(case), 0, []
    for n in sizes:
        offsets.append(at)
        at += -(-n // BLOCK) * BLOCK
    return sizes, offsets, at


def work(case):
    if case["operator"] == "norm":
        n, d, es = case["rows"], case["width"], 2 if case["dtype"] == "bf16" else 4
        gate = {"none": 0, "vector": d * es, "rows": n * d * es}[case["gate"]]
        weights = d * es * (2 if case["post"] else 1)
        if case["pass"] == "backward":
            b = n * d * (4 + 5 * es) + weights + gate * (2 if case["gate"] == "rows" else 1) + 8 * n + 4 * d * 3
        else:
            b = n * d * (3 * es + (1 if case["pass"] == "forward_fp8" else es)) + weights + gate + 8 * n
        return {"bytes": b, "flops": 10 * n * d}
    if case["operator"] == "loss":
        n, d, v, es = _counted(case), case["width"], case["vocab"], 2 if case["dtype"] == "bf16" else 4
        g = case["gradient"]
        return {"bytes": (n * d + v * d) * es * (2 if g else 1) + 12 * case["tokens"], "flops": 2.0 * n * d * v * (3 if g else 1)}
    n = sum(_sizes(case))
    ep, eg = (2 if case["param"] == "bf16" else 4), (2 if case["grad"] == "bf16" else 4)
    state = 16 if case["state_bits"] == 32 else 4 + 16 / BLOCK
    weights = 8 + ep if case["param"] == "bf16" else 8  # master read and written, weight written
    return {"bytes": n * (eg + state + weights), "flops": 16 * n}


# ------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, scale=1.0, shift=0.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV).mul_(scale).add_(shift).to(dtype)


def prepare(case, seed):
    s = {"norm": _norm_inputs, "loss": _loss_inputs, "step": _step_inputs}[case["operator"]](case, _gen(seed))
    s["case"] = case
    if own and case["operator"] == "step":
        import invariant_token_logprobs_lm_amd as itl

        # the plan a training program makes once over its weights and gradients
        s["plan"] = itl.adamw_plan(s["params"], s["grads"], lr=s["lr"], step=s["step"], weight_decay=WEIGHT_DECAY,
                                   state_bits=case["state_bits"], exp_avg=s["m"], exp_avg_sq=s["v"],
                                   exp_avg_scale=s.get("m_scale"), exp_avg_sq_scale=s.get("v_scale"),
                                   master=s.get("master"))
    return s


def _norm_inputs(case, g):
    n, d, dt = case["rows"], case["width"], _DTYPES[case["dtype"]]
    s = {"x": _randn(g, n, d, dtype=dt), "y": _randn(g, n, d, scale=0.7, dtype=dt),
         "w_pre": _randn(g, d, scale=0.1, shift=1.0, dtype=dt), "w_post": None, "gate": None}
    if case["post"]:
        s["w_post"] = _randn(g, d, scale=0.1, shift=0.8, dtype=dt)
    if case["gate"] != "none":
        s["gate"] = _randn(g, *((d,) if case["gate"] == "vector" else (n, d)), scale=0.3, shift=0.5, dtype=dt)
    if case["pass"] == "backward":  # what the forward left: h and the rows' statistics; and the gradients coming in
        y = s["y"].float()
        s["rstd_post"] = torch.rsqrt((y * y).mean(1) + EPS) if case["post"] else None
        s["h"] = s.pop("x")
        h = s["h"].float()
        s["rstd_pre"] = torch.rsqrt((h * h).mean(1) + EPS)
        s["du"] = _randn(g, n, d, scale=1e-2)  # fp32, as the head's backward writes dH
        s["dh"] = _randn(g, n, d, scale=1e-2, dtype=dt)
    return s


def _loss_inputs(case, g):
    n, d, v, dt = case["tokens"], case["width"], case["vocab"], _DTYPES[case["dtype"]]
    W = _randn(g, v, d, scale=0.02, dtype=dt)
    y = torch.randint(0, v, (n,), generator=g, device=DEV, dtype=torch.int64)
    # hidden states that know something of the next token, as a trained model's
    lean = W[y].float()
    lean *= 6.0 / lean.norm(dim=1, keepdim=True)
    H = (_randn(g, n, d) + lean).to(dt)
    period, prompt = _prompts(case)
    targets = torch.where(torch.arange(n, device=DEV) % period < prompt, torch.full_like(y, -100), y).to(torch.int32)
    return {"H": H, "W": W, "targets": targets}


def _step_inputs(case, g):
    sizes, offsets, total = _layout(case)
    dp, dg = _DTYPES[case["param"]], _DTYPES[case["grad"]]
    real = torch.zeros(total, dtype=torch.bool, device=DEV)
    for n, o in zip(sizes, offsets):
        real[o:o + n] = True
    fill = lambda scale: _randn(g, total, scale=scale).mul_(real)  # noqa: E731
    weights = fill(0.02)
    s = {"lr": torch.full((1,), LR, device=DEV), "step": torch.full((1,), 100, dtype=torch.int64, device=DEV)}
    s["weights"] = weights.to(dp)  # one allocation; the tensors are its pieces
    if case["param"] == "bf16":
        s["master"] = weights
    s["gradients"] = fill(1e-3).to(dg)
    s["params"] = [s["weights"][o:o + n] for n, o in zip(sizes, offsets)]
    s["grads"] = [s["gradients"][o:o + n] for n, o in zip(sizes, offsets)]
    m, r = fill(3e-4), fill(1e-3).abs_()
    if case["state_bits"] == 32:
        s["m"], s["v"] = m, r.square_()
    else:
        s["m"], s["m_scale"] = _quantize(m)
        s["v"], s["v_scale"] = _quantize(r)
    return s


def _quantize(x):
    """E4M3 codes (uint8) and a scale for each block of 256, largest value at 448."""
    x = x.view(-1, BLOCK)
    scale = x.abs().amax(1) / 448.0
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    return (x / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(-1), scale


# ---------------------------------------------------------------------- run

def run(s):
    return {"norm": _run_norm, "loss": _run_loss, "step": _run_step}[s["case"]["operator"]](s)


def _run_norm(s):
    c = s["case"]
    if own:
        import invariant_token_logprobs_lm_amd as itl

        kw = {"w_post": s["w_post"], "gate": s["gate"], "scale": RESIDUAL_SCALE}
        if c["pass"] == "backward":
            dx, dy, dw_pre, dw_post, dgate = itl.residual_norm_backward(
                s["du"], s["dh"], s["h"], s["y"], s["w_pre"], s["rstd_pre"], rstd_post=s["rstd_post"], **kw)
            return {"dx": dx, "dy": dy, "dw_pre": dw_pre, "dw_post": dw_post, "dgate": dgate}
        if c["pass"] == "forward_fp8":
            h, codes, scale, rstd_pre, rstd_post = itl.residual_norm_fp8(s["x"], s["y"], s["w_pre"], eps=EPS, **kw)
            return {"h": h, "u": codes.view(torch.float8_e4m3fn), "u_scale": scale, "rstd_pre": rstd_pre, "rstd_post": rstd_post}
        h, u, rstd_pre, rstd_post = itl.residual_norm(s["x"], s["y"], s["w_pre"], eps=EPS, **kw)
        return {"h": h, "u": u, "rstd_pre": rstd_pre, "rstd_post": rstd_post}
    return _plain_norm_backward(s) if c["pass"] == "backward" else _plain_norm(s)


def _plain_norm(s):
    dt = s["x"].dtype
    x, y, w_pre = s["x"].float(), s["y"].float(), s["w_pre"].float()
    rstd_post = None
    if s["w_post"] is not None:
        rstd_post = torch.rsqrt((y * y).mean(1) + EPS)
        y = y * rstd_post[:, None] * s["w_post"].float()
    if s["gate"] is not None:
        y = y * s["gate"].float()
    h = (x + RESIDUAL_SCALE * y).to(dt)  # the residual stream is kept in its type, and the norm is the kept values'
    hf = h.float()
    rstd_pre = torch.rsqrt((hf * hf).mean(1) + EPS)
    u = hf * rstd_pre[:, None] * w_pre
    if s["case"]["pass"] == "forward_fp8":
        scale = u.abs().amax(1) / 448.0
        scale = torch.where(scale > 0, scale, torch.ones_like(scale))
        return {"h": h, "u": (u / scale[:, None]).to(torch.float8_e4m3fn), "u_scale": scale, "rstd_pre": rstd_pre, "rstd_post": rstd_post}
    return {"h": h, "u": u.to(dt), "rstd_pre": rstd_pre, "rstd_post": rstd_post}


def _plain_norm_backward(s):
    dt = s["h"].dtype
    du, dh, h, y, w_pre = s["du"].float(), s["dh"].float(), s["h"].float(), s["y"].float(), s["w_pre"].float()
    r = s["rstd_pre"][:, None]
    dn, hn = du * w_pre, h * r
    dx = dh + r * (dn - hn * (dn * hn).mean(1, keepdim=True))
    dw_pre = (du * hn).sum(0)
    dp = RESIDUAL_SCALE * dx
    if s["gate"] is not None:
        dp = dp * s["gate"].float()
    dw_post = None
    if s["w_post"] is not None:
        w_post, rp = s["w_post"].float(), s["rstd_post"][:, None]
        yn = y * rp
        p = yn * w_post
        dw_post = (dp * yn).sum(0)
        dq = dp * w_post
        dy = rp * (dq - yn * (dq * yn).mean(1, keepdim=True))
    else:
        p, dy = y, dp
    dgate = None
    if s["gate"] is not None:
        dgate = RESIDUAL_SCALE * p * dx
        dgate = dgate.sum(0) if s["gate"].dim() == 1 else dgate.to(dt)
    return {"dx": dx.to(dt), "dy": dy.to(dt), "dw_pre": dw_pre, "dw_post": dw_post, "dgate": dgate}


def _run_loss(s):
    c = s["case"]
    if own:
        import invariant_token_logprobs_lm_amd as itl

        kw = {"label_smoothing": c["smoothing"], "z_weight": c["z_weight"]}
        if not c["gradient"]:
            loss, token_loss, lse = itl.cross_entropy(s["H"], s["W"], s["targets"], **kw)
            return {"loss": loss, "token_loss": token_loss}
        loss, token_loss, lse, dH, dW = itl.cross_entropy_grad(s["H"], s["W"], s["targets"], grad_dtype=s["H"].dtype, **kw)
        return {"loss": loss, "token_loss": token_loss, "dH": dH, "dW": dW}
    H, W, t = s["H"].float(), s["W"].float(), s["targets"].long()
    eps, lam, v = c["smoothing"], c["z_weight"], W.shape[0]
    keep = t >= 0
    y = t.clamp(min=0)[:, None]
    count = keep.sum().clamp(min=1)
    z = H @ W.t()
    top = z.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
    token = lse - (1.0 - eps) * z.gather(1, y) + lam * lse * lse
    if eps:
        token = token - eps * z.mean(1, keepdim=True)
    token_loss = torch.where(keep, token[:, 0], torch.zeros_like(token[:, 0]))
    loss = (token_loss.double().sum() / count).float().view(1)
    if not c["gradient"]:
        return {"loss": loss, "token_loss": token_loss}
    g = torch.exp(z.sub_(lse)).mul_(1.0 + 2.0 * lam * lse)
    if eps:
        g.sub_(eps / v)
    g.scatter_add_(1, y, torch.full_like(lse, -(1.0 - eps)))
    g.mul_((keep / count).float()[:, None])
    return {"loss": loss, "token_loss": token_loss, "dH": (g @ W).to(s["H"].dtype), "dW": (g.t() @ H).to(s["W"].dtype)}


def _run_step(s):
    c = s["case"]
    norm = None
    if own:
        import invariant_token_logprobs_lm_amd as itl

        norm = itl.adamw_step(s["plan"], betas=BETAS, eps=ADAM_EPS, max_norm=MAX_NORM if c["clip"] else None)
    else:
        b1, b2 = BETAS
        g = s["gradients"].float()
        if c["clip"]:
            norm = g.square().sum().sqrt().view(1)
            g = g * (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)
        s["step"] += 1
        t = s["step"].double()
        rate = (s["lr"].double() / (1.0 - b1 ** t)).float()
        root = (1.0 / torch.sqrt(1.0 - b2 ** t)).float()
        decay = 1.0 - s["lr"] * WEIGHT_DECAY
        if c["state_bits"] == 32:
            m, v = s["m"], s["v"]
        else:
            m = s["m"].view(torch.float8_e4m3fn).float().view(-1, BLOCK).mul_(s["m_scale"][:, None]).view(-1)
            v = s["v"].view(torch.float8_e4m3fn).float().view(-1, BLOCK).mul_(s["v_scale"][:, None]).square_().view(-1)
        m.mul_(b1).add_(g * (1.0 - b1))
        v.mul_(b2).add_(g.square().mul_(1.0 - b2))
        r = v.sqrt()
        p = s.get("master", s["weights"])
        p.mul_(decay).sub_(m / (r * root + ADAM_EPS) * rate)
        if "master" in s:
            s["weights"].copy_(p)
        if c["state_bits"] == 8:
            codes, scale = _quantize(m)
            s["m"].copy_(codes)
            s["m_scale"].copy_(scale)
            # a root that is not zero is never stored as zero: a later division by it would run away
            r = r.view(-1, BLOCK)
            scale = r.amax(1) / 448.0
            scale = torch.where(scale > 0, scale, torch.ones_like(scale))
            q = r / scale[:, None]
            q = torch.where(q > 0, q.clamp(min=2.0 ** -9), q)
            s["v"].copy_(q.to(torch.float8_e4m3fn).view(torch.uint8).view(-1))
            s["v_scale"].copy_(scale)
    out = {"weights": s["weights"], "master": s.get("master"), "norm": norm}
    if c["state_bits"] == 32:
        return {**out, "m": s["m"], "v": s["v"]}
    return {**out, "m": s["m"].view(torch.float8_e4m3fn), "m_scale": s["m_scale"],
            "v": s["v"].view(torch.float8_e4m3fn), "v_scale": s["v_scale"]}


# -------------------------------------------------------------------- exact

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    g = _gen(seed)
    if case["operator"] == "norm":
        return _exact_norm(case, _norm_inputs(case, g))
    if case["operator"] == "loss":
        return _exact_loss(case, _loss_inputs(case, g))
    return _exact_step(case, _step_inputs(case, g))


def _f64(v):
    return None if v is None else v.to(torch.float64)


def _exact_norm(case, s):
    s = {k: _f64(v) for k, v in s.items()}
    d = case["width"]
    gate = s["gate"] if s["gate"] is not None else torch.ones((), dtype=torch.float64, device=DEV)
    y = s["y"]
    if case["pass"] != "backward":
        rstd_post, branch = None, y
        if s["w_post"] is not None:
            rstd_post = 1.0 / torch.sqrt(torch.einsum("nd,nd->n", y, y) / d + EPS)
            branch = torch.einsum("nd,n,d->nd", y, rstd_post, s["w_post"])
        h = s["x"] + RESIDUAL_SCALE * gate * branch
        out = {"h": h, "rstd_post": rstd_post}
        h = h.to(_DTYPES[case["dtype"]]).double()  # the residual stream is kept in its type, and the norm is the kept values'
        rstd_pre = 1.0 / torch.sqrt(torch.einsum("nd,nd->n", h, h) / d + EPS)
        u = torch.einsum("nd,n,d->nd", h, rstd_pre, s["w_pre"])
        if case["pass"] == "forward_fp8":
            # the stored rows are a type's rounding of u over the row's largest value; their error is the type's
            top = u.abs().max(1, keepdim=True).values / 448.0
            return {**out, "u": u / top, "u_scale": top[:, 0], "rstd_pre": rstd_pre}
        return {**out, "u": u, "rstd_pre": rstd_pre}
    # backward by the Jacobian of a normalised row: J = r (I - n n^T / d), n = the row over its root mean square
    n_pre = s["h"] / torch.sqrt(torch.einsum("nd,nd->n", s["h"], s["h"]) / d + EPS)[:, None]
    r_pre = 1.0 / torch.sqrt(torch.einsum("nd,nd->n", s["h"], s["h"]) / d + EPS)[:, None]
    a = s["du"] * s["w_pre"]
    dx = s["dh"] + r_pre * a - r_pre * n_pre * (torch.einsum("nd,nd->n", a, n_pre) / d)[:, None]
    out = {"dx": dx, "dw_pre": torch.einsum("nd,nd->d", s["du"], n_pre)}
    db = RESIDUAL_SCALE * dx  # gradient of gate * branch
    if s["w_post"] is None:
        branch, out["dy"], out["dw_post"] = y, db * gate, None
    else:
        r_post = 1.0 / torch.sqrt(torch.einsum("nd,nd->n", y, y) / d + EPS)[:, None]
        n_post = y * r_post
        branch = n_post * s["w_post"]
        out["dw_post"] = torch.einsum("nd,nd->d", db * gate, n_post)
        a = db * gate * s["w_post"]
        out["dy"] = r_post * a - r_post * n_post * (torch.einsum("nd,nd->n", a, n_post) / d)[:, None]
    out["dgate"] = None
    if s["gate"] is not None:
        out["dgate"] = torch.einsum("nd,nd->d", db, branch) if s["gate"].dim() == 1 else db * branch
    return out


def _exact_loss(case, s):
    H, W, t = _f64(s["H"]), _f64(s["W"]), s["targets"].long()
    eps, lam, v = case["smoothing"], case["z_weight"], case["vocab"]
    rows = torch.nonzero(t >= 0)[:, 0]
    token_loss = torch.zeros(case["tokens"], dtype=torch.float64, device=DEV)
    if not len(rows):
        z = {"loss": token_loss[:1] * 0, "token_loss": token_loss}
        return {**z, "dH": torch.zeros_like(H), "dW": torch.zeros_like(W)} if case["gradient"] else z
    Hc, yc = H[rows], t[rows]
    q = torch.mm(Hc, W.t())
    lse = torch.logsumexp(q, 1)
    # cross entropy against the smoothed target: the target's share, then an even share over the vocabulary
    ce = -(1 - eps) * torch.log_softmax(q, 1)[torch.arange(len(rows), device=DEV), yc] + eps * (lse - q.mean(1))
    token_loss[rows] = ce + lam * lse ** 2
    out = {"loss": token_loss.sum().view(1) / len(rows), "token_loss": token_loss}
    if not case["gradient"]:
        return out
    q = torch.softmax(q, 1) * (1 + 2 * lam * lse)[:, None] - eps / v
    q[torch.arange(len(rows), device=DEV), yc] -= 1 - eps
    q /= len(rows)
    dH = torch.zeros_like(H)
    dH[rows] = torch.mm(q, W)
    return {**out, "dH": dH, "dW": torch.mm(q.t(), Hc)}


def _exact_step(case, s):
    b1, b2 = BETAS
    g, norm = _f64(s["gradients"]), None
    if case["clip"]:
        norm = torch.linalg.vector_norm(g).view(1)
        g = g * min(1.0, MAX_NORM / (float(norm) + 1e-6))
    t = 101
    if case["state_bits"] == 32:
        m, v = _f64(s["m"]), _f64(s["v"])
    else:
        m = _f64(s["m"].view(torch.float8_e4m3fn)) * _f64(s["m_scale"]).repeat_interleave(BLOCK)
        v = (_f64(s["v"].view(torch.float8_e4m3fn)) * _f64(s["v_scale"]).repeat_interleave(BLOCK)) ** 2
    m = torch.lerp(g, m, b1)
    v = torch.lerp(g ** 2, v, b2)
    lr = float(s["lr"])
    p = _f64(s.get("master", s["weights"]))
    new = p - lr * WEIGHT_DECAY * p - lr * (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + ADAM_EPS)
    out = {"weights": new, "master": new if "master" in s else None, "norm": norm}
    if case["state_bits"] == 32:
        return {**out, "m": m, "v": v}
    r = torch.sqrt(v).view(-1, BLOCK)
    m = m.view(-1, BLOCK)
    ms, vs = (x.abs().max(1, keepdim=True).values / 448.0 for x in (m, r))
    ms, vs = (torch.where(x > 0, x, torch.ones_like(x)) for x in (ms, vs))
    return {**out, "m": (m / ms).view(-1), "m_scale": ms.view(-1), "v": (r / vs).view(-1), "v_scale": vs.view(-1)}
