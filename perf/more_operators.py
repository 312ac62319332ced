"""The learner's block in 8 bits and with dropout, as measured cases.

Four families, used together around a block's output projection: the matrix
product in E4M3 with a scale for each block of 128 (forward, input gradient,
weight gradient), the quantisation that makes its operands, dropout from a
counter-based generator with a mask that is never stored, and the norms around
the block with that dropout in them. Each case runs either in its plain form
(elementary torch operations in float32) or, with ``own`` set, through the
package's entry points.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
RESIDUAL_SCALE = 0.5
BLOCK = 128  # values that share a scale
LARGEST = 448.0  # of E4M3
SITE = 3  # which dropout of the model

_DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decode token through a square projection of the 1.5B model: latency
        _product("product, one decode token", "forward", 1, 1536, 1536, "bf16"),
        # a decode batch's logits from the widest head, whose weights are read once
        _product("product, logits of 16 tokens", "forward", 16, 129280, 7168, "fp32"),
        # a chunk of a prompt, odd in every size
        _product("product, ragged chunk", "forward", 777, 1001, 1500, "bf16"),
        # a learner batch's gradient through a 4B block's projection from four times its width
        _product("product, input gradient", "input", 16384, 10240, 2560, "bf16"),
        # the gradient of the same layer's weights: the contraction runs over the tokens
        _product("product, weight gradient", "weight", 2560, 10240, 16384, "fp32"),
        # a decode token's row on its way into a product
        _quantise("quantise, one decode token", "blocks", 1, 7168, "bf16", False),
        # an output gradient for both products that it enters
        _quantise("quantise, gradient both ways", "blocks", 16384, 2560, "bf16", True),
        # fp32 weights after a step, for the forward and for the input gradient
        _quantise("quantise, weights both ways", "tiles", 8960, 1536, "fp32", True),
        # embeddings of a small fp32 model of odd width
        _dropout("dropout, odd fp32 rows", 777, 1001, "fp32", 0.1),
        # embeddings of a learner batch
        _dropout("dropout, learner batch", 16384, 2560, "bf16", 0.1),
        # a block's output with its dropout, through both norms, to the next product's rows
        _norm("norm with dropout, rows for the product", "forward_blocks", 8192, 2560, "bf16", True, "vector", 0.1),
        # its gradient, fed with a product's fp32 input gradient
        _norm("norm with dropout, backward", "backward", 16384, 2560, "bf16", True, "vector", 0.1),
    ]


def draw(rng):
    kind = rng.choice(["product", "product", "quantise", "dropout", "norm"])
    if kind == "product":
        use = rng.choice(["forward", "forward", "input", "weight"])
        k = _size(rng, 64, 16384)
        n = _size(rng, 64, min(129280, 7168 * 129280 // k))
        most = 16384 * 2560 * 10240 // (n * k)
        m = min(_size(rng, 64, 16384) if use == "weight" else _log(rng, 1, 16384), max(1, most))
        return _product(None, use, m, n, k, rng.choice(["bf16", "fp32"]))
    rows, p = _log(rng, 1, 16384), rng.choice([0.05, 0.1, 0.3])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if kind == "quantise":
        width = _size(rng, 64, 10240)
        return _quantise(None, rng.choice(["blocks", "tiles"]), min(rows, 16384 * 2560 // width), width, dtype, rng.random() < 0.6)
    width = _size(rng, 48, 7168)
    if kind == "dropout":
        return _dropout(None, min(rows, 16384 * 2560 // width), width, dtype, p)
    what = rng.choice(["forward", "forward_blocks", "backward"])
    width = 128 * max(1, width // 128) if what == "forward_blocks" else width if width % 64 == 0 else min(width, 4000)
    return _norm(None, what, min(rows, 16384 * 2560 // width), width, dtype, rng.random() < 0.5,
                 rng.choice(["none", "vector", "rows"]), p)


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _size(rng, low, high):
    """A width: mostly whole 64s, as models have them, sometimes any number."""
    v = _log(rng, low, high)
    return v if rng.random() < 0.3 else max(64, v // 64 * 64)


def _named(name, case):
    return case if name is None else {"name": name, **case}


def _product(name, use, m, n, k, out):
    """out[m, n] = sum over k. use: where the operands come from."""
    return _named(name, {"operator": "product", "use": use, "m": m, "n": n, "k": k, "out": out})


def _quantise(name, kind, rows, width, dtype, both):
    """kind: a scale for each 128 of a row ("blocks") or for each 128 x 128 tile; both: also the transposed codes."""
    return _named(name, {"operator": "quantise", "kind": kind, "rows": rows, "width": width, "dtype": dtype, "both": both})


def _dropout(name, rows, width, dtype, p):
    return _named(name, {"operator": "dropout", "rows": rows, "width": width, "dtype": dtype, "p": p})


def _norm(name, what, rows, width, dtype, post, gate, p):
    return _named(name, {"operator": "norm", "pass": what, "rows": rows, "width": width, "dtype": dtype, "post": post, "gate": gate, "p": p})


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    if case["operator"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        b = (m + n) * k + 4 * _blocks(k) * (m + _blocks(n)) + m * n * (2 if case["out"] == "bf16" else 4)
        return {"bytes": b, "flops": 2.0 * m * n * k}
    n, d, es = case["rows"], case["width"], 2 if case["dtype"] == "bf16" else 4
    if case["operator"] == "quantise":
        ways = 2 if case["both"] else 1
        scales = n * _blocks(d) + (d * _blocks(n) if case["both"] else 0) if case["kind"] == "blocks" else ways * _blocks(n) * _blocks(d)
        return {"bytes": n * d * (es + ways) + 4 * scales, "flops": 3 * n * d}
    if case["operator"] == "dropout":
        return {"bytes": 2 * n * d * es, "flops": 2 * n * d}
    gate = {"none": 0, "vector": d * es, "rows": n * d * es}[case["gate"]]
    weights = d * es * (2 if case["post"] else 1)
    if case["pass"] == "backward":
        b = n * d * (4 + 5 * es) + weights + gate * (2 if case["gate"] == "rows" else 1) + 8 * n + 4 * d * 3
    else:
        b = n * d * (3 * es + (1 + 4 / BLOCK if case["pass"] == "forward_blocks" else es)) + weights + gate + 8 * n
    return {"bytes": b, "flops": 12 * n * d}


# ------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, scale=1.0, shift=0.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV).mul_(scale).add_(shift).to(dtype)


def prepare(case, seed):
    make = {"product": _product_inputs, "quantise": _quantise_inputs, "dropout": _dropout_inputs, "norm": _norm_inputs}
    s = make[case["operator"]](case, _gen(seed))
    s["case"] = case
    return s


def _dropout_seed(g):
    return torch.randint(0, 2 ** 62, (1,), generator=g, device=DEV, dtype=torch.int64)


def _activations(g, n, d, scale):
    """Rows whose columns differ in size, some of them far larger, as a block's are."""
    x = torch.randn(n, d, generator=g, device=DEV)
    x *= torch.exp(0.7 * torch.randn(d, generator=g, device=DEV)) * scale
    return x


def _product_inputs(case, g):
    m, n, k = case["m"], case["n"], case["k"]
    if case["use"] == "forward":  # token rows against weights
        a, b = _activations(g, m, k, 1.0), torch.randn(n, k, generator=g, device=DEV).mul_(0.02)
    elif case["use"] == "input":  # rows of the output's gradient against the transposed weights
        a, b = _activations(g, m, k, 1e-3), torch.randn(n, k, generator=g, device=DEV).mul_(0.02)
    else:  # the output's gradient and the activations, both with the tokens along the contraction
        a, b = _activations(g, k, m, 1e-3).t().contiguous(), _activations(g, k, n, 1.0).t().contiguous()
    a, a_scale = _plain_blocks(a)
    b, b_scale = _plain_tiles(b)
    return {"a": a.view(torch.uint8), "a_scale": a_scale, "b": b.view(torch.uint8), "b_scale": b_scale}


def _quantise_inputs(case, g):
    n, d = case["rows"], case["width"]
    x = _activations(g, n, d, 1.0) if case["kind"] == "blocks" else torch.randn(n, d, generator=g, device=DEV).mul_(0.02)
    return {"x": x.to(_DTYPES[case["dtype"]])}


def _dropout_inputs(case, g):
    return {"x": _randn(g, case["rows"], case["width"], dtype=_DTYPES[case["dtype"]]), "seed": _dropout_seed(g)}


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
        s["du"] = _randn(g, n, d, scale=1e-2)  # fp32, as the product writes it
        s["dh"] = _randn(g, n, d, scale=1e-2, dtype=dt)
    s["seed"] = _dropout_seed(g)
    return s


# ---------------------------------------------------------------------- run

def run(s):
    return {"product": _run_product, "quantise": _run_quantise, "dropout": _run_dropout, "norm": _run_norm}[s["case"]["operator"]](s)


def _run_product(s):
    c = s["case"]
    if own:
        import invariant_token_logprobs_lm_amd as itl

        return itl.matmul_fp8_blocks(s["a"], s["a_scale"], s["b"], s["b_scale"], out_dtype=_DTYPES[c["out"]])
    m, n, kb = c["m"], c["n"], s["a_scale"].shape[0]
    a = s["a"].view(torch.float8_e4m3fn).float().view(m, kb, BLOCK)
    a = (a * s["a_scale"].t()[:, :, None]).view(m, kb * BLOCK)
    b = s["b"].view(torch.float8_e4m3fn).float().view(n, kb, BLOCK)
    b = (b * s["b_scale"].repeat_interleave(BLOCK, 0)[:n, :, None]).view(n, kb * BLOCK)
    return (a @ b.t()).to(_DTYPES[c["out"]])


def _run_quantise(s):
    c = s["case"]
    if own:
        import invariant_token_logprobs_lm_amd as itl

        make = itl.quantize_blocks_fp8 if c["kind"] == "blocks" else itl.quantize_tiles_fp8
        q, scale, qt, t_scale = make(s["x"], columns=c["both"])
        q, qt = (None if v is None else v.view(torch.float8_e4m3fn) for v in (q, qt))
    else:
        make = _plain_blocks if c["kind"] == "blocks" else _plain_tiles
        x = s["x"].float()
        q, scale = make(x)
        qt, t_scale = make(x.t()) if c["both"] else (None, None)
    return {"q": q, "scale": scale, "qt": qt, "t_scale": t_scale}


def _plain_blocks(x):
    """Codes [n, whole blocks] and scales [blocks, n], one for each 128 values of a row."""
    n, d = x.shape
    x = torch.nn.functional.pad(x, (0, -d % BLOCK)).view(n, -1, BLOCK)
    scale = _plain_scale(x.abs().amax(2))
    return (x / scale[:, :, None]).to(torch.float8_e4m3fn).view(n, -1), scale.t().contiguous()


def _plain_tiles(x):
    """Codes [n, whole blocks] and scales [tiles down, tiles across], one for each 128 x 128 tile."""
    n, d = x.shape
    x = torch.nn.functional.pad(x, (0, -d % BLOCK, 0, -n % BLOCK)).view(_blocks(n), BLOCK, -1, BLOCK)
    scale = _plain_scale(x.abs().amax((1, 3)))
    return (x / scale[:, None, :, None]).to(torch.float8_e4m3fn).view(_blocks(n) * BLOCK, -1)[:n].contiguous(), scale


def _plain_scale(top):
    return torch.where(top > 0, (top / LARGEST).clamp(min=2.0 ** -126), torch.ones_like(top))


def _run_dropout(s):
    c = s["case"]
    if own:
        import invariant_token_logprobs_lm_amd as itl

        return itl.dropout(s["x"], itl.Dropout(c["p"], s["seed"], site=SITE))
    keep, scale = _plain_keep(s, c)
    return torch.where(keep, s["x"].float() * scale, 0.0).to(s["x"].dtype)


def _plain_keep(s, c):
    """Which values stay, and what they are multiplied by.

    A call of the generator (Philox 4 x 32, ten rounds, keyed with the seed) at
    (8-column group, row, site) gives eight 16-bit numbers, the first in the low
    half of the first word; a value is dropped where its number is below p 2^16.
    """
    n, d = c["rows"], c["width"]
    low = 0xFFFFFFFF
    key = [s["seed"] & low, (s["seed"] >> 32) & low]
    groups = -(-d // 8)
    row = torch.arange(n, device=DEV)[:, None].expand(n, groups)
    w = [torch.arange(groups, device=DEV)[None, :].expand(n, groups), row & low, row >> 32, torch.full_like(row, SITE)]
    for _ in range(10):
        (h0, l0), (h1, l1) = _plain_multiply(w[0], 0xD2511F53), _plain_multiply(w[2], 0xCD9E8D57)
        w = [h1 ^ w[1] ^ key[0], l1, h0 ^ w[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) & low, (key[1] + 0xBB67AE85) & low]
    u = torch.stack([v for x in w for v in (x & 0xFFFF, x >> 16)], 2).view(n, 8 * groups)[:, :d]
    drop = round(c["p"] * 65536)
    return u >= drop, 65536 / (65536 - drop)


def _plain_multiply(x, m):
    """High and low 32 bits of x m, both below 2^32."""
    return ((x >> 16) * m + ((x & 0xFFFF) * m >> 16)) >> 16, (x * m) & 0xFFFFFFFF


def _run_norm(s):
    c = s["case"]
    if own:
        import invariant_token_logprobs_lm_amd as itl

        kw = {"w_post": s["w_post"], "gate": s["gate"], "scale": RESIDUAL_SCALE, "dropout": itl.Dropout(c["p"], s["seed"], site=SITE)}
        if c["pass"] == "backward":
            dx, dy, dw_pre, dw_post, dgate = itl.residual_norm_backward(
                s["du"], s["dh"], s["h"], s["y"], s["w_pre"], s["rstd_pre"], rstd_post=s["rstd_post"], **kw)
            return {"dx": dx, "dy": dy, "dw_pre": dw_pre, "dw_post": dw_post, "dgate": dgate}
        if c["pass"] == "forward_blocks":
            h, codes, scale, rstd_pre, rstd_post = itl.residual_norm_blocks_fp8(s["x"], s["y"], s["w_pre"], eps=EPS, **kw)
            return {"h": h, "u": codes.view(torch.float8_e4m3fn), "u_scale": scale, "rstd_pre": rstd_pre, "rstd_post": rstd_post}
        h, u, rstd_pre, rstd_post = itl.residual_norm(s["x"], s["y"], s["w_pre"], eps=EPS, **kw)
        return {"h": h, "u": u, "rstd_pre": rstd_pre, "rstd_post": rstd_post}
    return _plain_norm_backward(s) if c["pass"] == "backward" else _plain_norm(s)


def _plain_norm(s):
    c, dt = s["case"], s["x"].dtype
    x, y, w_pre = s["x"].float(), s["y"].float(), s["w_pre"].float()
    rstd_post = None
    if s["w_post"] is not None:
        rstd_post = torch.rsqrt((y * y).mean(1) + EPS)
        y = y * rstd_post[:, None] * s["w_post"].float()
    if s["gate"] is not None:
        y = y * s["gate"].float()
    keep, times = _plain_keep(s, c)
    y = torch.where(keep, y * times, 0.0)
    h = (x + RESIDUAL_SCALE * y).to(dt)  # the residual stream is kept in its type, and the norm is the kept values'
    hf = h.float()
    rstd_pre = torch.rsqrt((hf * hf).mean(1) + EPS)
    u = hf * rstd_pre[:, None] * w_pre
    if c["pass"] == "forward_blocks":
        codes, scale = _plain_blocks(u)
        return {"h": h, "u": codes, "u_scale": scale, "rstd_pre": rstd_pre, "rstd_post": rstd_post}
    return {"h": h, "u": u.to(dt), "rstd_pre": rstd_pre, "rstd_post": rstd_post}


def _plain_norm_backward(s):
    dt = s["h"].dtype
    du, dh, h, y, w_pre = s["du"].float(), s["dh"].float(), s["h"].float(), s["y"].float(), s["w_pre"].float()
    r = s["rstd_pre"][:, None]
    dn, hn = du * w_pre, h * r
    dx = dh + r * (dn - hn * (dn * hn).mean(1, keepdim=True))
    dw_pre = (du * hn).sum(0)
    keep, times = _plain_keep(s, s["case"])
    branch = torch.where(keep, dx * (RESIDUAL_SCALE * times), 0.0)  # gradient of gate * p
    dp = branch if s["gate"] is None else branch * s["gate"].float()
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
        dgate = p * branch
        dgate = dgate.sum(0) if s["gate"].dim() == 1 else dgate.to(dt)
    return {"dx": dx.to(dt), "dy": dy.to(dt), "dw_pre": dw_pre, "dw_post": dw_post, "dgate": dgate}


# -------------------------------------------------------------------- exact

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    g = _gen(seed)
    if case["operator"] == "product":
        return _exact_product(case, _product_inputs(case, g))
    if case["operator"] == "quantise":
        return _exact_quantise(case, _quantise_inputs(case, g)["x"].double())
    if case["operator"] == "dropout":
        s = _dropout_inputs(case, g)
        return s["x"].double() * _exact_mask(case, s["seed"])
    return _exact_norm(case, _norm_inputs(case, g))


def _exact_product(case, s):
    out = torch.zeros(case["m"], case["n"], dtype=torch.float64, device=DEV)
    tile = torch.arange(case["n"], device=DEV) // BLOCK
    for i in range(s["a_scale"].shape[0]):  # block by block: the codes' product, then both scales
        cut = slice(i * BLOCK, (i + 1) * BLOCK)
        dot = torch.mm(s["a"][:, cut].contiguous().view(torch.float8_e4m3fn).double(), s["b"][:, cut].contiguous().view(torch.float8_e4m3fn).double().t())
        out += dot * s["a_scale"][i].double()[:, None] * s["b_scale"][:, i].double()[tile][None, :]
    return out


def _exact_quantise(case, x):
    """The codes' values before their rounding, padding's zeros among them."""
    def one(x):
        n, d = x.shape
        full = torch.zeros(_blocks(n) * BLOCK, _blocks(d) * BLOCK, dtype=torch.float64, device=DEV)
        full[:n, :d] = x
        if case["kind"] == "blocks":
            top = torch.stack([c.abs().max(1).values for c in full[:n].split(BLOCK, 1)])  # [blocks, n]
            full_top = top.t()
        else:
            top = torch.stack([torch.stack([c.abs().max() for c in r.split(BLOCK, 1)]) for r in full.split(BLOCK, 0)])
            full_top = top.repeat_interleave(BLOCK, 0)[:n]
        scale, full_scale = (torch.where(t > 0, t / LARGEST, torch.ones_like(t)) for t in (top, full_top))
        return full[:n] / full_scale.repeat_interleave(BLOCK, 1), scale
    q, scale = one(x)
    qt, t_scale = one(x.t()) if case["both"] else (None, None)
    return {"q": q, "scale": scale, "qt": qt, "t_scale": t_scale}


def _exact_mask(case, seed):
    """1 / (1 - p) or 0 for every value, the generator written out in numpy's 64-bit words."""
    n, groups = case["rows"], -(-case["width"] // 8)
    seed, word = int(seed.item()), np.uint64(0xFFFFFFFF)
    k0, k1, half = seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF, np.uint64(32)
    x0 = np.tile(np.arange(groups, dtype=np.uint64), (n, 1))
    x1 = np.repeat(np.arange(n, dtype=np.uint64), groups).reshape(n, groups)
    x2, x3 = np.zeros_like(x0), np.full_like(x0, SITE)
    for _ in range(10):
        p0, p1 = x0 * np.uint64(0xD2511F53), x2 * np.uint64(0xCD9E8D57)
        x0, x1, x2, x3 = (p1 >> half) ^ x1 ^ np.uint64(k0), p1 & word, (p0 >> half) ^ x3 ^ np.uint64(k1), p0 & word
        k0, k1 = k0 + 0x9E3779B9 & 0xFFFFFFFF, k1 + 0xBB67AE85 & 0xFFFFFFFF
    words = np.ascontiguousarray(np.stack([x0, x1, x2, x3], -1).astype("<u4"))
    drop = int(round(case["p"] * 2 ** 16))
    keep = words.view("<u2").reshape(n, 8 * groups)[:, :case["width"]] >= drop
    return torch.from_numpy(keep).to(DEV).double() * (2 ** 16 / (2 ** 16 - drop))


def _exact_norm(case, s):
    mask = _exact_mask(case, s.pop("seed"))
    s = {k: None if v is None else v.double() for k, v in s.items()}
    d = case["width"]
    gate = mask * (s["gate"] if s["gate"] is not None else 1.0)  # dropout is one more gate
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
        if case["pass"] == "forward_blocks":
            top = u.view(-1, d // BLOCK, BLOCK).abs().max(2).values / LARGEST
            return {**out, "u": u / top.repeat_interleave(BLOCK, 1), "u_scale": top.t().contiguous(), "rstd_pre": rstd_pre}
        return {**out, "u": u, "rstd_pre": rstd_pre}
    # backward by the Jacobian of a normalised row: J = r (I - n n^T / d), n = the row over its root mean square
    r_pre = 1.0 / torch.sqrt(torch.einsum("nd,nd->n", s["h"], s["h"]) / d + EPS)[:, None]
    n_pre = s["h"] * r_pre
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
        dgate = db * mask * branch
        out["dgate"] = dgate.sum(0) if s["gate"].dim() == 1 else dgate
    return out
