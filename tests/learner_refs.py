"""Plain 64-bit forms of the learner's operators (norms, cross entropy,
AdamW), from their formulas, on the CPU. Nothing of the product is used."""

import math

import torch

EPS24 = 2.0 ** -24  # half a step of fp32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return None if t is None else t.detach().cpu().double()


def rms(x, eps):
    return 1.0 / torch.sqrt((x * x).mean(1) + eps)


def norm_forward(x, y, w_pre, w_post=None, gate=None, scale=1.0, eps=1e-6):
    """(h unrounded, its terms' magnitude, rstd_post); u follows from the kept h."""
    if y is None:
        return x, x.abs(), None
    p, r_post = y, None
    if w_post is not None:
        r_post = rms(y, eps)
        p = y * r_post[:, None] * w_post
    if gate is not None:
        p = p * gate
    return x + scale * p, x.abs() + abs(scale) * p.abs(), r_post


def norm_out(h, w_pre, eps=1e-6):
    r = rms(h, eps)
    return h * r[:, None] * w_pre, r


def norm_backward(du, dh, h, y, w_pre, r_pre, w_post=None, r_post=None, gate=None, scale=1.0):
    """dict of gradients and, under "mag", bounds of the magnitudes summed in each."""
    n = h * r_pre[:, None]
    dn = du * w_pre
    c = (dn * n).mean(1, keepdim=True)
    dx = r_pre[:, None] * (dn - n * c)
    mag_dx = r_pre[:, None] * (dn.abs() + n.abs() * (dn * n).abs().mean(1, keepdim=True))
    if dh is not None:
        dx = dx + dh
        mag_dx = mag_dx + dh.abs()
    out = {"dx": dx, "dw_pre": (du * n).sum(0)}
    mag = {"dx": mag_dx, "dw_pre": (du * n).abs().sum(0)}
    if y is None:
        return out, mag
    g = torch.ones((), dtype=torch.float64) if gate is None else gate
    dp, mag_dp = scale * dx * g, abs(scale) * mag_dx * g.abs()
    q = y if w_post is None else y * r_post[:, None]
    p = q if w_post is None else q * w_post
    if w_post is None:
        out["dy"], mag["dy"] = dp, mag_dp
    else:
        dq, mag_dq = dp * w_post, mag_dp * w_post.abs()
        out["dw_post"], mag["dw_post"] = (dp * q).sum(0), (mag_dp * q.abs()).sum(0)
        out["dy"] = r_post[:, None] * (dq - q * (dq * q).mean(1, keepdim=True))
        mag["dy"] = r_post[:, None] * (mag_dq + q.abs() * (mag_dq * q.abs()).mean(1, keepdim=True))
    if gate is not None:
        dg, mg = scale * p * dx, (scale * p).abs() * mag_dx
        out["dgate"], mag["dgate"] = (dg.sum(0), mg.sum(0)) if gate.dim() == 1 else (dg, mg)
    return out, mag


def cross_entropy(H, W, targets, smoothing=0.0, z_weight=0.0, mean=True, grad_scale=1.0):
    """loss, token_loss, lse, dH, dW and the magnitudes the last two sum."""
    V = W.shape[0]
    t = targets.cpu().long()
    live = (t >= 0) & (t < V)
    z = H @ W.t()
    lse = torch.logsumexp(z, 1)
    y = t.clamp(0, V - 1)
    zy = z.gather(1, y[:, None])[:, 0]
    token = (1 - smoothing) * (lse - zy) + smoothing * (lse - z.mean(1)) + z_weight * lse ** 2
    token = torch.where(live, token, torch.zeros_like(token))
    N = max(1, int(live.sum())) if mean else 1
    p = torch.exp(z - lse[:, None])
    G = p * (1 + 2 * z_weight * lse)[:, None] - smoothing / V
    G[torch.arange(len(t)), y] -= 1 - smoothing
    G = G * (grad_scale / N) * live[:, None]
    return {"loss": token.sum() / N, "token_loss": token, "lse": torch.where(live, lse, torch.zeros_like(lse)),
            "dH": G @ W, "dW": G.t() @ H, "mag_dH": G.abs() @ W.abs(), "mag_dW": G.abs().t() @ H.abs(),
            "mag_z": (H.abs() @ W.abs().t()).amax(1)}


def adamw(w, g, m, v, t, lr, wd, betas, eps, clip=1.0):
    """One step at count t (after the raise): (w, m, v)."""
    b1, b2 = betas
    g = g * clip
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    w = w * (1 - lr * wd) - lr / (1 - b1 ** t) * m / (torch.sqrt(v) / math.sqrt(1 - b2 ** t) + eps)
    return w, m, v


def e4m3_values(codes, scale, block):
    """What uint8 codes with a scale per block stand for, in fp64."""
    return codes.cpu().view(torch.float8_e4m3fn).double() * scale.cpu().double().repeat_interleave(block)
