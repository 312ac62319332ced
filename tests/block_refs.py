"""Plain 64-bit forms of the learner's block operators (dropout, block-scaled
E4M3 codes and their product), from their definitions, on the CPU. Nothing of
the product is used."""

import numpy as np
import torch

BLOCK = 128


def philox(counter, key):
    """Philox 4 x 32, ten rounds: four arrays of 32-bit words (as uint64) under a pair of words."""
    c = [np.asarray(w, dtype=np.uint64) for w in counter]
    k0, k1 = (int(w) for w in key)
    word, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> half) ^ c[1] ^ np.uint64(k0), p1 & word, (p0 >> half) ^ c[3] ^ np.uint64(k1), p0 & word]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def keep_factors(n, d, p, seed, site=0, first_row=0):
    """fp64 [n, d]: 0 where dropped, else 65536 / (65536 - threshold)."""
    groups = -(-d // 8)
    row = np.array([(first_row + r) & (2 ** 64 - 1) for r in range(n)], dtype=np.uint64)[:, None]
    row = np.broadcast_to(row, (n, groups))
    group = np.broadcast_to(np.arange(groups, dtype=np.uint64), (n, groups))
    w = philox((group, row & np.uint64(0xFFFFFFFF), row >> np.uint64(32), np.full_like(row, site)),
               (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF))
    u = np.stack([v for x in w for v in (x & np.uint64(0xFFFF), x >> np.uint64(16))], -1).reshape(n, 8 * groups)[:, :d]
    threshold = int(np.rint(np.float64(np.float32(p)) * 65536))
    scale = 65536 / (65536 - threshold) if threshold < 65536 else 0.0
    return torch.from_numpy((u >= threshold).astype(np.float64) * scale)


def padded(x):
    n, d = x.shape
    out = torch.zeros(n, -(-d // BLOCK) * BLOCK, dtype=x.dtype)
    out[:, :d] = x
    return out


def scale_of(top):
    """amax / 448 in fp32, at least 2^-126, 1 for zeros."""
    s = (top.float() / 448.0).clamp(min=2.0 ** -126)
    return torch.where(top > 0, s, torch.ones_like(s))


def blocks(x):
    """(codes uint8 [n, whole], scale fp32 [blocks, n]) of an fp32 CPU tensor, by the definition."""
    x = padded(x.float())
    n = x.shape[0]
    v = x.view(n, -1, BLOCK)
    s = scale_of(v.abs().amax(2))
    return (v / s[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(n, -1), s.t().contiguous()


def tiles(x):
    x = padded(x.float())
    n, d = x.shape
    full = padded(x.t().contiguous()).t()
    v = full.reshape(-(-n // BLOCK), BLOCK, d // BLOCK, BLOCK)
    s = scale_of(v.abs().amax((1, 3)))
    q = (v / s[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1, d)[:n]
    return q.contiguous(), s


def values(codes):
    return codes.cpu().view(torch.float8_e4m3fn).double()


def product(a, a_scale, b, b_scale):
    """(A B^T, the magnitudes its sums have) in fp64."""
    kb = a_scale.shape[0]
    va, vb = values(a).view(a.shape[0], kb, BLOCK), values(b).view(b.shape[0], kb, BLOCK)
    va = (va * a_scale.cpu().double().t()[:, :, None]).view(a.shape)
    rows = torch.arange(b.shape[0]) // BLOCK
    vb = (vb * b_scale.cpu().double()[rows][:, :, None]).view(b.shape)
    return va @ vb.t(), va.abs() @ vb.abs().t()
