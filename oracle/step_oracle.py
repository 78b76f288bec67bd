"""The operators round the MoE layer in a training step, in float64 on the CPU:
dropout, the block joint and the cross entropy of a linear layer, written from
their formulas (gradients by hand; the tests hold them against autograd and
against differences).  Shares no code with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np
import torch

_LOW = np.uint64(0xFFFFFFFF)
_HALF = np.uint64(32)


def _d(t):
    return None if t is None else t.detach().cpu().double()


def philox4x32_10(counter, key):
    """Four words per counter (arrays or ints of 32-bit values), after ten rounds."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(v) for v in key]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> _HALF) ^ c[1] ^ np.uint64(k[0]), b & _LOW,
             (a >> _HALF) ^ c[3] ^ np.uint64(k[1]), a & _LOW]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def threshold(p: float) -> int:
    return math.floor(65536 * float(np.float32(p)) + 0.5)


def keep(seed: int, offset: int, rows: int, d: int, p: float) -> torch.Tensor:
    """Which elements of [rows, d] dropout keeps (bool)."""
    blocks = -(-d // 8)
    seed, offset = seed & (2 ** 64 - 1), offset & (2 ** 64 - 1)
    words = philox4x32_10((np.arange(blocks)[None, :].repeat(rows, 0),
                           np.arange(rows)[:, None].repeat(blocks, 1), offset & 0xFFFFFFFF,
                           offset >> 32), (seed & 0xFFFFFFFF, seed >> 32))
    bits = np.stack([h for w in words for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], 2)
    return torch.from_numpy(bits.reshape(rows, -1)[:, :d] >= threshold(p))


def factors(rng, rows, d, p):
    """What dropout multiplies each element by: 0, or 1 / (1 - T / 65536)."""
    if threshold(p) == 0:
        return torch.ones(rows, d, dtype=torch.float64)
    seed, offset = (int(v) for v in rng.cpu())
    return keep(seed, offset, rows, d, p).double() * (65536 / (65536 - threshold(p)))


def dropout(x, rng, p):
    f = factors(rng, *x.shape, p)
    return torch.where(f > 0, _d(x) * f, torch.zeros_like(f))


def _vec(params, key, d, other):
    t = params.get(key)
    return torch.full((d,), float(other), dtype=torch.float64) if t is None else _d(t)


def normed(v, kind, gamma, beta, eps):
    """The norm's output, and its rows' mean and 1 / deviation."""
    rows = v.shape[0]
    if kind == "none":
        return v, torch.zeros(rows, dtype=torch.float64), torch.ones(rows, dtype=torch.float64)
    mean = v.mean(1) if kind == "layer" else torch.zeros(rows, dtype=torch.float64)
    c = v - mean[:, None]
    rstd = 1 / torch.sqrt((c * c).mean(1) + eps)
    return c * rstd[:, None] * gamma + beta, mean, rstd


def join(x, b, params, *, post, pre, scale=1.0, p=0.0, rng=None, eps=1e-5):
    """r, y (None without a pre norm), stats [4, rows], and z = post(b)."""
    x, b = _d(x), _d(b)
    n, d = b.shape
    z, m1, r1 = normed(b, post, _vec(params, "post_gamma", d, 1), _vec(params, "post_beta", d, 0),
                       eps)
    dz = z if p == 0 else torch.where(factors(rng, n, d, p) > 0, z * factors(rng, n, d, p), 0.0)
    r = scale * x + _vec(params, "gate", d, 1) * dz
    y, m2, r2 = normed(r, pre, _vec(params, "pre_gamma", d, 1), _vec(params, "pre_beta", d, 0), eps)
    return r, (None if pre == "none" else y), torch.stack((m1, r1, m2, r2)), z


def _back(w, h, rstd, kind):
    if kind == "none":
        return w
    t = w - h * (w * h).mean(1, keepdim=True)
    if kind == "layer":
        t = t - w.mean(1, keepdim=True)
    return rstd[:, None] * t


def join_backward(b, r, stats, params, dr, dy, *, post, pre, scale=1.0, p=0.0, rng=None):
    """dx, db, and the vectors' gradients by name."""
    b, r, dr, dy, st = map(_d, (b, r, dr, dy, stats))
    n, d = b.shape
    vec = lambda key, other: _vec(params, key, d, other)
    R = torch.zeros(n, d, dtype=torch.float64) if dr is None else dr
    g = {}
    if dy is not None:
        rh = (r - st[2][:, None]) * st[3][:, None]
        g["pre_gamma"], g["pre_beta"] = (dy * rh).sum(0), dy.sum(0)
        R = R + _back(dy * vec("pre_gamma", 1), rh, st[3], pre)
    bh = b if post == "none" else (b - st[0][:, None]) * st[1][:, None]
    z = bh * vec("post_gamma", 1) + vec("post_beta", 0)
    u = R * factors(rng, n, d, p)
    g["gate"] = (u * z).sum(0)
    dz = u * vec("gate", 1)
    g["post_gamma"], g["post_beta"] = (dz * bh).sum(0), dz.sum(0)
    return scale * R, _back(dz * vec("post_gamma", 1), bh, st[1], post), g


def cross_entropy(x, W, targets, z_loss=0.0):
    """loss and lse of each token (0 where the target is negative), and the logits."""
    x, W, t = _d(x), _d(W), targets.cpu().long()
    logits = x @ W.T
    lse = torch.logsumexp(logits, 1)
    loss = lse - logits[torch.arange(len(t)), t.clamp(min=0)] + z_loss * lse * lse
    zero = torch.zeros_like(lse)
    return torch.where(t >= 0, loss, zero), torch.where(t >= 0, lse, zero), logits


def cross_entropy_backward(x, W, targets, lse, dloss, z_loss=0.0):
    """dx, dW and the logits' gradient (rows of left out tokens zero)."""
    x, W, lse, dloss, t = _d(x), _d(W), _d(lse), _d(dloss), targets.cpu().long()
    counted = t >= 0
    dl = torch.zeros(len(t), W.shape[0], dtype=torch.float64)
    xr, ls = x[counted], lse[counted][:, None]
    p = torch.exp(xr @ W.T - ls) * (1 + 2 * z_loss * ls)
    p[torch.arange(len(p)), t[counted]] -= 1
    dl[counted] = p * dloss[counted][:, None]
    dW = dl[counted].T @ xr
    return dl @ W, dW, dl
