"""The training operators of the MoE layer in float64 on the CPU, written from
their formulas (the gradients by hand, not by autograd; the tests hold them
against autograd and against differences).

Shares no code with the CUDA path.  Weights are laid out as the library takes
them: W1, W3 [E, F, d]; W2 [E, d, F]; Wg [E, d].  Expert e owns rows
offsets[e] .. offsets[e+1] of the row arrays.
"""
from __future__ import annotations

import torch


def _d(t):
    return None if t is None else t.detach().cpu().double()


def norm(x, gamma, beta, eps):
    x, gamma, beta = _d(x), _d(gamma), _d(beta)
    mean = x.mean(1)
    var = ((x - mean[:, None]) ** 2).mean(1)
    rstd = 1 / torch.sqrt(var + eps)
    y = (x - mean[:, None]) * rstd[:, None] * gamma
    return (y if beta is None else y + beta), mean, rstd


def norm_backward(x, gamma, mean, rstd, dy):
    x, gamma, mean, rstd, dy = map(_d, (x, gamma, mean, rstd, dy))
    d = x.shape[1]
    xh = (x - mean[:, None]) * rstd[:, None]
    w = dy * gamma
    dx = rstd[:, None] * (w - w.sum(1, keepdim=True) / d - xh * (w * xh).sum(1, keepdim=True) / d)
    return dx, (dy * xh).sum(0), dy.sum(0)


def _silu(g):
    return g / (1 + torch.exp(-g))


def ffn(x, offsets, W1, W3, W2):
    """y, g, u, h (g and u None for ReLU); rows outside every segment stay zero."""
    x, W1, W3, W2 = map(_d, (x, W1, W3, W2))
    P, F = x.shape[0], W1.shape[1]
    y, h = torch.zeros_like(x), torch.zeros(P, F, dtype=torch.float64)
    g = u = None
    if W3 is not None:
        g, u = torch.zeros_like(h), torch.zeros_like(h)
    for e in range(W1.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        pre = x[a:b] @ W1[e].T
        if W3 is None:
            h[a:b] = pre.clamp(min=0)
        else:
            g[a:b], u[a:b] = pre, x[a:b] @ W3[e].T
            h[a:b] = _silu(pre) * u[a:b]
        y[a:b] = h[a:b] @ W2[e].T
    return y, g, u, h


def ffn_backward(x, offsets, W1, W3, W2, g, u, h, dy):
    """dx, dW1, dW3 (None for ReLU), dW2, dg, du from the kept g, u, h."""
    x, W1, W3, W2, g, u, h, dy = map(_d, (x, W1, W3, W2, g, u, h, dy))
    dx, dg = torch.zeros_like(x), torch.zeros_like(h)
    du = None if W3 is None else torch.zeros_like(h)
    dW1, dW2 = torch.zeros_like(W1), torch.zeros_like(W2)
    dW3 = None if W3 is None else torch.zeros_like(W3)
    for e in range(W1.shape[0]):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        dh = dy[r] @ W2[e]
        dW2[e] = dy[r].T @ h[r]
        if W3 is None:
            dg[r] = dh * (h[r] > 0)
        else:
            s = 1 / (1 + torch.exp(-g[r]))
            du[r] = dh * g[r] * s
            dg[r] = dh * u[r] * s * (1 + g[r] * (1 - s))
            dW3[e] = du[r].T @ x[r]
            dx[r] += du[r] @ W3[e]
        dW1[e] = dg[r].T @ x[r]
        dx[r] += dg[r] @ W1[e]
    return dx, dW1, dW3, dW2, dg, du


def combine_backward(dy, y_perm, inv_perm, gate):
    """dy_perm (rows that no pair maps to stay zero) and dgate."""
    dy, y_perm, gate = map(_d, (dy, y_perm, gate))
    n, k = gate.shape
    dyp, dgate = torch.zeros_like(y_perm), torch.zeros(n, k, dtype=torch.float64)
    inv = inv_perm.detach().cpu().long().view(n, k)
    for t in range(n):
        for j in range(k):
            q = int(inv[t, j])
            if 0 <= q < n * k:
                dyp[q] = gate[t, j] * dy[t]
                dgate[t, j] = (dy[t] * y_perm[q]).sum()
    return dyp, dgate


def logits_backward(gate_rule, probs, topk_idx, gate, dgate, f=None, aux=0.0):
    """dl [n, E]; E from probs, or from probs' width given as an int (RENORM without f)."""
    gate, dgate, f = map(_d, (gate, dgate, f))
    idx = topk_idx.detach().cpu().long()
    n, k = gate.shape
    E = probs if isinstance(probs, int) else probs.shape[1]
    p = None if isinstance(probs, int) else _d(probs)
    dl = torch.zeros(n, E, dtype=torch.float64)
    for t in range(n):
        ok = [j for j in range(k) if 0 <= int(idx[t, j]) < E]
        total = sum(float(gate[t, j] * dgate[t, j]) for j in ok)
        for j in ok:
            e = int(idx[t, j])
            dl[t, e] += gate[t, j] * (dgate[t, j] - total if gate_rule == "renorm" else dgate[t, j])
        if gate_rule != "renorm":
            dl[t] -= p[t] * total
        if f is not None:
            dl[t] += aux * E / n * p[t] * (f - (f * p[t]).sum())
    return dl


def route_backward(dl, x, Wg, inv_perm=None, dx_perm=None):
    """dx, dWg, dbias from the logits' gradient (and the expert rows' gradients)."""
    x, Wg, dx_perm = map(_d, (x, Wg, dx_perm))
    dx = dl @ Wg
    if dx_perm is not None:
        n = x.shape[0]
        k = dx_perm.shape[0] // n
        inv = inv_perm.detach().cpu().long().view(n, k)
        for j in range(k):
            ok = (inv[:, j] >= 0) & (inv[:, j] < n * k)
            dx[ok] += dx_perm[inv[ok, j]]
    return dx, dl.T @ x, dl.sum(0)
