"""The training operators of the MoE layer as measured cases.

Six calls make up a training step of a pre-norm MoE layer next to the forward
pass that the library already has: the layer norm in front of the layer and its
gradient, the gated feed-forward block over the expert segments and its
gradient, the combine's gradient, and the router's gradient (joined with the
gradient of the row copies that the dispatch makes).  Each case is one pass
through one of them; ``own`` picks the library's kernels, otherwise the plain
form computes the same from elementary torch operations in 32 bits.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SZ = {"f32": 4, "bf16": 2}
_EPS = 1e-5


# ---------------------------------------------------------------------- cases
def _norm(op, name, n, d, dtype, pad=0):
    return dict(name=name, op=op, n=n, d=d, dtype=dtype, pad=pad)


def _layer(op, name, n, d, F, E, k, dtype, act="swiglu", gate="renorm", skew=0.0, aux=0.0):
    return dict(name=name, op=op, n=n, d=d, F=F, E=E, k=k, dtype=dtype, act=act, gate=gate,
                skew=skew, aux=aux)


def listed():
    return [
        # the norm before one decoded token (the gpt-oss width): launch latency
        _norm("norm_forward", "norm_fwd_token", 1, 2880, "bf16"),
        # the norm before the fine-grained layer's batch: a stream through HBM
        _norm("norm_forward", "norm_fwd_batch", 16384, 7168, "bf16"),
        # fp32 rows of an odd width inside a wider buffer: no whole vectors
        _norm("norm_backward", "norm_bwd_odd", 1021, 1001, "f32", 3),
        # the gradient for the fine-grained layer's batch, with the column sums
        _norm("norm_backward", "norm_bwd_batch", 16384, 7168, "bf16"),
        # the tiny Switch layer (fp32, ReLU): a handful of short launches
        _layer("ffn_forward", "ffn_fwd_tiny_f32", 256, 128, 512, 4, 1, "f32", act="relu",
               gate="top_prob"),
        # the Mixtral-shaped layer's experts: large dense products per segment
        _layer("ffn_forward", "ffn_fwd_mixtral", 4096, 4096, 14336, 8, 2, "bf16"),
        # an eighth of the fine-grained layer's experts with few, uneven rows
        # each: bound by reading the weights and writing their gradients
        _layer("ffn_backward", "ffn_bwd_ragged", 149, 7168, 2048, 32, 4, "bf16", skew=0.6),
        # the Mixtral-shaped layer's gradients: the heaviest call of a step
        _layer("ffn_backward", "ffn_bwd_mixtral", 4096, 4096, 14336, 8, 2, "bf16"),
        # a small uneven batch at the gpt-oss width
        _layer("combine_backward", "combine_bwd_small", 37, 2880, 0, 128, 4, "bf16"),
        # the fine-grained batch: eight expert rows per token through HBM
        _layer("combine_backward", "combine_bwd_batch", 16384, 7168, 0, 256, 8, "bf16"),
        # the tiny Switch router with its load-balancing loss
        _layer("route_backward", "route_bwd_tiny_f32", 256, 128, 0, 4, 1, "f32", gate="top_prob",
               aux=0.01),
        # the fine-grained router: two thin products and the rows' sum
        _layer("route_backward", "route_bwd_batch", 16384, 7168, 0, 256, 8, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_forward", "norm_backward", "ffn_forward", "ffn_backward",
                     "ffn_backward", "combine_backward", "route_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        # (a width of a few elements leaves a gradient that is all cancellation)
        d = _log(rng, 8, 8192)
        if rng.random() < 0.5:
            d = max(8, d // 8 * 8)
        rows = _log(rng, 1, 16384)
        return _norm(op, None, min(rows, max(1, 16384 * 7168 // d)), d, dtype,
                     rng.choice([0, 0, 8, 3])) | {"name": "drawn"}
    E = _log(rng, 1, 64 if op.startswith("ffn") else 256)
    k = rng.randint(1, min(E, 8))
    step = 8 if dtype == "bf16" else 4
    gate = rng.choice(["renorm", "top_prob"])
    skew = rng.choice([0.0, 0.3, 0.6])
    aux = rng.choice([0.0, 0.01])
    act = rng.choice(["swiglu", "swiglu", "relu"])
    if op.startswith("ffn"):
        if dtype == "f32":
            # fp32 layers are the small ones: they run on the CUDA cores
            n, d, F = _log(rng, 1, 1024), _log(rng, 8, 512), _log(rng, 8, 1024)
            E = min(E, 16)
            k = min(k, E, 4)
        else:
            d, F = _log(rng, 16, 7168), _log(rng, 16, 14336)
            # a shorter inner width where the weights or the products would
            # outgrow the Mixtral-shaped layer's
            F = min(F, max(16, 8 * 14336 * 4096 // (E * d)))
            n = min(_log(rng, 1, 4096), max(1, 8192 * 4096 * 14336 // (k * d * F)))
        d, F = max(step, d // step * step), max(step, F // step * step)
    else:
        d, F = max(step, _log(rng, 8, 7168) // step * step), 0
        n = _log(rng, 1, 16384)
        if op == "route_backward":
            # one expert, or one renormalised gate, has a gradient of zero
            E = max(E, 2)
            gate = gate if k > 1 else "top_prob"
            if dtype == "f32":
                n, d = min(n, 2048), min(d, 1024)   # as above: on the CUDA cores
    return _layer(op, "drawn", n, d, F, E, k, dtype, act, gate, skew, aux)


# --------------------------------------------------------------------- inputs
def _randn(g, shape, dtype, std=1.0):
    t = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return t.mul_(std).to(dtype)


def _rows(g, n, d, pad, dtype, std=1.0):
    """n rows of d inside a buffer whose rows are pad elements longer."""
    return _randn(g, (n, d + pad), dtype, std)[:, :d]


def _empty_rows(n, d, pad, dtype):
    return torch.empty(n, d + pad, dtype=dtype, device="cuda")[:, :d]


def _router(c, g):
    """Top-k of noisy scores whose expert popularity falls as rank^-skew."""
    E, k = c["E"], c["k"]
    bias = -c["skew"] * torch.arange(1, E + 1, device="cuda", dtype=torch.float32).log()
    bias = bias[torch.randperm(E, generator=g, device="cuda")]
    logits = _randn(g, (c["n"], E), torch.float32) + bias
    probs = torch.softmax(logits, 1)
    p, idx = torch.sort(probs, dim=1, descending=True, stable=True)
    p, idx = p[:, :k].contiguous(), idx[:, :k].to(torch.int32).contiguous()
    gate = p / p.sum(1, keepdim=True) if c["gate"] == "renorm" else p
    return probs, idx, gate.contiguous()


def _positions(idx, E):
    """offsets [E+1] of the expert segments and inv_perm [n*k] of a stable dispatch."""
    flat = idx.reshape(-1).long()
    perm = torch.sort(flat, stable=True).indices
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(flat.numel(), device="cuda")
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.bincount(flat, minlength=E).cumsum(0)
    return offsets.to(torch.int32), inv.to(torch.int32)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    dt = _DT[c["dtype"]]
    n, d, op = c["n"], c["d"], c["op"]
    s = {"case": c}
    if op.startswith("norm"):
        pad = c["pad"]
        s["x"] = _rows(g, n, d, pad, dt, 2.0).add_(0.5)
        s["gamma"] = (1 + _randn(g, (d,), torch.float32, 0.1)).to(dt)
        if op == "norm_forward":
            s["beta"] = _randn(g, (d,), dt, 0.1)
            s["y"] = _empty_rows(n, d, pad, dt)
            s["mean"] = torch.empty(n, device="cuda")
            s["rstd"] = torch.empty(n, device="cuda")
        else:
            # the statistics that the forward pass left
            x64 = s["x"].double()
            mean = x64.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = torch.rsqrt((x64 - mean[:, None]).square().mean(1) + _EPS).float()
            s["dy"] = _rows(g, n, d, pad, dt)
            s["dx"] = _empty_rows(n, d, pad, dt)
            s["dgamma"] = torch.empty(d, device="cuda")
            s["dbeta"] = torch.empty(d, device="cuda")
        return s
    E, k, F = c["E"], c["k"], c["F"]
    P = n * k
    probs, idx, gate = _router(c, g)
    offsets, inv = _positions(idx, E)
    if op.startswith("ffn"):
        gated = c["act"] == "swiglu"
        s["offsets"] = offsets
        s["longest"] = int((offsets[1:] - offsets[:-1]).max())   # the plain form's padded length
        s["x_perm"] = _randn(g, (P, d), dt)
        s["W1"] = _randn(g, (E, F, d), dt, 0.02)
        s["W3"] = _randn(g, (E, F, d), dt, 0.02) if gated else None
        s["W2"] = _randn(g, (E, d, F), dt, 0.02)
        std = 0.02 * math.sqrt(d)
        if op == "ffn_forward":
            for key in ("g", "u", "h"):
                s[key] = torch.empty(P, F, dtype=dt, device="cuda") if gated or key == "h" else None
            s["y_perm"] = torch.empty(P, d, dtype=dt, device="cuda")
        else:
            # what the forward pass kept: pre-activations of the spread that
            # unit inputs and these weights give
            s["g"] = _randn(g, (P, F), dt, std)
            if gated:
                s["u"] = _randn(g, (P, F), dt, std)
                gf = s["g"].float()
                s["h"] = (gf * torch.sigmoid(gf) * s["u"].float()).to(dt)
            else:
                s["u"], s["h"], s["g"] = None, torch.relu(s["g"]), None
            s["dy_perm"] = _randn(g, (P, d), dt)
            s["dx_perm"] = torch.empty(P, d, dtype=dt, device="cuda")
            for key in ("W1", "W3", "W2"):
                s["d" + key] = None if s[key] is None else torch.empty_like(s[key])
        return s
    s.update(inv_perm=inv, topk_gate=gate)
    if op == "combine_backward":
        s["dy"] = _randn(g, (n, d), dt)
        s["y_perm"] = _randn(g, (P, d), dt)
        s["dy_perm"] = torch.empty(P, d, dtype=dt, device="cuda")
        s["dgate"] = torch.empty(n, k, device="cuda")
        return s
    s.update(probs=probs, topk_idx=idx)
    s["x"] = _randn(g, (n, d), dt)
    s["Wg"] = _randn(g, (E, d), dt, 0.02)
    s["dgate_in"] = _randn(g, (n, k), torch.float32)
    s["f"] = torch.bincount(idx[:, 0].long(), minlength=E).float() / n if c["aux"] else None
    s["dx_perm"] = _randn(g, (P, d), dt)
    s["dx"] = torch.empty(n, d, dtype=dt, device="cuda")
    s["dWg"] = torch.empty(E, d, dtype=dt, device="cuda")
    s["dbias"] = torch.empty(E, device="cuda")
    return s


# ----------------------------------------------------- the library's own calls
def _library(s):
    """The binding, the layer's configuration and its workspace: a program makes them once."""
    if "lib" not in s:
        from mixture_experts_layer_moe_gb300 import moe
        c = s["case"]
        if c["op"].startswith("norm"):
            ws = None
            if c["op"] == "norm_backward":
                ws = torch.zeros(moe.moe_layernorm_workspace_size(c["n"], c["d"], c["dtype"]),
                                 dtype=torch.uint8, device="cuda")
            s["lib"] = (moe, None, ws, None, None)
        else:
            # a call of the combine or the router does not meet the inner
            # width: the smallest legal one
            cfg = moe.moe_config(c["n"], c["d"], c["F"] or 8, c["E"], c["k"],
                                 moe._DTYPE[c["dtype"]], moe._DTYPE[c["dtype"]],
                                 moe._GATE[c["gate"]], moe._ACT[c["act"]], 0)
            w = moe.make_weights({key: s.get(key) for key in ("Wg", "W1", "W3", "W2")})
            grads = moe.make_expert_grads({key: s.get("d" + key) for key in ("W1", "W3", "W2")})
            s["lib"] = (moe, cfg, moe.alloc_train_workspace(cfg), w, grads)
    return s["lib"]


def _run_own(s):
    op = s["case"]["op"]
    moe, cfg, ws, w, grads = _library(s)
    if op == "norm_forward":
        moe.moe_layernorm(s["x"], s["gamma"], s["beta"], s["y"], s["mean"], s["rstd"], _EPS)
        return s["y"], s["mean"], s["rstd"]
    if op == "norm_backward":
        moe.moe_layernorm_backward(s["x"], s["gamma"], s["mean"], s["rstd"], s["dy"], s["dx"],
                                   s["dgamma"], s["dbeta"], ws)
        return s["dx"], s["dgamma"], s["dbeta"]
    if op == "ffn_forward":
        moe.moe_expert_ffn_train(cfg, s["x_perm"], s["offsets"], w, s["g"], s["u"], s["h"],
                                 s["y_perm"], ws)
        return [t for t in (s["y_perm"], s["g"], s["u"], s["h"]) if t is not None]
    if op == "ffn_backward":
        moe.moe_expert_ffn_backward(cfg, s["x_perm"], s["offsets"], w, s["g"], s["u"], s["h"],
                                    s["dy_perm"], s["dx_perm"], grads, ws)
        return [t for t in (s["dx_perm"], s["dW1"], s["dW3"], s["dW2"]) if t is not None]
    if op == "combine_backward":
        moe.moe_combine_backward(cfg, s["dy"], s["y_perm"], s["inv_perm"], s["topk_gate"],
                                 s["dy_perm"], s["dgate"], ws)
        return s["dy_perm"], s["dgate"]
    moe.moe_route_backward(cfg, s["x"], w, s["probs"], s["topk_idx"], s["topk_gate"],
                           s["dgate_in"], s["f"], s["case"]["aux"], s["inv_perm"], s["dx_perm"],
                           s["dx"], s["dWg"], s["dbias"], ws)
    return s["dx"], s["dWg"], s["dbias"]


# --------------------------------------------------------------- plain forms
def _plain_norm_forward(s):
    x = s["x"].float()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = torch.rsqrt(xc.square().mean(1) + _EPS)
    y = xc * rstd[:, None] * s["gamma"].float() + s["beta"].float()
    return y.to(s["x"].dtype), mean, rstd


def _plain_norm_backward(s):
    dy = s["dy"].float()
    xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    w = dy * s["gamma"].float()
    dx = s["rstd"][:, None] * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True))
    return dx.to(s["x"].dtype), (dy * xh).sum(0), dy.sum(0)


def _padded(s):
    """Row -> its slot in segments padded to the longest one, and the two copies."""
    off, E, longest = s["offsets"].long(), s["case"]["E"], s["longest"]
    rows = torch.arange(s["x_perm"].shape[0], device="cuda")
    e = torch.searchsorted(off[1:].contiguous(), rows, right=True)
    slot = e * longest + rows - off[e]

    def pad(t):
        out = torch.zeros(E * longest, t.shape[1], device="cuda")
        out[slot] = t.float()
        return out.view(E, longest, t.shape[1])

    def unpad(t):
        return t.reshape(E * longest, -1)[slot]

    return pad, unpad


def _plain_ffn_forward(s):
    pad, unpad = _padded(s)
    dt = s["x_perm"].dtype
    x = pad(s["x_perm"])
    g = torch.bmm(x, s["W1"].float().transpose(1, 2))
    if s["W3"] is None:
        h = torch.relu(g)
        y = torch.bmm(h, s["W2"].float().transpose(1, 2))
        return [unpad(y).to(dt), unpad(h).to(dt)]
    u = torch.bmm(x, s["W3"].float().transpose(1, 2))
    h = g / (1 + torch.exp(-g)) * u
    y = torch.bmm(h, s["W2"].float().transpose(1, 2))
    return [unpad(y).to(dt), unpad(g).to(dt), unpad(u).to(dt), unpad(h).to(dt)]


def _plain_ffn_backward(s):
    pad, unpad = _padded(s)
    dt = s["x_perm"].dtype
    x, dy, h = pad(s["x_perm"]), pad(s["dy_perm"]), pad(s["h"])
    dh = torch.bmm(dy, s["W2"].float())
    dW2 = torch.bmm(dy.transpose(1, 2), h).to(dt)
    if s["W3"] is None:
        dg = dh * (h > 0)
        dx = torch.bmm(dg, s["W1"].float())
        return [unpad(dx).to(dt), torch.bmm(dg.transpose(1, 2), x).to(dt), dW2]
    g, u = pad(s["g"]), pad(s["u"])
    sg = 1 / (1 + torch.exp(-g))
    dg = dh * u * sg * (1 + g * (1 - sg))
    du = dh * g * sg
    dx = torch.bmm(dg, s["W1"].float()) + torch.bmm(du, s["W3"].float())
    return [unpad(dx).to(dt), torch.bmm(dg.transpose(1, 2), x).to(dt),
            torch.bmm(du.transpose(1, 2), x).to(dt), dW2]


def _plain_combine_backward(s):
    c = s["case"]
    dy, inv = s["dy"].float(), s["inv_perm"].long()
    dgate = (s["y_perm"].float()[inv].view(c["n"], c["k"], -1) * dy[:, None]).sum(2)
    dyp = torch.empty_like(s["y_perm"])
    dyp[inv] = (s["topk_gate"][:, :, None] * dy[:, None]).reshape(-1, c["d"]).to(dyp.dtype)
    return dyp, dgate


def _plain_route_backward(s):
    c = s["case"]
    p, gate, dgate, idx = s["probs"], s["topk_gate"], s["dgate_in"], s["topk_idx"].long()
    dl = torch.zeros_like(p)
    if c["gate"] == "renorm":
        dl.scatter_(1, idx, gate * (dgate - (gate * dgate).sum(1, keepdim=True)))
    else:
        dl.scatter_(1, idx, gate * dgate)
        dl -= p * (gate * dgate).sum(1, keepdim=True)
    if s["f"] is not None:
        dl += c["aux"] * c["E"] / c["n"] * p * (s["f"] - (p * s["f"]).sum(1, keepdim=True))
    rows = s["dx_perm"].float()[s["inv_perm"].long()].view(c["n"], c["k"], -1).sum(1)
    dx = (rows + dl @ s["Wg"].float()).to(s["x"].dtype)
    return dx, (dl.t() @ s["x"].float()).to(s["x"].dtype), dl.sum(0)


_PLAIN = {"norm_forward": _plain_norm_forward, "norm_backward": _plain_norm_backward,
          "ffn_forward": _plain_ffn_forward, "ffn_backward": _plain_ffn_backward,
          "combine_backward": _plain_combine_backward, "route_backward": _plain_route_backward}


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


# ----------------------------------------------------------------------- work
def work(case):
    c = case
    z, n, d, op = _SZ[c["dtype"]], c["n"], c["d"], c["op"]
    if op == "norm_forward":
        return {"bytes": 2 * n * d * z + 8 * n + 2 * d * z, "flops": 8 * n * d}
    if op == "norm_backward":
        return {"bytes": 3 * n * d * z + 8 * n + d * z + 8 * d, "flops": 14 * n * d}
    k, E, F = c["k"], c["E"], c["F"]
    P = n * k
    mats = 3 if c["act"] == "swiglu" else 2
    if op == "ffn_forward":
        # the weights of the experts that can have rows; g, u and h are outputs
        return {"bytes": z * (2 * P * d + (1 if mats == 2 else 3) * P * F
                              + mats * min(E, P) * F * d),
                "flops": 2 * mats * P * F * d}
    if op == "ffn_backward":
        return {"bytes": z * (3 * P * d + (1 if mats == 2 else 3) * P * F
                              + mats * (min(E, P) + E) * F * d),
                "flops": 4 * mats * P * F * d}
    if op == "combine_backward":
        return {"bytes": z * (n * d + 2 * P * d) + 12 * P, "flops": 3 * P * d}
    dense = c["gate"] != "renorm" or c["aux"]
    return {"bytes": z * (2 * n * d + P * d + 2 * E * d) + (4 * n * E if dense else 0) + 16 * P,
            "flops": 4 * n * d * (E if dense else k) + P * d}


# --------------------------------------------------- the definitions in 64 bits
def _segments(s):
    off = s["offsets"].tolist()
    return list(zip(off[:-1], off[1:]))


def _exact_ffn(s, backward):
    out = {}
    P, d = s["x_perm"].shape
    F, E = s["W1"].shape[1], s["W1"].shape[0]
    gated = s["W3"] is not None
    f64 = dict(dtype=torch.float64, device="cuda")
    if backward:
        out["dx"] = torch.zeros(P, d, **f64)
        out["dW1"] = torch.zeros(E, F, d, **f64)
        if gated:
            out["dW3"] = torch.zeros(E, F, d, **f64)
        out["dW2"] = torch.zeros(E, d, F, **f64)
    else:
        out["y"] = torch.zeros(P, d, **f64)
        for key in (("g", "u", "h") if gated else ("h",)):
            out[key] = torch.zeros(P, F, **f64)
    for e, (a, b) in enumerate(_segments(s)):
        if a == b:
            continue
        x, W1, W2 = s["x_perm"][a:b].double(), s["W1"][e].double(), s["W2"][e].double()
        W3 = s["W3"][e].double() if gated else None
        if not backward:
            g = x @ W1.T
            if gated:
                u = x @ W3.T
                h = g * torch.sigmoid(g) * u
                out["g"][a:b], out["u"][a:b] = g, u
            else:
                h = g.clamp(min=0)
            out["h"][a:b], out["y"][a:b] = h, h @ W2.T
            continue
        dy, h = s["dy_perm"][a:b].double(), s["h"][a:b].double()
        dh = dy @ W2
        out["dW2"][e] = dy.T @ h
        if gated:
            g, u = s["g"][a:b].double(), s["u"][a:b].double()
            sg = torch.sigmoid(g)
            du = dh * g * sg
            dg = dh * u * (sg + g * sg * (1 - sg))
            out["dx"][a:b] = dg @ W1 + du @ W3
            out["dW3"][e] = du.T @ x
        else:
            dg = torch.where(h > 0, dh, torch.zeros_like(dh))
            out["dx"][a:b] = dg @ W1
        out["dW1"][e] = dg.T @ x
    return list(out.values())


def exact(case, seed):
    # about 1 TFLOP/s in 64 bits on this card
    if work(case)["flops"] > 12e12:
        return None
    s = prepare(case, seed)
    c = s["case"]
    op, n, d = c["op"], c["n"], c["d"]
    if op == "norm_forward":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1 / torch.sqrt(var + _EPS)
        y = torch.addcmul(s["beta"].double(), (x - mean[:, None]) * rstd[:, None],
                          s["gamma"].double())
        return y, mean, rstd
    if op == "norm_backward":
        x, dy, rstd = s["x"].double(), s["dy"].double(), s["rstd"].double()[:, None]
        xh = (x - s["mean"].double()[:, None]) * rstd
        w = dy * s["gamma"].double()
        dx = rstd * (w - (w.sum(1, keepdim=True) + xh * (w * xh).sum(1, keepdim=True)) / d)
        return dx, torch.einsum("nd,nd->d", dy, xh), dy.sum(0)
    if op.startswith("ffn"):
        return _exact_ffn(s, op == "ffn_backward")
    k, E = c["k"], c["E"]
    inv = s["inv_perm"].long().view(n, k)
    if op == "combine_backward":
        dyp = torch.zeros(n * k, d, dtype=torch.float64, device="cuda")
        dgate = torch.zeros(n, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            dyp[inv[:, j]] = s["dy"].double() * s["topk_gate"][:, j:j + 1].double()
            dgate[:, j] = torch.einsum("nd,nd->n", s["dy"].double(),
                                       s["y_perm"][inv[:, j]].double())
        return dyp, dgate
    # router: the Jacobian of the gates with respect to the logits, applied row by row
    p, gate, dg = s["probs"].double(), s["topk_gate"].double(), s["dgate_in"].double()
    chosen = torch.zeros(n, E, dtype=torch.float64, device="cuda")
    chosen.scatter_(1, s["topk_idx"].long(), gate * dg)
    total = chosen.sum(1, keepdim=True)
    if c["gate"] == "renorm":
        share = torch.zeros_like(chosen).scatter_(1, s["topk_idx"].long(), gate)
        dl = chosen - share * total
    else:
        dl = chosen - p * total
    if s["f"] is not None:
        f = s["f"].double()
        dl = dl + (c["aux"] * E / n) * p * (f - (p @ f)[:, None])
    dx = dl @ s["Wg"].double()
    for j in range(k):
        dx += s["dx_perm"][inv[:, j]].double()
    return dx, dl.T @ s["x"].double(), dl.sum(0)
