"""The operators round the MoE layer in a training step, as measured cases.

Three operators join the layer to the rest of a step: the block joint (the norm
after the block, its gate and dropout, the scaled residual and the norm before
the next block, in one pass) with its gradient, dropout from a counter-based
generator, and the softmax cross entropy of a linear layer over the vocabulary
with its gradient.  Each case is one pass through one of them; ``own`` picks the
library's kernels, otherwise the plain form computes the same from elementary
torch operations in 32 bits.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SZ = {"f32": 4, "bf16": 2}
_EPS = 1e-5
_NORMS = ("none", "rms", "layer")


# ---------------------------------------------------------------------- cases
def _join(op, name, n, d, dtype, post="rms", pre="rms", gate=True, p=0.0, scale=1.0, pad=0):
    return dict(name=name, op=op, n=n, d=d, dtype=dtype, post=post, pre=pre, gate=gate, p=p,
                scale=scale, pad=pad)


def _drop(name, n, d, dtype, p, pad=0):
    return dict(name=name, op="dropout", n=n, d=d, dtype=dtype, p=p, pad=pad)


def _loss(op, name, n, d, V, dtype, ignored=0.0, z_loss=0.0):
    return dict(name=name, op=op, n=n, d=d, V=V, dtype=dtype, ignored=ignored, z_loss=z_loss)


def listed():
    return [
        # the joint between two blocks for one decoded token (the gpt-oss
        # width): launch latency
        _join("join_forward", "join_fwd_token", 1, 2880, "bf16"),
        # the joint behind the fine-grained layer's training batch, with dropout
        # on the block's output: a stream through HBM
        _join("join_forward", "join_fwd_batch", 16384, 7168, "bf16", p=0.1),
        # fp32 rows of an odd width inside a wider buffer: no whole vectors
        _join("join_backward", "join_bwd_odd", 1021, 1001, "f32", "layer", "layer", p=0.1,
              scale=0.5, pad=3),
        # the gradient for the fine-grained layer's batch, with its column sums
        _join("join_backward", "join_bwd_batch", 16384, 7168, "bf16", p=0.1),
        # dropout on a small uneven batch at the gpt-oss width
        _drop("dropout_small", 37, 2880, "bf16", 0.1),
        # dropout on the fine-grained batch: a stream through HBM
        _drop("dropout_batch", 16384, 7168, "bf16", 0.1),
        # the loss of one token at the gpt-oss width over a large vocabulary:
        # bound by reading the matrix
        _loss("loss_forward", "loss_fwd_token", 1, 2880, 131072, "bf16"),
        # the loss of a batch at the Mixtral width: a large dense product whose
        # result is never stored
        _loss("loss_forward", "loss_fwd_batch", 4096, 4096, 131072, "bf16", z_loss=1e-4),
        # a tiny fp32 model's loss over an odd vocabulary: a few short launches
        _loss("loss_forward", "loss_fwd_tiny_f32", 256, 128, 4099, "f32"),
        # the gradient of a small, half padded batch at the fine-grained width
        # over an odd vocabulary: bound by the matrix and its gradient
        _loss("loss_backward", "loss_bwd_ragged", 149, 7168, 32003, "bf16", ignored=0.5),
        # the gradient of the batch at the Mixtral width: the heaviest call
        _loss("loss_backward", "loss_bwd_batch", 4096, 4096, 65536, "bf16", ignored=0.1,
              z_loss=1e-4),
        # the tiny fp32 model's gradient
        _loss("loss_backward", "loss_bwd_tiny_f32", 256, 128, 4099, "f32", ignored=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["join_forward", "join_backward", "dropout", "loss_forward", "loss_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if not op.startswith("loss"):
        # (a width of a few elements leaves a gradient that is all cancellation)
        d = _log(rng, 16, 8192)
        if rng.random() < 0.5:
            d = max(16, d // 8 * 8)
        n = min(_log(rng, 1, 16384), max(1, 16384 * 7168 // d))
        if dtype == "f32":
            n = max(1, n // 2)
        pad = rng.choice([0, 0, 8, 3])
        p = rng.choice([0.0, 0.1, 0.5])
        if op == "dropout":
            return _drop("drawn", n, d, dtype, p or 0.25, pad)
        return _join(op, "drawn", n, d, dtype, rng.choice(_NORMS), rng.choice(_NORMS),
                     rng.random() < 0.6, p, rng.choice([1.0, 0.5]), pad)
    if dtype == "f32":
        # fp32 models are the small ones: they run on the CUDA cores
        n, d, V = _log(rng, 1, 1024), _log(rng, 8, 512) // 4 * 4, _log(rng, 256, 8192)
    else:
        n, d, V = _log(rng, 1, 8192), _log(rng, 64, 8192) // 8 * 8, _log(rng, 256, 131072)
        # fewer tokens where the products, or the plain form's logits, would
        # outgrow the Mixtral width's batch
        n = min(n, max(1, 4096 * 4096 * 65536 // (d * V)), 4096 * 131072 // V)
    return _loss(op, "drawn", n, d, V, dtype, rng.choice([0.0, 0.1, 0.5]),
                 rng.choice([0.0, 1e-4]))


# --------------------------------------------------------------------- inputs
def _randn(g, shape, dtype, std=1.0):
    t = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return t.mul_(std).to(dtype)


def _rows(g, n, d, pad, dtype, std=1.0):
    """n rows of d inside a buffer whose rows are pad elements longer."""
    return _randn(g, (n, d + pad), dtype, std)[:, :d]


def _empty_rows(n, d, pad, dtype):
    return torch.empty(n, d + pad, dtype=dtype, device="cuda")[:, :d]


def _statistics(v, kind):
    """mean and 1 / deviation of the rows of v (64 bits) as a norm of this kind takes them."""
    n = v.shape[0]
    if kind == "none":
        return v.new_zeros(n), v.new_ones(n)
    mean = v.mean(1) if kind == "layer" else v.new_zeros(n)
    return mean, torch.rsqrt((v - mean[:, None]).square().mean(1) + _EPS)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 29)
    dt, n, d, op = _DT[c["dtype"]], c["n"], c["d"], c["op"]
    s = {"case": c}
    if op.startswith("loss"):
        V = c["V"]
        s["W"] = _randn(g, (V, d), dt, 1.5 / math.sqrt(d))
        t = torch.randint(V, (n,), generator=g, device="cuda")
        # hidden rows that point at their next token, some more than others
        boost = 10 * torch.rand(n, 1, generator=g, device="cuda") / (1.5 * 1.5)
        s["x"] = (_randn(g, (n, d), torch.float32) + boost * s["W"][t].float()).to(dt)
        ignored = torch.rand(n, generator=g, device="cuda") < c["ignored"]
        s["targets"] = torch.where(ignored, -1, t).to(torch.int32)
        s["lse"] = torch.empty(n, device="cuda")
        if op == "loss_forward":
            s["loss"] = torch.empty(n, device="cuda")
        else:
            # what the forward pass left, and the gradient of the mean over the tokens that count
            for a in range(0, n, 1024):
                s["lse"][a:a + 1024] = torch.logsumexp(s["x"][a:a + 1024].float() @ s["W"].float().T, 1)
            s["lse"].masked_fill_(ignored, 0.0)
            count = (~ignored).sum().clamp(min=1)
            s["dloss"] = torch.where(ignored, 0.0, 1.0 / count).float()
            s["dx"], s["dW"] = torch.empty_like(s["x"]), torch.empty_like(s["W"])
        return s
    pad = c["pad"]
    if c["p"]:
        # seed and offset of the generator, as a training step keeps them on the device
        s["rng"] = torch.randint(2 ** 62, (2,), generator=g, device="cuda")
    if op == "dropout":
        s["x"] = _rows(g, n, d, pad, dt)
        s["y"] = _empty_rows(n, d, pad, dt)
        return s
    s["params"] = {}
    if c["gate"]:
        s["params"]["gate"] = _randn(g, (d,), dt, 0.3).add_(0.5)
    for side in ("post", "pre"):
        if c[side] != "none":
            s["params"][side + "_gamma"] = (1 + _randn(g, (d,), torch.float32, 0.1)).to(dt)
        if c[side] == "layer":
            s["params"][side + "_beta"] = _randn(g, (d,), dt, 0.1)
    # the block's output, small against the residual stream
    s["b"] = _rows(g, n, d, pad, dt, 0.4).add_(0.05)
    if op == "join_forward":
        s["x"] = _rows(g, n, d, pad, dt, 2.0).add_(0.3)
        s["r"] = _empty_rows(n, d, pad, dt)
        s["y"] = _empty_rows(n, d, pad, dt) if c["pre"] != "none" else None
        s["stats"] = torch.empty(4, n, device="cuda")
        return s
    # what the forward pass left: the joined rows and the statistics of both norms
    s["r"] = _rows(g, n, d, pad, dt, 2.0).add_(0.3)
    s["stats"] = torch.empty(4, n, device="cuda")
    for i, (rows, kind) in enumerate(((s["b"], c["post"]), (s["r"], c["pre"]))):
        for a in range(0, n, 4096):
            mean, rstd = _statistics(rows[a:a + 4096].double(), kind)
            s["stats"][2 * i, a:a + 4096], s["stats"][2 * i + 1, a:a + 4096] = mean, rstd
    s["dr"] = _rows(g, n, d, pad, dt)
    s["dy"] = _rows(g, n, d, pad, dt) if c["pre"] != "none" else None
    s["dx"], s["db"] = _empty_rows(n, d, pad, dt), _empty_rows(n, d, pad, dt)
    s["grads"] = {key: torch.empty(d, device="cuda") for key in s["params"]}
    return s


# ----------------------------------------------------- the library's own calls
def _library(s):
    """The binding, the parameters' handles and the workspace: a program makes them once."""
    if "lib" not in s:
        from mixture_experts_layer_moe_gb300 import moe
        c, ws, params, grads = s["case"], None, None, None
        if c["op"].startswith("loss"):
            ws = moe.alloc_cross_entropy_workspace(c["n"], c["d"], c["V"], c["dtype"])
        elif c["op"].startswith("join"):
            params = moe.make_join_params(s["params"])
            if c["op"] == "join_backward":
                grads = moe.make_join_grads(s["grads"])
                ws = torch.zeros(moe.moe_block_join_workspace_size(c["n"], c["d"], c["dtype"]),
                                 dtype=torch.uint8, device="cuda")
        s["lib"] = (moe, ws, params, grads)
    return s["lib"]


def _run_own(s):
    c = s["case"]
    op = c["op"]
    moe, ws, params, grads = _library(s)
    if op == "dropout":
        moe.moe_dropout(s["x"], s["y"], c["p"], s["rng"])
        return s["y"]
    if op == "join_forward":
        moe.moe_block_join(s["x"], s["b"], params, s["r"], s["y"], s["stats"], post=c["post"],
                           pre=c["pre"], scale=c["scale"], p=c["p"], rng=s.get("rng"), eps=_EPS)
        return [t for t in (s["r"], s["y"], s["stats"]) if t is not None]
    if op == "join_backward":
        moe.moe_block_join_backward(s["b"], s["r"], s["stats"], params, s["dr"], s["dy"], s["dx"],
                                    s["db"], grads, ws, post=c["post"], pre=c["pre"],
                                    scale=c["scale"], p=c["p"], rng=s.get("rng"))
        return [s["dx"], s["db"], *s["grads"].values()]
    if op == "loss_forward":
        moe.moe_cross_entropy(s["x"], s["W"], s["targets"], s["loss"], s["lse"], ws,
                              z_loss=c["z_loss"])
        return s["loss"], s["lse"]
    moe.moe_cross_entropy_backward(s["x"], s["W"], s["targets"], s["lse"], s["dloss"], s["dx"],
                                   s["dW"], ws, z_loss=c["z_loss"])
    return s["dx"], s["dW"]


# --------------------------------------------------------------- plain forms
def _mul_hi_lo(a, b):
    """Upper and lower 32 bits of a * b, b a tensor of 32-bit values in int64."""
    high = (a * (b >> 16) + ((a * (b & 0xFFFF)) >> 16)) >> 16
    return high, (a * b) & 0xFFFFFFFF


def _threshold(p):
    return int(math.floor(p * 65536 + 0.5))


def _kept(rng, n, d, p):
    """Which elements of n rows of d dropout keeps: 16 bits each of Philox4x32-10, whose key is
    the seed rng[0] and whose counter is (column / 8, row, offset rng[1])."""
    mask = 0xFFFFFFFF
    blocks = (d + 7) // 8
    c0 = torch.arange(blocks, device="cuda").expand(n, blocks)
    c1 = torch.arange(n, device="cuda")[:, None].expand(n, blocks)
    c2, c3 = (rng[1] & mask).expand(n, blocks), ((rng[1] >> 32) & mask).expand(n, blocks)
    k0, k1 = rng[0] & mask, (rng[0] >> 32) & mask
    for _ in range(10):
        h0, l0 = _mul_hi_lo(0xD2511F53, c0)
        h1, l1 = _mul_hi_lo(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & mask, (k1 + 0xBB67AE85) & mask
    words = torch.stack((c0, c1, c2, c3), 2)
    bits = torch.stack((words & 0xFFFF, words >> 16), 3)
    return bits.reshape(n, blocks * 8)[:, :d] >= _threshold(p)


def _dropped(v, s):
    """Dropout of the fp32 rows v."""
    c = s["case"]
    if not c["p"]:
        return v
    keep = _kept(s["rng"], *v.shape, c["p"])
    return torch.where(keep, v * (1 / (1 - _threshold(c["p"]) / 65536)), 0.0)


def _plain_norm(v, kind, gamma, beta):
    n = v.shape[0]
    if kind == "none":
        return v, v.new_zeros(n), v.new_ones(n)
    mean = v.mean(1) if kind == "layer" else v.new_zeros(n)
    vc = v - mean[:, None]
    rstd = torch.rsqrt(vc.square().mean(1) + _EPS)
    out = vc * rstd[:, None] * gamma.float()
    return (out if beta is None else out + beta.float()), mean, rstd


def _plain_dropout(s):
    return _dropped(s["x"].float(), s).to(s["x"].dtype)


def _plain_join_forward(s):
    c, get = s["case"], s["params"].get
    dt = s["x"].dtype
    z, m1, r1 = _plain_norm(s["b"].float(), c["post"], get("post_gamma"), get("post_beta"))
    z = _dropped(z, s)
    if c["gate"]:
        z = z * get("gate").float()
    r = c["scale"] * s["x"].float() + z
    y, m2, r2 = _plain_norm(r, c["pre"], get("pre_gamma"), get("pre_beta"))
    stats = torch.stack((m1, r1, m2, r2))
    return [r.to(dt), stats] if c["pre"] == "none" else [r.to(dt), y.to(dt), stats]


def _plain_norm_gradient(w, xh, rstd, kind):
    """Gradient of the normed rows from w = the output's gradient times gamma."""
    if kind == "none":
        return w
    t = w - xh * (w * xh).mean(1, keepdim=True)
    if kind == "layer":
        t = t - w.mean(1, keepdim=True)
    return rstd[:, None] * t


def _plain_join_backward(s):
    c, get = s["case"], s["params"].get
    dt = s["b"].dtype
    m1, r1, m2, r2 = s["stats"]
    grads = {}
    d_r = s["dr"].float()
    if c["pre"] != "none":
        rh = (s["r"].float() - m2[:, None]) * r2[:, None]
        dy = s["dy"].float()
        grads["pre_gamma"], grads["pre_beta"] = (dy * rh).sum(0), dy.sum(0)
        d_r = d_r + _plain_norm_gradient(dy * get("pre_gamma").float(), rh, r2, c["pre"])
    bh = (s["b"].float() - m1[:, None]) * r1[:, None]
    u = _dropped(d_r, s)
    z = bh
    if c["post"] != "none":
        z = z * get("post_gamma").float()
    if c["post"] == "layer":
        z = z + get("post_beta").float()
    dz = u
    if c["gate"]:
        grads["gate"] = (u * z).sum(0)
        dz = u * get("gate").float()
    w = dz
    if c["post"] != "none":
        grads["post_gamma"], grads["post_beta"] = (dz * bh).sum(0), dz.sum(0)
        w = dz * get("post_gamma").float()
    db = _plain_norm_gradient(w, bh, r1, c["post"])
    return [(c["scale"] * d_r).to(dt), db.to(dt), *(grads[key] for key in s["params"])]


def _plain_logits(s):
    logits = s["x"].float() @ s["W"].float().T
    t = s["targets"].long()
    return logits, t, t >= 0


def _plain_loss_forward(s):
    logits, t, valid = _plain_logits(s)
    top = logits.amax(1)
    lse = top + torch.log(torch.exp(logits - top[:, None]).sum(1))
    at = logits.gather(1, t.clamp(min=0)[:, None])[:, 0]
    loss = lse - at + s["case"]["z_loss"] * lse * lse
    return torch.where(valid, loss, 0.0), torch.where(valid, lse, 0.0)


def _plain_loss_backward(s):
    logits, t, valid = _plain_logits(s)
    lse = s["lse"]
    dl = torch.exp(logits - lse[:, None]) * (1 + 2 * s["case"]["z_loss"] * lse)[:, None]
    dl[torch.arange(len(t), device="cuda"), t.clamp(min=0)] -= 1
    dl = torch.where(valid[:, None], dl * s["dloss"][:, None], 0.0)
    dt = s["x"].dtype
    return (dl @ s["W"].float()).to(dt), (dl.T @ s["x"].float()).to(dt)


_PLAIN = {"dropout": _plain_dropout, "join_forward": _plain_join_forward,
          "join_backward": _plain_join_backward, "loss_forward": _plain_loss_forward,
          "loss_backward": _plain_loss_backward}


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


# ----------------------------------------------------------------------- work
def work(case):
    c = case
    z, n, d, op = _SZ[c["dtype"]], c["n"], c["d"], c["op"]
    if op == "dropout":
        return {"bytes": 2 * n * d * z + 16, "flops": 2 * n * d}
    if op.startswith("loss"):
        counted = n * (1 - c["ignored"])
        if op == "loss_forward":
            return {"bytes": z * d * (n + c["V"]) + 12 * n, "flops": 2 * counted * c["V"] * d}
        return {"bytes": 2 * z * d * (n + c["V"]) + 12 * n, "flops": 6 * counted * c["V"] * d}
    pre, post = c["pre"] != "none", c["post"] != "none"
    vectors = c["gate"] + sum({"none": 0, "rms": 1, "layer": 2}[c[k]] for k in ("post", "pre"))
    if op == "join_forward":
        return {"bytes": z * d * ((3 + pre) * n + vectors) + 16 * n,
                "flops": (4 + 6 * post + 6 * pre) * n * d}
    rows = 3 + (1 if post or c["gate"] else 0) + 2 * pre
    return {"bytes": z * d * (rows * n + vectors) + 4 * d * vectors + 16 * n,
            "flops": (4 + 12 * post + 12 * pre) * n * d}


# --------------------------------------------------- the definitions in 64 bits
def _exact_keep(rng, n, d, p):
    """The kept elements as a factor of each: 0, or 1 / (1 - p)."""
    seed, offset = (int(v) for v in rng.cpu())
    low = np.uint64(0xFFFFFFFF)
    shift = np.uint64(32)
    out = np.empty((n, -(-d // 8), 8), dtype=bool)
    drop = round(p * 65536)
    col = np.arange(out.shape[1], dtype=np.uint64)[None, :]
    for a in range(0, n, 1024):
        row = np.arange(a, min(n, a + 1024), dtype=np.uint64)[:, None]
        x = [np.broadcast_to(v, (row.shape[0], col.shape[1])) for v in
             (col, row, np.uint64(offset & 0xFFFFFFFF), np.uint64(offset >> 32))]
        key = [seed & 0xFFFFFFFF, seed >> 32]
        for _ in range(10):
            even, odd = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
            x = [(odd >> shift) ^ x[1] ^ np.uint64(key[0]), odd & low,
                 (even >> shift) ^ x[3] ^ np.uint64(key[1]), even & low]
            key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
        for i, word in enumerate(x):
            out[a:a + 1024, :, 2 * i] = word % np.uint64(65536) >= drop
            out[a:a + 1024, :, 2 * i + 1] = word // np.uint64(65536) >= drop
    keep = torch.from_numpy(out.reshape(n, -1)[:, :d].copy()).cuda()
    return keep.double() * (65536 / (65536 - drop))


def _exact_join(s, forward):
    c = s["case"]
    n, d = s["b"].shape
    P = {key: v.double() for key, v in s["params"].items()}
    gate = P.get("gate", torch.ones(d, dtype=torch.float64, device="cuda"))
    factor = _exact_keep(s["rng"], n, d, c["p"]) if c["p"] else None
    out, sums = None, {key: torch.zeros(d, dtype=torch.float64, device="cuda") for key in P}

    def normed(v, side, given=None):
        if c[side] == "none":
            return v, v, None
        if given is None:
            mean = v.sum(1, keepdim=True) / d if c[side] == "layer" else 0 * v[:, :1]
            dev = torch.sqrt(((v - mean) ** 2).sum(1, keepdim=True) / d + _EPS)
            stats = (mean, 1 / dev)
        else:
            stats = given
        h = (v - stats[0]) * stats[1]
        return h, h * P[side + "_gamma"] + P.get(side + "_beta", 0.0), stats

    def back(w, h, rstd, side):
        if c[side] == "none":
            return w
        dot = torch.einsum("nd,nd->n", w, h)[:, None] / d
        return rstd * (w - h * dot - (w.sum(1, keepdim=True) / d if c[side] == "layer" else 0.0))

    for a in range(0, n, 2048):
        sl = slice(a, min(n, a + 2048))
        f = 1.0 if factor is None else factor[sl]
        b = s["b"][sl].double()
        if forward:
            _, z, st1 = normed(b, "post")
            r = c["scale"] * s["x"][sl].double() + gate * (f * z)
            _, y, st2 = normed(r, "pre")
            one = torch.ones_like(r[:, :1])
            st = [t for pair in (st1, st2) for t in (pair or (0 * one, one))]
            part = [r] + ([y] if c["pre"] != "none" else []) + [torch.cat(st, 1).T]
        else:
            st = [v[sl, None].double() for v in s["stats"]]
            total = s["dr"][sl].double()
            if c["pre"] != "none":
                h, _, _ = normed(s["r"][sl].double(), "pre", st[2:])
                dy = s["dy"][sl].double()
                total = total + back(dy * P["pre_gamma"], h, st[3], "pre")
                sums["pre_gamma"] += torch.einsum("nd,nd->d", dy, h)
                if "pre_beta" in sums:
                    sums["pre_beta"] += dy.sum(0)
            h, z, _ = normed(b, "post", st[:2])
            u = f * total
            if c["gate"]:
                sums["gate"] += torch.einsum("nd,nd->d", u, z)
            w = u * gate
            if c["post"] != "none":
                sums["post_gamma"] += torch.einsum("nd,nd->d", w, h)
                if "post_beta" in sums:
                    sums["post_beta"] += w.sum(0)
                w = w * P["post_gamma"]
            part = [c["scale"] * total, back(w, h, st[1], "post")]
        if out is None:
            out = [torch.empty((4, n) if forward and i == len(part) - 1 else (n, d),
                               dtype=torch.float64, device="cuda") for i in range(len(part))]
        for i, t in enumerate(part):
            if out[i].shape == (4, n) and forward and i == len(part) - 1:
                out[i][:, sl] = t
            else:
                out[i][sl] = t
    return out if forward else [*out, *(sums[key] for key in s["params"])]


def _exact_loss(s, forward):
    c = s["case"]
    n, V, d = c["n"], c["V"], c["d"]
    f64 = dict(dtype=torch.float64, device="cuda")
    x, t = s["x"].double(), s["targets"].long()
    rows = torch.nonzero(t >= 0)[:, 0]
    step = 16384
    if forward:
        total, top = torch.zeros(n, **f64), torch.full((n,), -math.inf, **f64)
        at = torch.zeros(n, **f64)
        for v in range(0, V, step):
            logits = x @ s["W"][v:v + step].double().T
            new = torch.maximum(top, logits.max(1).values)
            total = total * torch.exp(top - new) + torch.exp(logits - new[:, None]).sum(1)
            top = new
            here = torch.nonzero((t >= v) & (t < v + step))[:, 0]
            at[here] = logits[here, t[here] - v]
        lse = top + torch.log(total)
        loss = lse - at + c["z_loss"] * lse ** 2
        zero = torch.zeros(n, **f64)
        return torch.where(t >= 0, loss, zero), torch.where(t >= 0, lse, zero)
    lse, dloss = s["lse"].double()[rows, None], s["dloss"].double()[rows, None]
    dx, dW = torch.zeros(n, d, **f64), torch.zeros(V, d, **f64)
    xr, tr = x[rows], t[rows]
    for v in range(0, V, step):
        W = s["W"][v:v + step].double()
        p = torch.exp(xr @ W.T - lse)
        dl = p + 2 * c["z_loss"] * lse * p
        here = torch.nonzero((tr >= v) & (tr < v + step))[:, 0]
        dl[here, tr[here] - v] -= 1.0
        dl *= dloss
        dx[rows] += dl @ W
        dW[v:v + step] = dl.T @ xr
    return dx, dW


def exact(case, seed):
    # about 1 TFLOP/s in 64 bits on this card
    if work(case)["flops"] > 12e12:
        return None
    s = prepare(case, seed)
    op = case["op"]
    if op == "dropout":
        return s["x"].double() * _exact_keep(s["rng"], case["n"], case["d"], case["p"])
    if op.startswith("join"):
        return _exact_join(s, op == "join_forward")
    return _exact_loss(s, op == "loss_forward")
