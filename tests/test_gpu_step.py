"""GPU: dropout, the block joint and the cross entropy against the float64 oracle
(oracle/step_oracle.py).

Tolerances are element by element and come from the arithmetic.  With u the half
step of the output type (bf16 2^-8, fp32 2^-24) and v = 2^-24: a value rounded
once is off by u |value|; an fp32 operation by v; a sum of m fp32 terms by at most
m v sum |term| in any order (2 m v for products on the tensor cores, whose adders
may truncate); an operand's error goes through a product with the absolute values
of the other one; e^a with the hardware's exponential by 2^-20 + 2^-22 |a|
relative (its argument is rounded in fp32).  Each bound below is that, written out.
"""
import itertools

import numpy as np
import pytest
import torch

from oracle import step_oracle as S

pytestmark = pytest.mark.gpu

V = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TINY = 1e-37


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_layer_moe_gb300 import build
    build.build()
    from mixture_experts_layer_moe_gb300 import moe
    assert torch.cuda.is_available()
    return moe


def _u(dtype):
    return torch.finfo(DT[dtype]).eps / 2


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype="f32", std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(DT[dtype])


def _within(got, want, bound, what):
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - bound - TINY
    assert over.max().item() <= 0, (what, over.max().item(),
                                    ((got - want).abs() / (bound + TINY)).max().item())


def _rows(t, pad, fill=float("nan")):
    """t's rows inside a buffer whose rows are pad elements longer, the rest filled."""
    if pad == 0:
        return t.contiguous()
    buf = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


def _out(rows, d, pad, dtype):
    return _rows(torch.full((rows, d), float("nan"), dtype=DT[dtype], device="cuda"), pad, 7.0)


def _gaps_stay(t, pad):
    rows, d = t.shape
    return pad == 0 or bool((t.as_strided((rows, pad), (d + pad, 1), d) == 7.0).all())


def _rng(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


# -------------------------------------------------------------------- dropout
# rows, d, pad, dtype: single elements, widths round the vectors, rows apart, wide rows
ROWS = [(r, d, pad, dt)
        for dt in ("bf16", "f32")
        for r, d, pad in ((1, 1, 0), (3, 2, 0), (1, 2880, 0), (9, 8, 0), (33, 127, 0), (17, 128, 3),
                          (700, 256, 8), (5, 511, 1), (40, 520, 0), (257, 1001, 3), (6, 1024, 0),
                          (900, 2880, 0), (3, 4104, 8), (77, 7168, 0), (4, 8192, 0), (3, 8200, 0),
                          (2, 16392, 0), (3, 9001, 2))]


@pytest.mark.parametrize("rows,d,pad,dtype", ROWS)
def test_dropout(lib, rows, d, pad, dtype):
    g = _gen(rows * 3 + d)
    x, y = _rows(_randn(g, rows, d, dtype=dtype), pad), _out(rows, d, pad, dtype)
    rng = _rng(2 ** 62 + 12345 * rows, -7 - d)
    lib.moe_dropout(x, y, 0.3, rng)
    want = S.dropout(x, rng, 0.3)
    # the factor is rounded to fp32, then the product, then the result
    _within(y, want, (2 * V + _u(dtype)) * want.abs(), "y")
    assert torch.equal(y.cpu() == 0, want == 0) and _gaps_stay(y, pad)
    # in place, and no dropout
    z = _rows(x.contiguous(), pad, 7.0)
    lib.moe_dropout(z, z, 0.3, rng)
    assert torch.equal(z, y) and _gaps_stay(z, pad)
    lib.moe_dropout(x, y, 0.0)
    assert torch.equal(y, x)


def test_dropout_hides_what_it_drops(lib):
    """A NaN or infinity in a dropped place becomes 0; a kept one stays."""
    keep = S.keep(5, 6, 9, 300, 0.5)
    for bad in (float("nan"), float("inf")):
        x = torch.full((9, 300), bad, device="cuda")
        y = torch.empty_like(x)
        lib.moe_dropout(x, y, 0.5, _rng(5, 6))
        assert (y.cpu()[~keep] == 0).all() and not torch.isfinite(y.cpu()[keep]).any()


def test_dropout_in_a_graph_follows_the_state(lib):
    x, y = torch.ones(64, 512, device="cuda"), torch.empty(64, 512, device="cuda")
    rng = _rng(1, 0)
    lib.moe_dropout(x, y, 0.5, rng)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.moe_dropout(x, y, 0.5, rng)
        rng[1] += 1
    rng[1] = 0
    for offset in range(3):
        graph.replay()
        assert torch.equal(y.cpu() != 0, S.keep(1, offset, 64, 512, 0.5))


# ----------------------------------------------------------------- block joint
def _adds(d):
    """Terms that one fp32 sum over a row adds up in sequence, at most."""
    return 64 + d / 256


def _join_case(rows, d, pad, dtype, post, pre, gate, p, scale, beta=True, seed=0):
    g = _gen(seed + rows * 7 + d)
    params = {}
    if gate:
        params["gate"] = _randn(g, d, dtype=dtype, std=0.5, mean=0.5)
    for side, kind in (("post", post), ("pre", pre)):
        if kind != "none":
            params[side + "_gamma"] = _randn(g, d, dtype=dtype, std=0.2, mean=1.0)
        if kind == "layer" and beta:
            params[side + "_beta"] = _randn(g, d, dtype=dtype)
    x = _rows(_randn(g, rows, d, dtype=dtype, std=2.0, mean=0.3), pad)
    b = _rows(_randn(g, rows, d, dtype=dtype, std=0.7, mean=0.1), pad)
    dr, dy = (_rows(_randn(g, rows, d, dtype=dtype), pad) for _ in range(2))
    kw = dict(post=post, pre=pre, scale=scale, p=p, rng=_rng(seed + 99, rows + d) if p else None)
    return params, x, b, dr, (dy if pre != "none" else None), kw


def _vec(params, key, d, other):
    t = params.get(key)
    return torch.full((d,), float(other), dtype=torch.float64) if t is None else t.cpu().double()


def _norm_bound(v, ev, mean, rstd, out, gamma, beta, kind, d):
    """Error bounds of a norm's output, mean and rstd whose rows v are off by ev."""
    if kind == "none":
        return ev, torch.zeros_like(rstd), torch.zeros_like(rstd)
    n, c = _adds(d), (v - mean[:, None]).abs()
    dm = n * V * v.abs().mean(1) + ev.mean(1) if kind == "layer" else torch.zeros_like(rstd)
    er = ((n + 8) * V + (dm * rstd) ** 2 + (c * ev).mean(1) * rstd ** 2 + (ev ** 2).mean(1) * rstd ** 2)
    eo = (gamma.abs() * rstd[:, None] * (ev + dm[:, None] + c * (4 * V + er[:, None]))
          + 2 * V * (out.abs() + beta.abs()))
    return eo, dm + V * mean.abs(), rstd * er


def _check_join(lib, case, pad, dtype):
    params, x, b, _, _, kw = case
    rows, d = x.shape
    r, stats = _out(rows, d, pad, dtype), torch.full((4, rows), float("nan"), device="cuda")
    y = _out(rows, d, pad, dtype) if kw["pre"] != "none" else None
    lib.moe_block_join(x, b, lib.make_join_params(params), r, y, stats, **kw)
    wr, wy, ws, wz = S.join(x, b, params, **kw)
    vec = lambda key, other: _vec(params, key, d, other)
    zero = torch.zeros(rows, d, dtype=torch.float64)
    b64 = b.cpu().double()
    ez, em1, er1 = _norm_bound(b64, zero, ws[0], ws[1], wz, vec("post_gamma", 1),
                               vec("post_beta", 0), kw["post"], d)
    f = S.factors(kw["rng"], rows, d, kw["p"])
    gz = f * wz * vec("gate", 1)
    er = (vec("gate", 1).abs() * f * (ez + 2 * V * wz.abs()) + 2 * V * gz.abs()
          + V * (kw["scale"] * x.cpu().double()).abs() + V * wr.abs())
    _within(r, wr, er + _u(dtype) * (wr.abs() + er), "r")
    bounds = [em1, er1 + TINY]
    if y is not None:
        ey, em2, er2 = _norm_bound(wr, er, ws[2], ws[3], wy, vec("pre_gamma", 1), vec("pre_beta", 0),
                                   kw["pre"], d)
        _within(y, wy, ey + _u(dtype) * (wy.abs() + ey), "y")
    else:
        em2 = er2 = torch.zeros(rows, dtype=torch.float64)
    _within(stats, ws, torch.stack((bounds[0], bounds[1], em2, er2)) + V * ws.abs(), "stats")
    assert _gaps_stay(r, pad) and (y is None or _gaps_stay(y, pad))
    # without statistics, and in place: the same bits
    r2 = _rows(x.contiguous(), pad, 7.0)
    y2 = _out(rows, d, pad, dtype) if y is not None else None
    lib.moe_block_join(r2, b, lib.make_join_params(params), r2, y2, None, **kw)
    assert torch.equal(r2, r) and (y is None or torch.equal(y2, y)) and _gaps_stay(r2, pad)
    return r, stats


def _back_bound(w, ew, h, eh, rstd, kind, d):
    """The norm's gradient from w and the normed rows h: its value's error bound."""
    if kind == "none":
        return ew
    n = _adds(d)
    mean = lambda t: t.mean(1, keepdim=True)
    m1, m2 = mean(w) if kind == "layer" else 0 * mean(w), mean(w * h)
    e1 = mean(ew) + (n + 2) * V * mean(w.abs()) if kind == "layer" else 0 * mean(w)
    e2 = mean(ew * h.abs() + w.abs() * eh) + (n + 8) * V * mean((w * h).abs())
    return rstd[:, None] * (ew + e1 + h.abs() * e2 + m2.abs() * eh
                            + 4 * V * (w.abs() + m1.abs() + (h * m2).abs()))


def _check_join_backward(lib, case, r, stats, pad, dtype):
    params, _, b, dr, dy, kw = case
    rows, d = b.shape
    kept = [k for k in ("gate", "post_gamma", "post_beta", "pre_gamma", "pre_beta")
            if (k in params or (k.endswith("beta") and kw[k.split("_")[0]] == "layer"))]
    grads = {k: torch.full((d,), 9.0, device="cuda") for k in kept}
    dx, db = _out(rows, d, pad, dtype), _out(rows, d, pad, dtype)
    ws = torch.empty(lib.moe_block_join_workspace_size(rows, d, dtype), dtype=torch.uint8,
                     device="cuda")
    w = lib.make_join_params(params)
    back = lambda dr, dy, dx, db, grads: lib.moe_block_join_backward(
        b, r, stats, w, dr, dy, dx, db, lib.make_join_grads(grads), ws, **kw)
    back(dr, dy, dx, db, grads)
    wdx, wdb, wg = S.join_backward(b, r, stats, params, dr, dy, **kw)
    vec = lambda key, other: _vec(params, key, d, other)
    st = stats.cpu().double()
    R = dr.cpu().double()
    eR = torch.zeros_like(R)
    eg = {}
    if dy is not None:
        dy64 = dy.cpu().double()
        rh = (r.cpu().double() - st[2][:, None]) * st[3][:, None]
        wy = dy64 * vec("pre_gamma", 1)
        G = S._back(wy, rh, st[3], kw["pre"])
        eR = _back_bound(wy, V * wy.abs(), rh, 3 * V * rh.abs(), st[3], kw["pre"], d)
        eR = eR + 2 * V * (R.abs() + G.abs())
        R = R + G
        eg["pre_gamma"] = (rows + 16) * V * (dy64 * rh).abs().sum(0) + 3 * V * (dy64 * rh).abs().sum(0)
        eg["pre_beta"] = (rows + 16) * V * dy64.abs().sum(0)
    _within(dx, wdx, abs(kw["scale"]) * eR + V * wdx.abs() + _u(dtype) * (wdx.abs() + eR), "dx")
    f = S.factors(kw["rng"], rows, d, kw["p"])
    b64 = b.cpu().double()
    bh = b64 if kw["post"] == "none" else (b64 - st[0][:, None]) * st[1][:, None]
    ebh = 0 * bh if kw["post"] == "none" else 3 * V * bh.abs()
    u, eu = f * R, f * (eR + 2 * V * R.abs())
    a = (vec("gate", 1) * vec("post_gamma", 1)).abs()
    wz = u * vec("gate", 1) * vec("post_gamma", 1)
    ew = a * eu + 3 * V * wz.abs()
    eb = _back_bound(wz, ew, bh, ebh, st[1], kw["post"], d)
    _within(db, wdb, eb + _u(dtype) * (wdb.abs() + eb), "db")
    A, B = (u * bh).sum(0), u.sum(0)
    eA = (eu * bh.abs() + u.abs() * ebh).sum(0) + (rows + 16) * V * (u * bh).abs().sum(0)
    eB = eu.sum(0) + (rows + 16) * V * u.abs().sum(0)
    gamma, beta, gate = vec("post_gamma", 1).abs(), vec("post_beta", 0).abs(), vec("gate", 1).abs()
    eg["gate"] = gamma * eA + beta * eB + 3 * V * (gamma * A.abs() + beta * B.abs())
    eg["post_gamma"] = gate * (eA + 2 * V * A.abs())
    eg["post_beta"] = gate * (eB + 2 * V * B.abs())
    for k in kept:
        _within(grads[k], wg[k], eg[k], k)
    assert _gaps_stay(dx, pad) and _gaps_stay(db, pad)
    # each output alone: the same bits
    for k in kept:
        one = {k: torch.full((d,), 5.0, device="cuda")}
        back(dr, dy, None, None, one)
        assert torch.equal(one[k], grads[k]), k
    dx2, db2 = _out(rows, d, pad, dtype), _out(rows, d, pad, dtype)
    back(dr, dy, dx2, None, {})
    back(dr, dy, None, db2, {})
    assert torch.equal(dx2, dx) and torch.equal(db2, db)


KINDS = list(itertools.product(("none", "rms", "layer"), repeat=2))


@pytest.mark.parametrize("i,rows,d,pad,dtype", [(i, *c) for i, c in enumerate(ROWS)])
def test_join(lib, i, rows, d, pad, dtype):
    post, pre = KINDS[i % 9]
    if d < 3:      # (a norm's gradient over one or two elements is all cancellation)
        post = pre = "none"
    case = _join_case(rows, d, pad, dtype, post, pre, gate=i % 2 == 0, p=(0.0, 0.25, 0.5)[i % 3],
                      scale=(1.0, 0.75)[i % 2])
    r, stats = _check_join(lib, case, pad, dtype)
    _check_join_backward(lib, case, r, stats, pad, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,pad", [(96, 0), (96, 3), (1160, 0), (8448, 0)])
@pytest.mark.parametrize("post,pre", KINDS)
def test_join_kinds(lib, post, pre, d, pad, dtype):
    for gate, p, beta in ((True, 0.1, True), (False, 0.0, False)):
        case = _join_case(41, d, pad, dtype, post, pre, gate, p, 0.5, beta, seed=3)
        r, stats = _check_join(lib, case, pad, dtype)
        _check_join_backward(lib, case, r, stats, pad, dtype)


@pytest.mark.parametrize("d", [64, 100, 9000])
def test_join_backward_of_one_gradient(lib, d):
    """dr alone, dy alone, neither: the missing one counts as zero."""
    params, x, b, dr, dy, kw = _join_case(11, d, 0, "f32", "layer", "rms", True, 0.2, 1.0)
    r, stats = torch.empty_like(x), torch.empty(4, 11, device="cuda")
    w = lib.make_join_params(params)
    lib.moe_block_join(x, b, w, r, torch.empty_like(x), stats, **kw)
    ws = torch.empty(lib.moe_block_join_workspace_size(11, d, "f32"), dtype=torch.uint8,
                     device="cuda")

    def back(dr, dy):
        out = [torch.full_like(x, float("nan")) for _ in range(2)]
        grads = {k: torch.full((d,), float("nan"), device="cuda") for k in params}
        lib.moe_block_join_backward(b, r, stats, w, dr, dy, *out, lib.make_join_grads(grads), ws, **kw)
        return out + list(grads.values())

    zero = torch.zeros_like(x)
    for given, full in (((dr, None), (dr, zero)), ((None, dy), (zero, dy)), ((None, None), (zero, zero))):
        for got, want in zip(back(*given), back(*full)):
            assert torch.equal(got, want)


@pytest.mark.parametrize("d", [64, 67, 9000])
def test_join_keeps_a_nan_in_its_row(lib, d):
    params, x, b, dr, dy, kw = _join_case(6, d, 0, "bf16", "rms", "rms", False, 0.0, 1.0)
    x[2, 5] = float("nan")
    dr[4, 7] = float("inf")
    r, y, stats = torch.empty_like(x), torch.empty_like(x), torch.empty(4, 6, device="cuda")
    w = lib.make_join_params(params)
    lib.moe_block_join(x, b, w, r, y, stats, **kw)
    others = [0, 1, 3, 4, 5]
    assert torch.isnan(y[2]).all() and torch.isfinite(y[others]).all()
    assert torch.isfinite(r[2, torch.arange(d) != 5]).all()
    dx, db = torch.empty_like(x), torch.empty_like(x)
    ws = torch.empty(lib.moe_block_join_workspace_size(6, d, "bf16"), dtype=torch.uint8, device="cuda")
    lib.moe_block_join_backward(b, r, stats, w, dr, dy, dx, db, lib.make_join_grads({}), ws, **kw)
    clean = [0, 1, 3, 5]
    assert torch.isfinite(dx[clean]).all() and torch.isfinite(db[clean]).all()


def test_join_without_rows(lib):
    e, v = torch.empty(0, 16, device="cuda"), torch.ones(16, device="cuda")
    params = lib.make_join_params(dict(gate=v, post_gamma=v, pre_gamma=v))
    st, ws = torch.empty(4, 0, device="cuda"), torch.empty(0, dtype=torch.uint8, device="cuda")
    lib.moe_block_join(e, e, params, e, e, st)
    grads = {k: torch.full((16,), 3.0, device="cuda") for k in ("gate", "post_gamma", "pre_gamma")}
    lib.moe_block_join_backward(e, e, st, params, e, e, e, e, lib.make_join_grads(grads), ws)
    assert all(t.abs().max() == 0 for t in grads.values())
    lib.moe_dropout(e, e, 0.5, _rng(1, 1))


# --------------------------------------------------------------- cross entropy
# n, d, vocab, dtype, share left out: single tokens and entries, sizes round the tiles, odd
# vocabularies, long reductions, several pieces of the vocabulary
LOSS_CASES = [
    (1, 8, 1, "bf16", 0.0), (1, 8, 2, "bf16", 0.0), (3, 16, 5, "bf16", 0.0), (2, 64, 257, "bf16", 0.0),
    (33, 72, 300, "bf16", 0.3), (5, 264, 4099, "bf16", 0.0), (128, 256, 1000, "bf16", 0.1),
    (129, 512, 513, "bf16", 0.5), (255, 1024, 2051, "bf16", 0.0), (256, 64, 256, "bf16", 0.0),
    (257, 128, 8200, "bf16", 0.2), (600, 320, 3001, "bf16", 0.1), (1, 2880, 20011, "bf16", 0.0),
    (40, 4096, 769, "bf16", 0.5), (1100, 512, 511, "bf16", 0.05), (2500, 64, 777, "bf16", 0.1),
    (1, 4, 1, "f32", 0.0), (1, 4, 3, "f32", 0.0), (3, 12, 5, "f32", 0.0), (2, 64, 257, "f32", 0.5),
    (33, 36, 300, "f32", 0.3), (256, 128, 4099, "f32", 0.1), (70, 260, 515, "f32", 0.0),
    (1000, 64, 1027, "f32", 0.2), (2500, 16, 130, "f32", 0.1), (17000, 8, 40, "f32", 0.5),
    # few fp32 tokens, up to and past what is held of them
    (1, 64, 1, "f32", 0.0), (1, 512, 8192, "f32", 0.0), (1, 2884, 20011, "f32", 0.0),
    (2, 132, 65, "f32", 0.0), (3, 100, 999, "f32", 0.3), (4, 68, 33, "f32", 0.0),
    (5, 260, 5155, "f32", 0.4), (6, 64, 30, "f32", 0.0), (7, 1028, 70, "f32", 0.3),
    (8, 64, 9001, "f32", 0.2), (8, 6144, 333, "f32", 0.0), (8, 6148, 333, "f32", 0.0),
    (9, 256, 700, "f32", 0.0),
]


def _loss_case(n, d, vocab, dtype, out, seed=0):
    g = _gen(seed + n + d + vocab)
    W = _randn(g, vocab, d, dtype=dtype, std=1.5 * d ** -0.5)
    t = torch.randint(vocab, (n,), generator=g, device="cuda")
    boost = 4 * torch.rand(n, 1, generator=g, device="cuda")
    x = (_randn(g, n, d) + boost * W[t].float()).to(DT[dtype])
    left = torch.rand(n, generator=g, device="cuda") < out
    t = torch.where(left, -1 - t, t).to(torch.int32)
    x[left] = float("nan")          # (what a left out row holds is not read)
    return x, W, t, left


def _ok(lib, ws):
    st, detail = lib.moe_status_check(ws)
    assert st == 0, (lib.status_string(st), detail)


def _logit_error(x, W, dtype):
    """Bound of the logits' errors (rows that count)."""
    k = 2 if dtype == "bf16" else 1
    return k * x.shape[1] * V * (x.cpu().double().abs() @ W.cpu().double().abs().T)


@pytest.mark.parametrize("z_loss", [0.0, 1e-3])
@pytest.mark.parametrize("n,d,vocab,dtype,out", LOSS_CASES)
def test_cross_entropy(lib, n, d, vocab, dtype, out, z_loss):
    x, W, t, left = _loss_case(n, d, vocab, dtype, out)
    ws = lib.alloc_cross_entropy_workspace(n, d, vocab, dtype)
    ws[256:] = 0xFF                 # (a NaN wherever the call reads what it did not write)
    loss, lse = (torch.full((n,), float("nan"), device="cuda") for _ in range(2))
    lib.moe_cross_entropy(x, W, t, loss, lse, ws, z_loss)
    _ok(lib, ws)
    clean = torch.where(left[:, None], 0, x)
    wloss, wlse, logits = S.cross_entropy(clean, W, t, z_loss)
    el = _logit_error(clean, W, dtype)
    p = torch.softmax(logits, 1)
    top = logits.amax(1, keepdim=True)
    e = ((p * (el + 2 ** -20 + 2 ** -22 * (top - logits))).sum(1) + (64 + vocab / 8192) * V
         + 2 * V * (wlse.abs() + top[:, 0].abs()))
    at = t.cpu().long().clamp(min=0)[:, None]
    counted = (t >= 0).cpu()
    _within(lse, wlse, torch.where(counted, e, 0.0), "lse")
    eloss = (e + el.gather(1, at)[:, 0] + 2 * V * (wlse.abs() + logits.gather(1, at)[:, 0].abs())
             + z_loss * (2 * wlse.abs() * e + e * e + 4 * V * wlse ** 2))
    _within(loss, wloss, torch.where(counted, eloss, 0.0), "loss")
    again = torch.empty_like(loss), torch.empty_like(lse)
    lib.moe_cross_entropy(x, W, t, *again, ws, z_loss)
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)


@pytest.mark.parametrize("z_loss", [0.0, 1e-3])
@pytest.mark.parametrize("n,d,vocab,dtype,out", LOSS_CASES)
def test_cross_entropy_backward(lib, n, d, vocab, dtype, out, z_loss):
    x, W, t, left = _loss_case(n, d, vocab, dtype, out, 5)
    clean = torch.where(left[:, None], 0, x)
    lse = S.cross_entropy(clean, W, t, z_loss)[1].float().cuda()
    dloss = _randn(_gen(n), n, std=1.0)
    dloss[left] = float("nan")
    ws = lib.alloc_cross_entropy_workspace(n, d, vocab, dtype)
    ws[256:] = 0xFF
    dx, dW = torch.full_like(x, float("nan")), torch.full_like(W, float("nan"))
    lib.moe_cross_entropy_backward(x, W, t, lse, dloss, dx, dW, ws, z_loss)
    _ok(lib, ws)
    wdx, wdW, wdl = S.cross_entropy_backward(clean, W, t, lse, torch.where(left, 0, dloss), z_loss)
    aW, ax = W.cpu().double().abs(), clean.cpu().double().abs()
    counted = (t >= 0).cpu()[:, None]
    ls = lse.cpu().double()[:, None]
    logits = clean.cpu().double() @ W.cpu().double().T
    f = (1 + 2 * z_loss * ls).abs()
    p = torch.exp(logits - ls) * f
    hot = torch.zeros_like(p).scatter_(1, t.cpu().long().clamp(min=0)[:, None], 1.0)
    el = _logit_error(clean, W, dtype)
    edl = (torch.where(left, 0, dloss).abs().cpu().double()[:, None]
           * (p * (el + el * el + 2 ** -20 + 2 ** -22 * (logits - ls).abs() + 4 * V) + 3 * V * (p + hot)))
    edl = torch.where(counted, edl, 0.0)
    edl = edl + _u(dtype) * (wdl.abs() + edl)
    k = 2 if dtype == "bf16" else 1
    adl = wdl.abs() + edl
    ex = (edl + k * (vocab + 16) * V * adl) @ aW
    _within(dx, wdx, ex + _u(dtype) * (wdx.abs() + ex), "dx")
    assert (dx[left] == 0).all()
    eW = (edl + k * (n + 16) * V * adl).T @ ax
    _within(dW, wdW, eW + _u(dtype) * (wdW.abs() + eW), "dW")
    # either alone: the same bits
    one = torch.empty_like(dx), torch.empty_like(dW)
    lib.moe_cross_entropy_backward(x, W, t, lse, dloss, one[0], None, ws, z_loss)
    lib.moe_cross_entropy_backward(x, W, t, lse, dloss, None, one[1], ws, z_loss)
    assert torch.equal(one[0], dx) and torch.equal(one[1], dW)


@pytest.mark.parametrize("n,d,vocab,dtype", [(40, 64, 500, "bf16"), (300, 512, 3000, "bf16"),
                                             (40, 64, 500, "f32"), (4, 64, 500, "f32")])
def test_cross_entropy_of_no_counted_token(lib, n, d, vocab, dtype):
    x, W, t, _ = _loss_case(n, d, vocab, dtype, 1.1)
    ws = lib.alloc_cross_entropy_workspace(n, d, vocab, dtype)
    ws[256:] = 0xFF
    loss, lse = (torch.full((n,), float("nan"), device="cuda") for _ in range(2))
    lib.moe_cross_entropy(x, W, t, loss, lse, ws)
    assert (loss == 0).all() and (lse == 0).all()
    dx, dW = torch.full_like(x, float("nan")), torch.full_like(W, float("nan"))
    lib.moe_cross_entropy_backward(x, W, t, lse, loss, dx, dW, ws)
    _ok(lib, ws)
    assert (dx == 0).all() and (dW == 0).all()


@pytest.mark.parametrize("n,d,vocab,dtype", [(40, 64, 500, "bf16"), (300, 512, 3000, "bf16"),
                                             (40, 64, 500, "f32")])
def test_cross_entropy_reports_a_target_outside(lib, n, d, vocab, dtype):
    x, W, t, _ = _loss_case(n, d, vocab, dtype, 0.0)
    t[7] = vocab
    ws = lib.alloc_cross_entropy_workspace(n, d, vocab, dtype)
    loss, lse = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    lib.moe_cross_entropy(x, W, t, loss, lse, ws)
    assert lib.moe_status_check(ws) == (5, 7)
    # the status stays until it is cleared; then the workspace serves again
    lib.moe_cross_entropy_backward(x, W, t, lse, loss, torch.empty_like(x), None, ws)
    assert lib.moe_status_check(ws)[0] == 5
    lib.moe_status_clear(ws)
    t[7] = vocab - 1
    lib.moe_cross_entropy(x, W, t, loss, lse, ws)
    _ok(lib, ws)
    wloss = S.cross_entropy(x, W, t)[0]
    assert (loss.cpu().double() - wloss).abs().max() < 1e-3


def test_cross_entropy_of_far_logits(lib):
    """Logits of thousands: the maximum is subtracted first, lse and loss stay exact to fp32."""
    x = torch.zeros(3, 64, device="cuda")
    x[:, 0] = torch.tensor([1.0, -1.0, 100.0])
    W = torch.zeros(300, 64, device="cuda")
    W[:, 0] = torch.arange(300, device="cuda") * 10.0
    t = torch.tensor([299, 0, 5], dtype=torch.int32, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        xt, Wt = x.to(dtype), W.to(dtype)
        ws = lib.alloc_cross_entropy_workspace(3, 64, 300, "f32")
        loss, lse = torch.zeros(3, device="cuda"), torch.zeros(3, device="cuda")
        lib.moe_cross_entropy(xt, Wt, t, loss, lse, ws)
        wloss, wlse, _ = S.cross_entropy(xt, Wt, t)
        _within(lse, wlse, 4 * V * wlse.abs() + 2 ** -19, "lse")
        _within(loss, wloss, 8 * V * wlse.abs() + 2 ** -19, "loss")


def test_cross_entropy_without_tokens(lib):
    e = torch.empty(0, 64, device="cuda")
    W, dW = torch.ones(10, 64, device="cuda"), torch.full((10, 64), 3.0, device="cuda")
    t, v = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, device="cuda")
    ws = lib.alloc_cross_entropy_workspace(0, 64, 10, "f32")
    lib.moe_cross_entropy(e, W, t, v, v, ws)
    lib.moe_cross_entropy_backward(e, W, t, v, v, e, dW, ws)
    assert (dW == 0).all()


# --------------------------------------------------------- together, as used
def _step(lib, s, ws):
    """The last block's joint, the loss, and back to the block's output."""
    n, d = s["x"].shape
    kw = dict(post="rms", pre="rms", p=0.1, rng=s["rng"])
    lib.moe_block_join(s["x"], s["b"], s["w"], s["r"], s["y"], s["stats"], **kw)
    lib.moe_cross_entropy(s["y"], s["W"], s["t"], s["loss"], s["lse"], ws)
    lib.moe_cross_entropy_backward(s["y"], s["W"], s["t"], s["lse"], s["dloss"], s["dy"], s["dW"], ws)
    lib.moe_block_join_backward(s["b"], s["r"], s["stats"], s["w"], None, s["dy"], s["dx"], s["db"],
                                lib.make_join_grads(s["grads"]), s["scratch"], **kw)


@pytest.mark.parametrize("n,d,vocab", [(37, 64, 300), (300, 512, 4001)])
def test_a_step_captured_and_replayed(lib, n, d, vocab):
    """A run of the operators in a graph, replayed on other inputs and on another stream, gives the
    bits of the eager calls, and follows the generator's state."""
    g = _gen(8)
    vectors = {k: _randn(g, d, dtype="bf16", std=0.2, mean=1.0) for k in
               ("gate", "post_gamma", "pre_gamma")}
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    s = dict(x=bf(n, d), b=bf(n, d), r=bf(n, d), y=bf(n, d), dy=bf(n, d), dx=bf(n, d), db=bf(n, d),
             W=_randn(g, vocab, d, dtype="bf16", std=d ** -0.5), dW=bf(vocab, d),
             t=torch.zeros(n, dtype=torch.int32, device="cuda"), rng=_rng(3, 0),
             stats=torch.zeros(4, n, device="cuda"), loss=torch.zeros(n, device="cuda"),
             lse=torch.zeros(n, device="cuda"), dloss=torch.full((n,), 1.0 / n, device="cuda"),
             w=lib.make_join_params(vectors),
             grads={k: torch.zeros(d, device="cuda") for k in vectors},
             scratch=torch.zeros(lib.moe_block_join_workspace_size(n, d, "bf16"), dtype=torch.uint8,
                                 device="cuda"))
    ws = lib.alloc_cross_entropy_workspace(n, d, vocab, "bf16")
    _step(lib, s, ws)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        _step(lib, s, ws)
    names = ("r", "y", "stats", "loss", "lse", "dy", "dW", "dx", "db")
    for turn in range(3):
        s["x"].copy_(_randn(g, n, d, dtype="bf16"))
        s["b"].copy_(_randn(g, n, d, dtype="bf16"))
        s["t"].copy_(torch.randint(-vocab // 4, vocab, (n,), generator=g, device="cuda"))
        s["rng"][1] = turn
        _step(lib, s, ws)
        want = [s[k].clone() for k in names] + [v.clone() for v in s["grads"].values()]
        for k in names:
            s[k].fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        for name, a, b in zip((*names, *s["grads"]), want, [s[k] for k in names] + list(s["grads"].values())):
            assert torch.equal(a, b), name
    _ok(lib, ws)


def test_the_layer_between_joints(lib):
    """norm, the MoE layer, its joint, the loss and the whole way back: the gradient of the residual
    stream against differences of the loss (fp32)."""
    import moe_synth
    n, d, F, E, k, vocab = 24, 32, 48, 4, 2, 60
    cfg = moe_synth.MoEConfig("t", n, d, F, E, k, "f32", "f32", "renorm", "swiglu")
    g = _gen(17)
    f = lambda *s, std=1.0: _randn(g, *s, std=std)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    x, one = f(n, d), torch.ones(d, device="cuda")
    t = dict(Wg=f(E, d, std=0.3), W1=f(E, F, d, std=0.2), W3=f(E, F, d, std=0.2),
             W2=f(E, d, F, std=0.2))
    w, W = lib.make_weights(t), f(vocab, d, std=0.3)
    targets = torch.randint(vocab, (n,), generator=g, device="cuda").to(torch.int32)
    targets[3] = -1
    ws, rng = lib.alloc_train_workspace(cfg), _rng(4, 4)
    lws = lib.alloc_cross_entropy_workspace(n, d, vocab, "f32")
    join = lib.make_join_params(dict(gate=0.5 * one, post_gamma=one, pre_gamma=one))
    kw = dict(post="rms", pre="rms", p=0.2, rng=rng)
    dloss = (targets >= 0).float() / (n - 1)

    def forward(x):
        s = dict(y=torch.empty(n, d, device="cuda"), mean=torch.empty(n, device="cuda"),
                 rstd=torch.empty(n, device="cuda"), idx=i32(n, k), gate=torch.empty(n, k, device="cuda"),
                 probs=torch.empty(n, E, device="cuda"), counts=i32(E), off=i32(E + 1),
                 perm=i32(n * k), inv=i32(n * k), xp=torch.empty(n * k, d, device="cuda"),
                 g=torch.empty(n * k, F, device="cuda"), u=torch.empty(n * k, F, device="cuda"),
                 h=torch.empty(n * k, F, device="cuda"), yp=torch.empty(n * k, d, device="cuda"),
                 b=torch.empty(n, d, device="cuda"), r=torch.empty(n, d, device="cuda"),
                 out=torch.empty(n, d, device="cuda"), stats=torch.empty(4, n, device="cuda"),
                 loss=torch.empty(n, device="cuda"), lse=torch.empty(n, device="cuda"))
        lib.moe_layernorm(x, one, None, s["y"], s["mean"], s["rstd"])
        lib.moe_route(cfg, s["y"], w, s["idx"], s["gate"], s["probs"], ws)
        lib.moe_dispatch(cfg, s["idx"], s["y"], s["counts"], s["off"], s["perm"], s["inv"], s["xp"], ws)
        lib.moe_expert_ffn_train(cfg, s["xp"], s["off"], w, s["g"], s["u"], s["h"], s["yp"], ws)
        lib.moe_combine(cfg, s["yp"], s["inv"], s["gate"], None, s["b"], ws)
        lib.moe_block_join(x, s["b"], join, s["r"], s["out"], s["stats"], **kw)
        lib.moe_cross_entropy(s["out"], W, targets, s["loss"], s["lse"], lws)
        return s

    s = forward(x)
    e = lambda *shape: torch.empty(*shape, device="cuda")
    dout, dx, db, dyp, dgate, dxp, dy, dn = (e(n, d), e(n, d), e(n, d), e(n * k, d), e(n, k),
                                            e(n * k, d), e(n, d), e(n, d))
    scratch = torch.zeros(max(lib.moe_block_join_workspace_size(n, d, "f32"),
                              lib.moe_layernorm_workspace_size(n, d, "f32")), dtype=torch.uint8,
                          device="cuda")
    lib.moe_cross_entropy_backward(s["out"], W, targets, s["lse"], dloss, dout, None, lws)
    lib.moe_block_join_backward(s["b"], s["r"], s["stats"], join, None, dout, dx, db,
                                lib.make_join_grads({}), scratch, **kw)
    lib.moe_combine_backward(cfg, db, s["yp"], s["inv"], s["gate"], dyp, dgate, ws)
    lib.moe_expert_ffn_backward(cfg, s["xp"], s["off"], w, s["g"], s["u"], s["h"], dyp, dxp,
                                lib.make_expert_grads({}), ws)
    lib.moe_route_backward(cfg, s["y"], w, s["probs"], s["idx"], s["gate"], dgate, None, 0.0,
                           s["inv"], dxp, dy, None, None, ws)
    lib.moe_layernorm_backward(x, one, s["mean"], s["rstd"], dy, dn, None, None, scratch)
    _ok(lib, ws)
    _ok(lib, lws)
    grad = (dx + dn).double()
    h = 2e-3
    for seed in range(3):
        step = _randn(_gen(seed), n, d)
        ends = []
        for sign in (1, -1):
            moved = forward(x + sign * h * step)
            assert torch.equal(moved["idx"], s["idx"])     # (the choice of experts stays)
            ends.append((moved["loss"].double() * dloss.double()).sum().item())
        slope, want = (ends[0] - ends[1]) / (2 * h), (grad * step.double()).sum().item()
        # fp32 losses of about 4, off by some 2^-22, over 2 h; the third derivative times h^2 / 6
        assert abs(slope - want) <= 4 * 2 ** -20 / (2 * h) + 50 * h * h, (slope, want)


# ------------------------------------------- large problems, against 64 bits on the GPU
def _loss_reference(x, W, t, lse, dloss, z_loss, dtype, step=4096):
    """loss, lse, dx, dW in float64 and their error bounds as in the tests above, over pieces of the
    vocabulary."""
    n, d = x.shape
    V_, k, u = W.shape[0], 2 if dtype == "bf16" else 1, _u(dtype)
    x64, ax = x.double(), x.double().abs()
    t, counted = t.long(), (t >= 0)[:, None]
    ls, dl_scale = lse.double()[:, None], torch.where(counted, dloss.double()[:, None], 0.0)
    f64 = dict(dtype=torch.float64, device="cuda")
    dx, ex, dW, eW = (torch.zeros(s, **f64) for s in ((n, d), (n, d), (V_, d), (V_, d)))
    for v in range(0, V_, step):
        Wp = W[v:v + step].double()
        l = x64 @ Wp.T
        el = k * d * V * (ax @ Wp.abs().T)
        p = torch.exp(l - ls) * (1 + 2 * z_loss * ls).abs()
        hot = torch.zeros_like(p)
        here = torch.nonzero((t >= v) & (t < v + step))[:, 0]
        hot[here, t[here] - v] = 1.0
        dl = dl_scale * (p - hot)
        e = dl_scale.abs() * (p * (el + el * el + 2 ** -20 + 2 ** -22 * (l - ls).abs() + 4 * V)
                              + 5 * V * (p + hot))
        e = e + u * (dl.abs() + e)
        a = dl.abs() + e
        dx += dl @ Wp
        ex += (e + k * (V_ + 16) * V * a) @ Wp.abs()
        dW[v:v + step] = dl.T @ x64
        eW[v:v + step] = (e + k * (n + 16) * V * a).T @ ax
    return dx, ex + u * (dx.abs() + ex), dW, eW + u * (dW.abs() + eW)


def _close(got, want, bound, what):
    _within(got, want.cpu(), bound.cpu(), what)


# several pieces of the vocabulary: on the tensor cores, for few tokens, on the CUDA cores; runs of
# the tokens there
@pytest.mark.parametrize("n,d,vocab,dtype", [(2500, 64, 60001, "bf16"), (190, 8, 720001, "bf16"),
                                             (3001, 8, 30001, "f32"), (5000, 16, 27777, "bf16"),
                                             (20000, 64, 9001, "bf16"), (12000, 8, 9001, "f32"),
                                             (5001, 16, 203, "bf16"), (9001, 36, 77, "f32"),
                                             (2, 64, 4194561, "f32")])
def test_cross_entropy_in_pieces(lib, n, d, vocab, dtype):
    x, W, t, left = _loss_case(n, d, vocab, dtype, 0.1, 7)
    clean = torch.where(left[:, None], 0, x)
    lse64 = torch.zeros(n, dtype=torch.float64, device="cuda")
    top = torch.zeros_like(lse64)
    for a in range(0, n, 256):
        l = clean[a:a + 256].double() @ W.double().T
        lse64[a:a + 256], top[a:a + 256] = torch.logsumexp(l, 1), l.amax(1)
    ws = lib.alloc_cross_entropy_workspace(n, d, vocab, dtype)
    ws[256:] = 0xFF
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    lib.moe_cross_entropy(x, W, t, loss, lse, ws, 1e-3)
    counted = t >= 0
    # |l| <= sum |x| |W| <= |x| |W| (norms), the largest of the rows of W
    el = 2 * d * V * clean.double().norm(dim=1) * W.double().norm(dim=1).max()
    e = el + 2 ** -20 + 2 ** -22 * 20 + (64 + vocab / 8192) * V + 2 * V * (lse64.abs() + top.abs())
    _close(lse, torch.where(counted, lse64, 0.0), torch.where(counted, e, 0.0), "lse")
    dloss = _randn(_gen(3), n)
    dx, dW = torch.full_like(x, float("nan")), torch.full_like(W, float("nan"))
    lib.moe_cross_entropy_backward(x, W, t, lse, dloss, dx, dW, ws, 1e-3)
    _ok(lib, ws)
    wdx, ex, wdW, eW = _loss_reference(clean, W, t, lse, dloss, 1e-3, dtype)
    _close(dx, wdx, ex, "dx")
    _close(dW, wdW, eW, "dW")
    again = torch.empty_like(dx), torch.empty_like(dW)
    lib.moe_cross_entropy_backward(x, W, t, lse, dloss, again[0], None, ws, 1e-3)
    lib.moe_cross_entropy_backward(x, W, t, lse, dloss, None, again[1], ws, 1e-3)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dW)


# counted tokens round the boxes that few tokens are cut into, with rows of NaN between
@pytest.mark.parametrize("counted", [1, 15, 16, 17, 31, 32, 33, 64, 65, 96, 97, 127, 128, 129, 144, 160,
                                     161, 191, 192])
@pytest.mark.parametrize("d,vocab", [(328, 1300), (1032, 259)])
def test_cross_entropy_backward_of_few_tokens(lib, counted, d, vocab):
    x, W, t, _ = _loss_case(192, d, vocab, "bf16", 0.0, counted)
    out = torch.randperm(192, generator=torch.Generator().manual_seed(counted))[counted:].cuda()
    t[out], x[out] = -5, float("nan")
    clean = x.clone()
    clean[out] = 0
    lse = torch.where(t >= 0, torch.logsumexp(clean.double() @ W.double().T, 1), 0.0).float()
    dloss = _randn(_gen(counted), 192)
    ws = lib.alloc_cross_entropy_workspace(192, d, vocab, "bf16")
    ws[256:] = 0xFF
    dx, dW = torch.full_like(x, float("nan")), torch.full_like(W, float("nan"))
    lib.moe_cross_entropy_backward(x, W, t, lse, dloss, dx, dW, ws)
    _ok(lib, ws)
    wdx, ex, wdW, eW = _loss_reference(clean, W, t, lse, dloss, 0.0, "bf16")
    _close(dx, wdx, ex, "dx")
    _close(dW, wdW, eW, "dW")
    assert (dx[out] == 0).all()


@pytest.mark.parametrize("n,d,vocab,dtype", [(50, 320, 1100, "bf16"), (400, 320, 1100, "bf16"),
                                             (50, 64, 300, "f32")])
def test_cross_entropy_backward_of_uneven_weights(lib, n, d, vocab, dtype):
    """dloss of any size, zero and not finite: the result of a token goes by its own."""
    x, W, t, _ = _loss_case(n, d, vocab, dtype, 0.0, 1)
    lse = torch.logsumexp(x.double() @ W.double().T, 1).float()
    dloss = _randn(_gen(9), n) * 10.0 ** torch.linspace(-18, 3, n, device="cuda")
    dloss[5] = 0.0
    ws = lib.alloc_cross_entropy_workspace(n, d, vocab, dtype)
    dx, dW = torch.empty_like(x), torch.empty_like(W)
    lib.moe_cross_entropy_backward(x, W, t, lse, dloss, dx, dW, ws)
    wdx, ex, wdW, eW = _loss_reference(x, W, t, lse, dloss, 0.0, dtype)
    _close(dx, wdx, ex, "dx")
    _close(dW, wdW, eW, "dW")
    assert (dx[5] == 0).all()
    for bad in (float("nan"), float("inf")):
        spoilt = dloss.clone()
        spoilt[7] = bad
        dx2 = torch.empty_like(x)
        lib.moe_cross_entropy_backward(x, W, t, lse, spoilt, dx2, dW, ws)
        others = torch.arange(n, device="cuda") != 7
        assert torch.equal(dx2[others], dx[others]) and not torch.isfinite(dx2[7]).any()
    lib.moe_cross_entropy_backward(x, W, t, lse, torch.zeros_like(dloss), dx, dW, ws)
    assert (dx == 0).all() and (dW == 0).all()


def test_calls_on_two_streams(lib):
    """Two problems at once, each on a stream and in a workspace of its own; one workspace for
    problems of several shapes in turn."""
    cases = [_loss_case(300, 512, 5000, "bf16", 0.1, 1), _loss_case(120, 256, 9000, "bf16", 0.3, 2)]
    size = max(lib.moe_cross_entropy_workspace_size(c[0].shape[0], c[0].shape[1], c[1].shape[0], "bf16")
               for c in cases)

    def call(c, ws):
        x, W, t, _ = c
        n = x.shape[0]
        loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        dx, dW = torch.empty_like(x), torch.empty_like(W)
        lib.moe_cross_entropy(x, W, t, loss, lse, ws)
        lib.moe_cross_entropy_backward(x, W, t, lse, torch.ones_like(loss), dx, dW, ws)
        return loss, lse, dx, dW

    shared = torch.zeros(size, dtype=torch.uint8, device="cuda")
    want = [call(c, shared) for c in cases]
    spaces = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for c, ws, s in zip(cases, spaces, streams):
            with torch.cuda.stream(s):
                got.append(call(c, ws))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            for p, q in zip(a, b):
                assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [17, 40, 264, 1003, 5000])
def test_join_rows_anywhere(lib, d, dtype):
    """Rows at every distance from a vector's boundary, in tensors of different distances, give the
    bits of dense rows."""
    params, x, b, dr, dy, kw = _join_case(37, d, 0, dtype, "rms", "layer", True, 0.2, 0.5)
    w = lib.make_join_params(params)
    ws = torch.empty(lib.moe_block_join_workspace_size(37, d, dtype), dtype=torch.uint8, device="cuda")

    def run(pads):
        pad = iter(pads)
        place = lambda t: _rows(t, next(pad))
        out = lambda: _out(37, d, next(pad), dtype)
        r, y, stats = out(), out(), torch.empty(4, 37, device="cuda")
        lib.moe_block_join(place(x), place(b), w, r, y, stats, **kw)
        grads = {k: torch.empty(d, device="cuda") for k in params}
        dx, db = out(), out()
        lib.moe_block_join_backward(place(b), r, stats, w, place(dr), place(dy), dx, db,
                                    lib.make_join_grads(grads), ws, **kw)
        return [r, y, stats, dx, db, *grads.values()]

    want = run([1] * 9)
    for shift in range(1, 16, 3):
        got = run([(shift * (i + 1)) % 17 + 1 for i in range(9)])
        for a, c in zip(want, got):
            assert torch.equal(a, c)


# ------------------------------------------------------- offsets past 32 bits
def test_dropout_past_32_bits(lib):
    rows = 2 ** 31 + 77
    x = torch.ones(rows, 1, dtype=torch.bfloat16, device="cuda")
    rng = _rng(21, 22)
    lib.moe_dropout(x, x, 0.5, rng)
    words = S.philox4x32_10((np.zeros(100, np.uint64), np.arange(rows - 100, rows).astype(np.uint64),
                             22, 0), (21, 0))
    keep = torch.from_numpy((words[0] & np.uint64(0xFFFF)) >= S.threshold(0.5))
    assert torch.equal(x[-100:, 0].cpu().float(), torch.where(keep, 2.0, 0.0))


def test_join_past_32_bits(lib):
    """The last of rows that hold more than 2^32 elements (without dropout a row's result is its
    own), and column sums over all of them."""
    rows, d = 1_100_001, 4096
    g = _gen(2)
    v = _randn(g, d, dtype="bf16", std=0.2, mean=1.0)
    w = lib.make_join_params(dict(post_gamma=v, pre_gamma=v))
    kw = dict(post="rms", pre="rms")
    tail = [_randn(g, 8, d, dtype="bf16") for _ in range(4)]
    big = [torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for t, s in zip(big, tail):
        t[-8:] = s
    r, y = torch.empty_like(big[0]), torch.empty_like(big[0])
    stats = torch.empty(4, rows, device="cuda")
    lib.moe_block_join(*big, w, r, y, stats, **kw)
    few = [torch.empty(8, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    few_stats = torch.empty(4, 8, device="cuda")
    lib.moe_block_join(*tail[:2], w, *few, few_stats, **kw)
    # few rows are summed by more threads, in another order: each order is off by at most
    # (adds + 8) v relative for sums of squares, so the two by e; then r = x + z with |z| <= |r| + |x|,
    # y = r gamma rstd, and each is rounded once on either side
    e = 2 * (_adds(d) + 8) * V
    near = lambda got, want, bound: ((got.double() - want.double()).abs() <= bound + TINY).all()
    assert near(stats[:, -8:], few_stats, 2 * e * few_stats.abs())
    u, ax = _u("bf16"), tail[0].double().abs()
    assert near(r[-8:], few[0], 2 * u * few[0].double().abs() + 2 * e * (few[0].double().abs() + ax))
    scale = v.double().abs() * few_stats[3].double()[:, None]
    assert near(y[-8:], few[1], 2 * u * few[1].double().abs() + 8 * e * (few[1].double().abs() + scale * ax))
    # (b is needed again; x and y make room for dy, dx and db)
    dy = y.zero_()
    dy[-8:] = tail[2]
    dx, db = big[0], torch.empty_like(r)
    grads = dict(pre_gamma=torch.empty(d, device="cuda"))
    ws = torch.empty(lib.moe_block_join_workspace_size(rows, d, "bf16"), dtype=torch.uint8, device="cuda")
    lib.moe_block_join_backward(big[1], r, stats, w, None, dy, dx, db, lib.make_join_grads(grads), ws, **kw)
    few_dx, few_db = torch.empty_like(few[0]), torch.empty_like(few[0])
    few_grads = dict(pre_gamma=torch.empty(d, device="cuda"))
    few, few_stats = [r[-8:]], stats[:, -8:].contiguous()
    lib.moe_block_join_backward(tail[1], few[0], few_stats, w, None, tail[2], few_dx, few_db,
                                lib.make_join_grads(few_grads), ws, **kw)
    assert torch.equal(dx[-8:], few_dx) and torch.equal(db[-8:], few_db)
    # (the other rows add zeros; sums of 8 terms in another order)
    a, b = grads["pre_gamma"], few_grads["pre_gamma"]
    rh = (few[0].double() * few_stats[3].double()[:, None])
    assert ((a - b).abs() <= 16 * V * (tail[2].double() * rh).abs().sum(0) + TINY).all()


@pytest.mark.parametrize("n,d,vocab", [(5, 4096, 600_000), (600_000, 4096, 40)])
def test_cross_entropy_past_32_bits(lib, n, d, vocab):
    """More than 2^31 elements in W, or in x."""
    g = _gen(4)
    W = torch.randn(vocab, d, dtype=torch.bfloat16, generator=g, device="cuda") * 0.02
    x = torch.randn(n, d, dtype=torch.bfloat16, generator=g, device="cuda")
    t = torch.randint(vocab, (n,), generator=g, device="cuda").to(torch.int32)
    t[-1], t[0] = vocab - 1, -1
    ws = lib.alloc_cross_entropy_workspace(n, d, vocab, "bf16")
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    lib.moe_cross_entropy(x, W, t, loss, lse, ws)
    dloss = torch.full((n,), 1.0 / n, device="cuda")
    dx, dW = torch.empty_like(x), torch.empty_like(W)
    lib.moe_cross_entropy_backward(x, W, t, lse, dloss, dx, dW, ws)
    _ok(lib, ws)
    # the last tokens, and the last entries of the vocabulary
    k, m = min(n, 5), min(vocab, 40)
    l = x[-k:].double() @ W.double().T if vocab * d < 2 ** 31 else torch.cat(
        [x[-k:].double() @ W[v:v + 65536].double().T for v in range(0, vocab, 65536)], 1)
    counted = t[-k:] >= 0
    wlse = torch.where(counted, torch.logsumexp(l, 1), 0.0)
    bound = 2 * d * V * x[-k:].double().norm(dim=1) * W[:1000].double().norm(dim=1).max() * 1.2 + 1e-4
    assert ((lse[-k:].double() - wlse).abs() <= bound).all()
    p = torch.exp(l - wlse[:, None])
    p[torch.arange(k, device="cuda"), t[-k:].long().clamp(min=0)] -= 1
    p = torch.where(counted[:, None], p / n, 0.0)
    wdx = sum(p[:, v:v + 65536] @ W[v:v + 65536].double() for v in range(0, vocab, 65536))
    # norms: dl and the result rounded to bf16 (2^-8 at most each), fp32 sums far below
    for got, want in ((dx[-k:], wdx),):
        assert ((got.double() - want).norm(dim=1) <= 2.2 * 2 ** -8 * want.norm(dim=1) + 1e-30).all()
    pm = torch.zeros(n, m, dtype=torch.float64, device="cuda")
    for a in range(0, n, 65536):
        ls = lse[a:a + 65536].double()[:, None]
        q = torch.exp(x[a:a + 65536].double() @ W[-m:].double().T - ls)
        tt = t[a:a + 65536].long() - (vocab - m)
        hot = torch.nonzero(tt >= 0)[:, 0]
        q[hot, tt[hot]] -= 1
        pm[a:a + 65536] = torch.where((t[a:a + 65536] >= 0)[:, None], q / n, 0.0)
    wdW = sum(pm[a:a + 65536].T @ x[a:a + 65536].double() for a in range(0, n, 65536))
    assert (dW[-m:].double() - wdW).norm() <= 2.2 * 2 ** -8 * wdW.norm()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [(29, 2051), (7, 4099), (33, 2048), (5, 250)])
def test_dropout_rows_anywhere(lib, rows, d, dtype):
    """Rows at every distance from a vector's boundary, alike in x and y and not, give the bits of
    dense rows."""
    g = _gen(d)
    x, rng = _randn(g, rows, d, dtype=dtype), _rng(77, 78)
    want = torch.empty_like(x)
    lib.moe_dropout(x, want, 0.4, rng)
    assert torch.equal(want.cpu() == 0, S.dropout(x, rng, 0.4) == 0)
    for pad in range(1, 9):
        for other in (pad, pad + 8, pad + 3):
            y = _out(rows, d, other, dtype)
            lib.moe_dropout(_rows(x, pad), y, 0.4, rng)
            assert torch.equal(y, want) and _gaps_stay(y, other)


def test_tensors_of_another_device_are_refused(lib, monkeypatch):
    x, t = torch.zeros(4, 64, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    f, ws = torch.zeros(4, device="cuda"), torch.zeros(1024, dtype=torch.uint8, device="cuda")
    v, none = lib.make_join_params({}), lib.make_join_grads({})
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (lambda: lib.moe_dropout(x, x, 0.0),
                 lambda: lib.moe_block_join(x, x, v, x, None, None, post="none", pre="none"),
                 lambda: lib.moe_block_join_backward(x, None, None, v, x, None, x, x, none, ws,
                                                     post="none", pre="none"),
                 lambda: lib.moe_cross_entropy(x, x, t, f, f, ws),
                 lambda: lib.moe_cross_entropy_backward(x, x, t, f, f, x, x, ws)):
        with pytest.raises(ValueError, match="current device"):
            call()


@pytest.mark.parametrize("n,d,vocab,dtype", [(1, 512, 5000, "bf16"), (50, 320, 1100, "bf16"),
                                             (400, 320, 1100, "bf16"), (50, 64, 300, "bf16"),
                                             (50, 64, 300, "f32"), (4, 64, 300, "f32")])
def test_cross_entropy_backward_of_no_finite_weight(lib, n, d, vocab, dtype):
    """A step gone wrong shows in the gradient: no finite dloss leaves no finite gradient."""
    x, W, t, _ = _loss_case(n, d, vocab, dtype, 0.0, 3)
    lse = torch.logsumexp(x.double() @ W.double().T, 1).float()
    ws = lib.alloc_cross_entropy_workspace(n, d, vocab, dtype)
    for bad in (float("nan"), float("inf"), -float("inf")):
        dx, dW = torch.zeros_like(x), torch.zeros_like(W)
        lib.moe_cross_entropy_backward(x, W, t, lse, torch.full_like(lse, bad), dx, dW, ws)
        _ok(lib, ws)
        assert not torch.isfinite(dx).any() and not torch.isfinite(dW).any()
    # beside tokens of weight zero, whose rows stay zero
    weights = torch.zeros_like(lse)
    weights[n // 2] = float("nan")
    dx = torch.zeros_like(x)
    lib.moe_cross_entropy_backward(x, W, t, lse, weights, dx, None, ws)
    others = torch.arange(n, device="cuda") != n // 2
    assert (dx[others] == 0).all() and not torch.isfinite(dx[n // 2]).any()


# vocabularies whose tiles of 96, 160 and 224 entries end in their last 32, of odd length
@pytest.mark.parametrize("n,d,vocab", [(40, 264, 4871), (600, 72, 1601), (257, 136, 4931), (600, 72, 4899),
                                       (257, 64, 7361), (40, 72, 14755)])
def test_cross_entropy_backward_of_tiles_of_any_width(lib, n, d, vocab):
    x, W, t, left = _loss_case(n, d, vocab, "bf16", 0.2, 11)
    t[::3] = torch.where(t[::3] >= 0, vocab - 1 - torch.arange(len(t[::3]), device="cuda") % 40,
                         t[::3].long()).to(torch.int32)      # (targets at the last tile's end)
    clean = torch.where(left[:, None], 0, x)
    lse = torch.where(t >= 0, torch.logsumexp(clean.double() @ W.double().T, 1), 0.0).float()
    dloss = _randn(_gen(n), n)
    ws = lib.alloc_cross_entropy_workspace(n, d, vocab, "bf16")
    ws[256:] = 0xFF
    dx, dW = torch.full_like(x, float("nan")), torch.full_like(W, float("nan"))
    lib.moe_cross_entropy_backward(x, W, t, lse, dloss, dx, dW, ws)
    _ok(lib, ws)
    wdx, ex, wdW, eW = _loss_reference(clean, W, t, lse, dloss, 0.0, "bf16")
    _close(dx, wdx, ex, "dx")
    _close(dW, wdW, eW, "dW")
    assert (dx[left] == 0).all()
