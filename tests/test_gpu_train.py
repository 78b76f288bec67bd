"""GPU: the training operators against the float64 oracle (oracle/train_oracle.py).

Tolerances are element by element and come from the arithmetic, not from what
was measured.  With u the half step of the output type (bf16 2^-8, fp32 2^-24;
torch.finfo(t).eps / 2) and v = 2^-24:
  * a value rounded once is off by u |value|;
  * a sum of m fp32 terms is off by at most m v sum |term|, in any order (2 m v
    for products on the tensor cores, whose adders may truncate);
  * an error in an operand goes through a product with the absolute values of
    the other one;
  * exp and the division of silu (hardware approximations on the bf16 path, at
    most 2^-17 relative over the range of these inputs; CUDA's expf on the fp32
    path) move s = 1 / (1 + e^-g) and g s by `act` relative.
Each bound below is that, written out.
"""
import pytest
import torch

import moe_synth
from oracle import train_oracle as T

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


def _act(dtype):
    return 2.0 ** -16 if dtype == "bf16" else 2.0 ** -20


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype="f32", std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(DT[dtype])


def _within(got, want, bound, what):
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - bound - TINY
    assert over.max().item() <= 0, (what, over.max().item(),
                                    ((got - want).abs() / (bound + TINY)).max().item())


# ------------------------------------------------------------------ layer norm
def _norm_adds(d):
    """Terms that one fp32 sum over a row adds up in sequence, at most."""
    return 64 + d / 256


def _rows(t, pad, fill=float("nan")):
    """t's rows inside a buffer whose rows are pad elements longer, the rest filled."""
    if pad == 0:
        return t.contiguous()
    buf = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


NORM_CASES = [(r, d, pad, dt)
              for dt in ("bf16", "f32")
              for r, d, pad in ((1, 1, 0), (3, 2, 0), (1, 2880, 0), (9, 8, 0), (33, 127, 0),
                                (17, 128, 3), (700, 256, 8), (5, 511, 1), (40, 520, 0),
                                (1021, 1001, 3), (6, 1024, 0), (2500, 2880, 0), (3, 4104, 8),
                                (77, 7168, 0), (4, 8192, 0), (3, 8200, 0), (2, 16392, 0), (3, 9001, 2))]


@pytest.mark.parametrize("rows,d,pad,dtype", NORM_CASES)
def test_layernorm(lib, rows, d, pad, dtype):
    g = _gen(rows * 31 + d)
    x = _rows(_randn(g, rows, d, dtype=dtype, std=2.0) + 0.5, pad)
    gamma = (1 + _randn(g, d, std=0.2)).to(DT[dtype])
    beta = _randn(g, d, dtype=dtype)
    y = _rows(torch.zeros(rows, d, dtype=DT[dtype], device="cuda"), pad, 7.0)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    lib.moe_layernorm(x, gamma, beta, y, mean, rstd, 1e-5)
    wy, wm, wr = T.norm(x, gamma, beta, 1e-5)
    x64, na = x.cpu().double(), _norm_adds(d)
    dm = na * V * x64.abs().mean(1)
    # relative error of rstd: half that of the variance, plus division and root
    er = (na + 8) * V + (dm * wr) ** 2
    _within(mean, wm, dm + V * wm.abs(), "mean")
    _within(rstd, wr, wr * er, "rstd")
    xc = (x64 - wm[:, None]).abs()
    b = gamma.cpu().double().abs() * wr[:, None] * (dm[:, None] + xc * (4 * V + er[:, None]))
    _within(y, wy, b + 2 * V * (wy.abs() + beta.cpu().double().abs()) + _u(dtype) * wy.abs(), "y")
    if pad:
        assert (y.as_strided((rows, pad), (d + pad, 1), d) == 7.0).all()   # the gaps stay
    y2 = torch.empty(rows, d, dtype=DT[dtype], device="cuda")
    lib.moe_layernorm(x, gamma, None, y2, None, None, 1e-5)
    _within(y2, wy - beta.cpu().double(), b + 2 * V * (wy.abs() + beta.cpu().double().abs())
            + _u(dtype) * (wy - beta.cpu().double()).abs(), "y without beta")


@pytest.mark.parametrize("rows,d,pad,dtype", NORM_CASES)
def test_layernorm_backward(lib, rows, d, pad, dtype):
    g = _gen(rows * 37 + d)
    x = _rows(_randn(g, rows, d, dtype=dtype, std=2.0) + 0.5, pad)
    gamma = (1 + _randn(g, d, std=0.2)).to(DT[dtype])
    dy = _rows(_randn(g, rows, d, dtype=dtype), pad)
    _, m64, r64 = T.norm(x, gamma, None, 1e-5)
    mean, rstd = m64.float().cuda(), r64.float().cuda()
    dx = _rows(torch.zeros(rows, d, dtype=DT[dtype], device="cuda"), pad, 7.0)
    dg, db = torch.full((d,), 9.0, device="cuda"), torch.full((d,), 9.0, device="cuda")
    ws = torch.empty(max(256, lib.moe_layernorm_workspace_size(rows, d, dtype)), dtype=torch.uint8,
                     device="cuda")
    lib.moe_layernorm_backward(x, gamma, mean, rstd, dy, dx, dg, db, ws)
    wdx, wdg, wdb = T.norm_backward(x, gamma, mean, rstd, dy)
    na = _norm_adds(d)
    m, r = mean.cpu().double()[:, None], rstd.cpu().double()[:, None]
    dy64 = dy.cpu().double()
    xh = (x.cpu().double() - m) * r
    w = dy64 * gamma.cpu().double()
    m1, m2 = w.mean(1, keepdim=True), (w * xh).mean(1, keepdim=True)
    exh = 3 * V * xh.abs()
    em1 = (na + 2) * V * w.abs().mean(1, keepdim=True)
    em2 = (na + 8) * V * (w * xh).abs().mean(1, keepdim=True)
    b = r * (2 * V * w.abs() + em1 + xh.abs() * em2 + m2.abs() * exh
             + 4 * V * (w.abs() + m1.abs() + (xh * m2).abs()))
    _within(dx, wdx, b + _u(dtype) * wdx.abs(), "dx")
    _within(dg, wdg, (rows + 8) * V * (dy64 * xh).abs().sum(0), "dgamma")
    _within(db, wdb, (rows + 8) * V * dy64.abs().sum(0), "dbeta")
    if pad:
        assert (dx.as_strided((rows, pad), (d + pad, 1), d) == 7.0).all()
    # one of the sums, none of them, and the same bits again
    dx2, dg2, db2 = torch.empty_like(dx), torch.empty_like(dg), torch.empty_like(db)
    lib.moe_layernorm_backward(x, gamma, mean, rstd, dy, dx2, dg2, None, ws)
    lib.moe_layernorm_backward(x, gamma, mean, rstd, dy, dx2, None, db2, ws)
    lib.moe_layernorm_backward(x, gamma, mean, rstd, dy, dx2, None, None, ws)
    assert torch.equal(dx2, dx) and torch.equal(dg2, dg) and torch.equal(db2, db)


def test_layernorm_backward_without_rows(lib):
    e = torch.empty(0, 16, device="cuda")
    s, v = torch.empty(0, device="cuda"), torch.ones(16, device="cuda")
    dg, db = torch.full((16,), 3.0, device="cuda"), torch.full((16,), 3.0, device="cuda")
    lib.moe_layernorm(e, v, v, e, s, s)
    lib.moe_layernorm_backward(e, v, s, s, e, e, dg, db, torch.empty(0, dtype=torch.uint8,
                                                                     device="cuda"))
    assert dg.abs().max() == 0 and db.abs().max() == 0


def test_layernorm_constant_and_nan_rows(lib):
    """A constant row has variance 0 (y = beta); a NaN row does not reach the others."""
    x = torch.randn(4, 64, device="cuda", generator=_gen(1))
    x[1] = 3.0
    x[2, 5] = float("nan")
    gamma, beta = torch.ones(64, device="cuda"), torch.full((64,), 0.25, device="cuda")
    y = torch.empty_like(x)
    lib.moe_layernorm(x, gamma, beta, y, None, None, 1e-5)
    assert torch.equal(y[1], beta) and torch.isnan(y[2]).all()
    assert torch.isfinite(y[[0, 1, 3]]).all()


# ----------------------------------------------------------- the expert FFNs
def _cfg(n, d, F, E, k, dtype, act="swiglu", gate="renorm"):
    return moe_synth.MoEConfig("t", n, d, F, E, k, dtype, dtype, gate, act)


def _counts(P, E, how, seed):
    g = torch.Generator().manual_seed(seed)
    if how == "even":
        c = torch.bincount(torch.randint(0, E, (P,), generator=g), minlength=E)
    elif how == "one":
        c = torch.zeros(E, dtype=torch.int64)
        c[E // 2] = P
    else:
        c = torch.tensor(how)
        assert c.numel() == E and int(c.sum()) == P
    return torch.cat([torch.zeros(1, dtype=torch.int64), c.cumsum(0)]).to(torch.int32).cuda()


EDGES = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 0, 255, 256, 257, 300]
TAILS = [2, 31, 0, 33, 66, 95, 7, 198]
MANY = [0, 1, 300, 17, 20] * 8

# n, d, F, E, k, dtype, act, counts
FFN_CASES = [
    (1, 8, 8, 1, 1, "bf16", "swiglu", "even"),
    (1, 8, 8, 4, 1, "bf16", "relu", "even"),
    (200, 256, 384, 8, 2, "bf16", "swiglu", "even"),
    (37, 72, 136, 5, 2, "bf16", "swiglu", "even"),
    (37, 72, 136, 5, 2, "bf16", "relu", "even"),
    (sum(EDGES), 72, 264, len(EDGES), 1, "bf16", "swiglu", EDGES),
    (sum(EDGES), 264, 72, len(EDGES), 1, "bf16", "relu", EDGES),
    (sum(TAILS), 520, 520, len(TAILS), 1, "bf16", "swiglu", TAILS),
    (300, 128, 200, 6, 2, "bf16", "swiglu", "one"),
    (40, 64, 96, 256, 4, "bf16", "swiglu", "even"),
    (9, 1544, 64, 3, 2, "bf16", "swiglu", "even"),
    (700, 512, 1024, 1, 1, "bf16", "swiglu", "even"),
    # few tiles and many rows: the weight gradients' reduction is cut into runs
    (2100, 72, 136, 2, 1, "bf16", "swiglu", [2099, 1]),
    (2500, 264, 64, 2, 1, "bf16", "relu", [1233, 1267]),
    (1600, 72, 72, 1, 1, "bf16", "swiglu", "even"),
    # few tiles and long reductions: the row products are cut into ranges
    (33, 72, 2104, 2, 1, "bf16", "swiglu", [20, 13]),
    (33, 2104, 72, 2, 1, "bf16", "swiglu", [0, 33]),
    (300, 136, 1096, 1, 1, "bf16", "relu", "even"),
    (7, 1096, 136, 1, 1, "bf16", "relu", "even"),
    # few rows per expert and many tiles: weight gradients beside the row products
    (sum(MANY), 264, 520, len(MANY), 1, "bf16", "swiglu", MANY),
    (450, 520, 264, 40, 2, "bf16", "relu", "even"),
    (1, 4, 4, 1, 1, "f32", "swiglu", "even"),
    (256, 128, 512, 4, 1, "f32", "relu", "even"),
    (83, 36, 100, 7, 2, "f32", "swiglu", "even"),
    (sum(TAILS), 68, 132, len(TAILS), 1, "f32", "swiglu", TAILS),
    (1400, 36, 68, 2, 1, "f32", "swiglu", [1399, 1]),
    (700, 68, 36, 1, 1, "f32", "relu", "even"),
    (1027, 36, 24, 1, 1, "f32", "swiglu", "even"),
]


def _ffn_inputs(case, seed=3):
    n, d, F, E, k, dtype, act, how = case
    cfg = _cfg(n, d, F, E, k, dtype, act)
    g = _gen(seed + d)
    P = n * k
    s = dict(cfg=cfg, offsets=_counts(P, E, how, seed), x=_randn(g, P, d, dtype=dtype),
             W1=_randn(g, E, F, d, dtype=dtype, std=d ** -0.5),
             W3=_randn(g, E, F, d, dtype=dtype, std=d ** -0.5) if act == "swiglu" else None,
             W2=_randn(g, E, d, F, dtype=dtype, std=F ** -0.5), dy=_randn(g, P, d, dtype=dtype))
    return s


def _empty(s, width, fill=float("nan")):
    return torch.full((s["x"].shape[0], width), fill, dtype=s["x"].dtype, device="cuda")


def _train(lib, s, ws):
    F, gated = s["W1"].shape[1], s["W3"] is not None
    g, u = (_empty(s, F), _empty(s, F)) if gated else (None, None)
    h, y = _empty(s, F), _empty(s, s["x"].shape[1])
    lib.moe_expert_ffn_train(s["cfg"], s["x"], s["offsets"], lib.make_weights(s), g, u, h, y, ws)
    return g, u, h, y


def _ok(lib, ws):
    st, detail = lib.moe_status_check(ws)
    assert st == 0, (lib.status_string(st), detail)


def _seg(fn, offsets, *ts):
    """fn(e, rows of each t) joined over the segments."""
    off = offsets.tolist()
    return torch.cat([fn(e, *(t[a:b] for t in ts)) for e, (a, b) in enumerate(zip(off, off[1:]))])


@pytest.mark.parametrize("case", FFN_CASES, ids=str)
def test_ffn_train(lib, case):
    n, d, F, E, k, dtype, act, _ = case
    s = _ffn_inputs(case)
    ws = lib.alloc_train_workspace(s["cfg"])
    g, u, h, y = _train(lib, s, ws)
    _ok(lib, ws)
    off = s["offsets"].cpu()
    wy, wg, wu, wh = T.ffn(s["x"], off, s["W1"], s["W3"], s["W2"])
    ax = s["x"].cpu().double().abs()
    aW = {key: None if s[key] is None else s[key].cpu().double().abs() for key in ("W1", "W3", "W2")}
    eg = 2 * d * V * _seg(lambda e, x: x @ aW["W1"][e].T, off, ax)
    if act == "swiglu":
        eu = 2 * d * V * _seg(lambda e, x: x @ aW["W3"][e].T, off, ax)
        _within(g, wg, eg + _u(dtype) * wg.abs(), "g")
        _within(u, wu, eu + _u(dtype) * wu.abs(), "u")
        # |silu'| <= 1.1
        eh = (1.1 * eg * (wu.abs() + eu) + (wh / wu.where(wu != 0, torch.ones_like(wu))).abs() * eu
              + _act(dtype) * wh.abs())
    else:
        eh = eg
    eh = eh + _u(dtype) * (wh.abs() + eh)
    _within(h, wh, eh, "h")
    ey = _seg(lambda e, a, b: (a + 2 * F * V * b) @ aW["W2"][e].T, off, eh, wh.abs() + eh)
    _within(y, wy, ey + _u(dtype) * (wy.abs() + ey), "y")


def _grads(s):
    return {key: None if s[key] is None else torch.full_like(s[key], float("nan"))
            for key in ("W1", "W3", "W2")}


@pytest.mark.parametrize("case", FFN_CASES, ids=str)
def test_ffn_backward(lib, case):
    n, d, F, E, k, dtype, act, _ = case
    s = _ffn_inputs(case, 11)
    ws = lib.alloc_train_workspace(s["cfg"])
    g, u, h, _y = _train(lib, s, ws)
    dx, gr = _empty(s, d), _grads(s)
    w = lib.make_weights(s)
    back = lambda dx, gr: lib.moe_expert_ffn_backward(s["cfg"], s["x"], s["offsets"], w, g, u, h,
                                                      s["dy"], dx, lib.make_expert_grads(gr), ws)
    back(dx, gr)
    _ok(lib, ws)
    off = s["offsets"].cpu()
    wdx, wW1, wW3, wW2, wdg, wdu = T.ffn_backward(s["x"], off, s["W1"], s["W3"], s["W2"], g, u, h,
                                                  s["dy"])
    a = {key: None if t is None else t.cpu().double().abs() for key, t in
         dict(x=s["x"], dy=s["dy"], W1=s["W1"], W3=s["W3"], W2=s["W2"], g=g, u=u, h=h).items()}
    adh = _seg(lambda e, t: t @ a["W2"][e], off, a["dy"])       # sum of |terms| of dh, >= |dh|
    edh = 2 * d * V * adh
    if act == "swiglu":
        # the factors: |s (1 + g (1 - s))| <= 1.1, |g s| <= |g|
        edg = 1.1 * edh * a["u"] + 3 * _act(dtype) * adh * a["u"]
        edu = edh * a["g"] + 3 * _act(dtype) * adh * a["g"]
        edu = edu + _u(dtype) * (wdu.abs() + edu)
    else:
        edg = edh
    edg = edg + _u(dtype) * (wdg.abs() + edg)
    rows = 2 * F * V * (2 if act == "swiglu" else 1)
    ex = _seg(lambda e, p, q: (p + rows * q) @ a["W1"][e], off, edg, wdg.abs() + edg)
    if act == "swiglu":
        ex = ex + _seg(lambda e, p, q: (p + rows * q) @ a["W3"][e], off, edu, wdu.abs() + edu)
    _within(dx, wdx, ex + _u(dtype) * (wdx.abs() + ex), "dx")

    def weight(got, want, left, eleft, right, what):
        o = off.tolist()
        b = torch.stack([(eleft[p:q] + 2 * (q - p) * V * left[p:q]).T @ right[p:q]
                         for p, q in zip(o, o[1:])])
        _within(got, want, b + _u(dtype) * (want.abs() + b), what)
        for e, (p, q) in enumerate(zip(o, o[1:])):
            if p == q:
                assert got[e].abs().max() == 0, (what, e)

    weight(gr["W2"], wW2, a["dy"], torch.zeros_like(a["dy"]), a["h"], "dW2")
    weight(gr["W1"], wW1, wdg.abs() + edg, edg, a["x"], "dW1")
    if act == "swiglu":
        weight(gr["W3"], wW3, wdu.abs() + edu, edu, a["x"], "dW3")
    # every part alone gives the same bits
    dx2, gr2 = _empty(s, d), _grads(s)
    back(dx2, dict(W1=None, W3=None, W2=None))
    back(None, dict(W1=gr2["W1"]))
    back(None, dict(W2=gr2["W2"]))
    if act == "swiglu":
        back(None, dict(W3=gr2["W3"]))
    _ok(lib, ws)
    assert torch.equal(dx, dx2)
    for key in gr:
        assert gr[key] is None or torch.equal(gr[key], gr2[key]), key


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_ffn_backward_keeps_experts_apart(lib, dtype, bad):
    """NaN and infinity in one segment's rows reach no other expert's results, although
    the segments meet inside a tile."""
    counts = [5, 3, 70, 1, 50]
    s = _ffn_inputs((sum(counts), 136, 72, 5, 1, dtype, "swiglu", counts))
    ws = lib.alloc_train_workspace(s["cfg"])
    off = s["offsets"].tolist()

    def run():
        g, u, h, y = _train(lib, s, ws)
        dx, gr = _empty(s, 136), _grads(s)
        lib.moe_expert_ffn_backward(s["cfg"], s["x"], s["offsets"], lib.make_weights(s), g, u, h,
                                    s["dy"], dx, lib.make_expert_grads(gr), ws)
        _ok(lib, ws)
        return [y, dx], [gr["W1"], gr["W3"], gr["W2"]]

    rows0, w0 = run()
    for e in (1, 3):
        for key in ("x", "dy"):
            s[key][off[e]:off[e + 1]] = bad
    rows1, w1 = run()
    keep = [e for e in range(5) if e not in (1, 3)]
    for p, q in zip(rows0, rows1):
        for e in keep:
            assert torch.equal(p[off[e]:off[e + 1]], q[off[e]:off[e + 1]])
    for p, q in zip(w0, w1):
        for e in keep:
            assert torch.equal(p[e], q[e])
        assert not torch.isfinite(q[1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ffn_rows_outside_the_segments_stay(lib, dtype):
    """Offsets that end before the last row (pairs that the dispatch skipped)."""
    counts = [20, 0, 13]
    s = _ffn_inputs((40, 64, 72, 3, 1, dtype, "swiglu", [20, 0, 20]))
    s["offsets"] = torch.tensor([0, 20, 20, 33], dtype=torch.int32, device="cuda")
    s["x"][33:] = float("nan")
    s["dy"][33:] = float("nan")
    ws = lib.alloc_train_workspace(s["cfg"])
    F = 72
    g, u, h, y = (_empty(s, w, 5.0) for w in (F, F, F, 64))
    lib.moe_expert_ffn_train(s["cfg"], s["x"], s["offsets"], lib.make_weights(s), g, u, h, y, ws)
    dx, gr = _empty(s, 64, 5.0), _grads(s)
    lib.moe_expert_ffn_backward(s["cfg"], s["x"], s["offsets"], lib.make_weights(s), g, u, h, s["dy"],
                                dx, lib.make_expert_grads(gr), ws)
    _ok(lib, ws)
    for t in (g, u, h, y, dx):
        assert (t[33:] == 5.0).all() and torch.isfinite(t[:33]).all()
    for t in gr.values():
        assert torch.isfinite(t).all()
    assert sum(counts) == 33


@pytest.mark.parametrize("d,F", [(1096, 72), (72, 1096)])
def test_ffn_rows_outside_the_segments_stay_with_cut_reductions(lib, d, F):
    s = _ffn_inputs((40, d, F, 2, 1, "bf16", "swiglu", [20, 20]))
    s["offsets"] = torch.tensor([3, 20, 33], dtype=torch.int32, device="cuda")
    for key in ("x", "dy"):
        s[key][:3] = float("nan")
        s[key][33:] = float("nan")
    ws = lib.alloc_train_workspace(s["cfg"])
    ws[256:] = 255                                       # (NaN wherever scratch is not written)
    g, u, h, y = (_empty(s, w, 5.0) for w in (F, F, F, d))
    lib.moe_expert_ffn_train(s["cfg"], s["x"], s["offsets"], lib.make_weights(s), g, u, h, y, ws)
    dx, gr = _empty(s, d, 5.0), _grads(s)
    lib.moe_expert_ffn_backward(s["cfg"], s["x"], s["offsets"], lib.make_weights(s), g, u, h, s["dy"],
                                dx, lib.make_expert_grads(gr), ws)
    _ok(lib, ws)
    for t in (g, u, h, y, dx):
        assert (t[:3] == 5.0).all() and (t[33:] == 5.0).all() and torch.isfinite(t[3:33]).all()
    for t in gr.values():
        assert torch.isfinite(t).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offsets", [[0, 20, 10, 40], [0, 10, 20, 41], [-1, 10, 20, 40]])
def test_ffn_bad_offsets_are_reported(lib, dtype, offsets):
    s = _ffn_inputs((40, 64, 72, 3, 1, dtype, "swiglu", "even"))
    s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    ws = lib.alloc_train_workspace(s["cfg"])
    _train(lib, s, ws)
    assert lib.moe_status_check(ws)[0] == 5
    lib.moe_status_clear(ws)
    h = _empty(s, 72, 1.0)
    lib.moe_expert_ffn_backward(s["cfg"], s["x"], s["offsets"], lib.make_weights(s), h, h, h, s["dy"],
                                _empty(s, 64), lib.make_expert_grads(_grads(s)), ws)
    assert lib.moe_status_check(ws)[0] == 5


# ------------------------------------------------------------ combine, router
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,k,d", [(1, 1, 8), (37, 4, 2880), (5, 7, 24), (600, 8, 264), (3, 256, 16),
                                   (2, 3, 7168)])
def test_combine_backward(lib, n, k, d, dtype):
    cfg = _cfg(n, d, 8, 256, k, dtype)
    g = _gen(n + k + d)
    P = n * k
    dy, yp = _randn(g, n, d, dtype=dtype), _randn(g, P, d, dtype=dtype)
    gate = torch.rand(n, k, generator=g, device="cuda")
    inv = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    dyp, dgate = torch.full_like(yp, 5.0), torch.full_like(gate, 5.0)
    ws = lib.alloc_train_workspace(cfg)
    lib.moe_combine_backward(cfg, dy, yp, inv, gate, dyp, dgate, ws)
    _ok(lib, ws)
    wdy, wdg = T.combine_backward(dy, yp, inv, gate)
    _within(dyp, wdy, (_u(dtype) + 2 * V) * wdy.abs(), "dy_perm")
    rows = yp[inv.long()].cpu().double().view(n, k, d)
    terms = (rows * dy.cpu().double()[:, None]).abs().sum(2)
    _within(dgate, wdg, (d / 32 + 16) * V * terms, "dgate")
    dyp2 = torch.empty_like(dyp)
    lib.moe_combine_backward(cfg, dy, None, inv, gate, dyp2, None, ws)
    assert torch.equal(dyp, dyp2)


def test_combine_backward_bad_index(lib):
    cfg = _cfg(4, 16, 8, 4, 2, "bf16")
    g = _gen(2)
    dy, yp = _randn(g, 4, 16, dtype="bf16"), _randn(g, 8, 16, dtype="bf16")
    gate = torch.rand(4, 2, generator=g, device="cuda")
    inv = torch.tensor([0, 1, 2, -1, 8, 5, 6, 7], dtype=torch.int32, device="cuda")
    dyp, dgate = torch.full_like(yp, 5.0), torch.full_like(gate, 5.0)
    ws = lib.alloc_train_workspace(cfg)
    lib.moe_combine_backward(cfg, dy, yp, inv, gate, dyp, dgate, ws)
    st, detail = lib.moe_status_check(ws)
    assert st == 5 and detail in (3, 4)
    assert (dyp[3:5] == 5.0).all()                  # the rows that no pair maps to


ROUTE_CASES = [(n, d, E, k, dt, gate, aux)
               for dt in ("bf16", "f32")
               for n, d, E, k, gate, aux in (
                   (1, 8, 1, 1, "top_prob", 0.01), (256, 128, 4, 1, "top_prob", 0.01),
                   (200, 72, 8, 2, "renorm", 0.0), (33, 520, 37, 5, "renorm", 0.3),
                   (700, 264, 256, 8, "renorm", 0.0), (65, 136, 200, 6, "top_prob", 0.2),
                   (3, 64, 40, 40, "renorm", 0.0), (2500, 24, 3, 2, "top_prob", 0.0),
                   (1537, 520, 130, 4, "renorm", 0.1))]


@pytest.mark.parametrize("n,d,E,k,dtype,gate,aux", ROUTE_CASES)
def test_route_backward(lib, n, d, E, k, dtype, gate, aux):
    cfg = _cfg(n, d, 8, E, k, dtype, gate=gate)
    g = _gen(n + d + E)
    x, Wg = _randn(g, n, d, dtype=dtype), _randn(g, E, d, dtype=dtype, std=0.1)
    probs = torch.softmax(_randn(g, n, E, std=1.5), 1)
    p, idx = torch.sort(probs, dim=1, descending=True, stable=True)
    p, idx = p[:, :k].contiguous(), idx[:, :k].to(torch.int32).contiguous()
    gates = (p / p.sum(1, keepdim=True) if gate == "renorm" else p).contiguous()
    dgate = _randn(g, n, k)
    f = torch.bincount(idx[:, 0].long(), minlength=E).float() / n if aux else None
    inv = torch.randperm(n * k, generator=g, device="cuda").to(torch.int32)
    dxp = _randn(g, n * k, d, dtype=dtype)
    ws = lib.alloc_train_workspace(cfg)
    w = lib.make_weights(dict(Wg=Wg))

    def run(inv, dxp, dx, dWg, db, probs=probs):
        lib.moe_route_backward(cfg, x, w, probs, idx, gates, dgate, f, aux, inv, dxp, dx, dWg, db, ws)
        _ok(lib, ws)

    nan = float("nan")
    dx, dWg, db = torch.full_like(x, nan), torch.full_like(Wg, nan), torch.full((E,), nan,
                                                                              device="cuda")
    run(inv, dxp, dx, dWg, db)
    dl = T.logits_backward(gate, probs, idx, gates, dgate, f, aux)
    wdx, wdWg, wdb = T.route_backward(dl, x, Wg, inv, dxp)
    # fp32 error of dl: k + E terms, each a product of two or three factors
    mag = torch.zeros(n, E, dtype=torch.float64)
    ag, adg, p64 = gates.cpu().double(), dgate.cpu().double().abs(), probs.cpu().double()
    total = (ag * adg).sum(1, keepdim=True)
    mag.scatter_(1, idx.cpu().long(), ag * (adg + (total if gate == "renorm" else 0)))
    if gate != "renorm":
        mag += p64 * total
    if aux:
        f64 = f.cpu().double()
        mag += aux * E / n * p64 * (f64 + p64 @ f64[:, None])
    el = (k + E + 10) * V * mag
    ea = el + (_u(dtype) if dtype == "bf16" else 0) * (dl.abs() + el)
    aW, ax = Wg.cpu().double().abs(), x.cpu().double().abs()
    er = (ea + 2 * E * V * (dl.abs() + ea)) @ aW
    er = er + _u(dtype) * ((dl @ Wg.cpu().double()).abs() + er)     # kept in the rows' type
    rows = dxp[inv.long()].cpu().double().view(n, k, d)
    ex = er + (k + 2) * V * (rows.abs().sum(1) + (dl.abs() + ea) @ aW)
    _within(dx, wdx, ex + _u(dtype) * (wdx.abs() + ex), "dx")
    ew = (ea + 2 * n * V * (dl.abs() + ea)).T @ ax
    _within(dWg, wdWg, ew + _u(dtype) * (wdWg.abs() + ew), "dWg")
    _within(db, wdb, (el + (n + 8) * V * (dl.abs() + el)).sum(0), "dbias")
    # the router's share alone, each output alone, and probs where they are not needed
    dx2 = torch.full_like(x, nan)
    run(None, None, dx2, None, None)
    _within(dx2, dl @ Wg.cpu().double(), er, "dx of the router alone")
    dx3, dW3, db3 = torch.full_like(dx, nan), torch.full_like(dWg, nan), torch.full_like(db, nan)
    run(inv, dxp, dx3, None, None, None if gate == "renorm" and not aux else probs)
    run(None, None, None, dW3, None)
    run(None, None, None, None, db3)
    run(None, None, None, None, None)
    assert torch.equal(dx, dx3) and torch.equal(dWg, dW3) and torch.equal(db, db3)


@pytest.mark.parametrize("n,d,E,k,gate", [(1, 16, 3, 3, "renorm"), (21, 168, 2, 1, "top_prob"),
                                          (600, 24, 40, 2, "top_prob"), (5, 264, 37, 4, "renorm")])
def test_route_backward_of_small_bf16_layers_rounds_once(lib, n, d, E, k, gate):
    """dl stays in fp32 between the launches of a small layer: the only rounding to bf16 is
    the output's."""
    cfg = _cfg(n, d, 8, E, k, "bf16", gate=gate)
    g = _gen(n + E)
    x, Wg = _randn(g, n, d, dtype="bf16"), _randn(g, E, d, dtype="bf16", std=0.1)
    probs = torch.softmax(_randn(g, n, E, std=1.5), 1)
    p, idx = torch.sort(probs, dim=1, descending=True, stable=True)
    p, idx = p[:, :k].contiguous(), idx[:, :k].to(torch.int32).contiguous()
    gates = (p / p.sum(1, keepdim=True) if gate == "renorm" else p).contiguous()
    dgate = _randn(g, n, k)
    f = torch.full((E,), 1 / E, device="cuda")
    ws = lib.alloc_train_workspace(cfg)
    dx, dWg = torch.full_like(x, float("nan")), torch.full_like(Wg, float("nan"))
    lib.moe_route_backward(cfg, x, lib.make_weights(dict(Wg=Wg)), probs, idx, gates, dgate, f, 0.1,
                           None, None, dx, dWg, None, ws)
    _ok(lib, ws)
    dl = T.logits_backward(gate, probs, idx, gates, dgate, f, 0.1)
    # (dl's own fp32 error as in test_route_backward)
    mag = torch.zeros(n, E, dtype=torch.float64)
    ag, adg, p64 = gates.cpu().double(), dgate.cpu().double().abs(), probs.cpu().double()
    total = (ag * adg).sum(1, keepdim=True)
    mag.scatter_(1, idx.cpu().long(), ag * (adg + (total if gate == "renorm" else 0)))
    if gate != "renorm":
        mag += p64 * total
    mag += 0.1 * E / n * p64 * 2 / E
    el = (k + E + 10) * V * mag
    aW, ax = Wg.cpu().double().abs(), x.cpu().double().abs()
    want = dl @ Wg.cpu().double()
    ex = (el + 2 * E * V * (dl.abs() + el)) @ aW
    _within(dx, want, ex + _u("bf16") * (want.abs() + ex), "dx")
    want = dl.T @ x.cpu().double()
    ew = (el + 2 * n * V * (dl.abs() + el)).T @ ax
    _within(dWg, want, ew + _u("bf16") * (want.abs() + ew), "dWg")


@pytest.mark.parametrize("n,d,F,E,act", [(1, 200, 104, 1, "swiglu"), (14, 200, 24, 3, "swiglu"),
                                         (7, 24, 248, 4, "relu"), (100, 72, 136, 5, "swiglu")])
def test_ffn_backward_of_small_bf16_layers_rounds_once(lib, n, d, F, E, act):
    """dg and du stay in fp32 between the launches of a small layer."""
    s = _ffn_inputs((n, d, F, E, 1, "bf16", act, "even"), 17)
    ws = lib.alloc_train_workspace(s["cfg"])
    g, u, h, _y = _train(lib, s, ws)
    dx, gr = _empty(s, d), _grads(s)
    lib.moe_expert_ffn_backward(s["cfg"], s["x"], s["offsets"], lib.make_weights(s), g, u, h,
                                s["dy"], dx, lib.make_expert_grads(gr), ws)
    _ok(lib, ws)
    off = s["offsets"].cpu()
    wdx, wW1, wW3, _wW2, wdg, wdu = T.ffn_backward(s["x"], off, s["W1"], s["W3"], s["W2"], g, u, h,
                                                   s["dy"])
    a = {key: None if t is None else t.cpu().double().abs() for key, t in
         dict(x=s["x"], dy=s["dy"], W1=s["W1"], W3=s["W3"], W2=s["W2"], g=g, u=u).items()}
    adh = _seg(lambda e, t: t @ a["W2"][e], off, a["dy"])
    edg, edu = 2 * d * V * adh, None
    if act == "swiglu":     # (the factors as in test_ffn_backward)
        edu = 2 * d * V * adh * a["g"] + 3 * _act("bf16") * adh * a["g"]
        edg = 1.1 * edg * a["u"] + 3 * _act("bf16") * adh * a["u"]
    ex = _seg(lambda e, p, q: (p + 4 * F * V * q) @ a["W1"][e], off, edg, wdg.abs() + edg)
    if act == "swiglu":
        ex = ex + _seg(lambda e, p, q: (p + 4 * F * V * q) @ a["W3"][e], off, edu, wdu.abs() + edu)
    _within(dx, wdx, ex + _u("bf16") * (wdx.abs() + ex), "dx")
    o = off.tolist()
    for got, want, dv, edv in ((gr["W1"], wW1, wdg, edg), (gr["W3"], wW3, wdu, edu)):
        if got is not None:
            b = torch.stack([(edv[p:q] + 2 * (q - p) * V * (dv[p:q].abs() + edv[p:q])).T
                             @ a["x"][p:q] for p, q in zip(o, o[1:])])
            _within(got, want, b + _u("bf16") * (want.abs() + b), "dW")


def test_route_backward_masked_experts_and_bad_index(lib):
    """An expert that a -inf bias masks (probability 0) has no gradient; a choice outside
    the experts is reported and counts as a gate of zero."""
    n, d, E, k = 9, 64, 6, 2
    cfg = _cfg(n, d, 8, E, k, "f32", gate="top_prob")
    g = _gen(4)
    x, Wg = _randn(g, n, d), _randn(g, E, d)
    logits = _randn(g, n, E)
    logits[:, 2] = -float("inf")
    probs = torch.softmax(logits, 1)
    p, idx = torch.sort(probs, dim=1, descending=True, stable=True)
    p, idx = p[:, :k].contiguous(), idx[:, :k].to(torch.int32).contiguous()
    dgate = _randn(g, n, k)
    f = torch.full((E,), 1 / E, device="cuda")
    ws = lib.alloc_train_workspace(cfg)
    dx, dWg, db = torch.empty_like(x), torch.empty_like(Wg), torch.empty(E, device="cuda")
    w = lib.make_weights(dict(Wg=Wg))
    lib.moe_route_backward(cfg, x, w, probs, idx, p, dgate, f, 0.1, None, None, dx, dWg, db, ws)
    _ok(lib, ws)
    assert dWg[2].abs().max() == 0 and db[2] == 0 and torch.isfinite(dx).all()
    idx[3, 1] = E
    lib.moe_route_backward(cfg, x, w, probs, idx, p, dgate, f, 0.1, None, None, dx, dWg, db, ws)
    assert lib.moe_status_check(ws) == (5, 3 * k + 1)


# ------------------------------------------------------------------ a whole step
def test_gradients_against_differences(lib):
    """The fp32 layer's loss, moved along each gradient: (L(t + e v) - L(t - e v)) / 2e against
    <grad, v>.  The differences' own error: the third derivative's e^2 / 6 term and fp32 rounding
    of L over e; with e = 2^-6 both stay under 2 % of |grad| |v| here."""
    n, d, F, E, k = 24, 32, 48, 4, 2
    cfg = _cfg(n, d, F, E, k, "f32")
    g = _gen(8)
    p = dict(x=_randn(g, n, d), gamma=1 + _randn(g, d, std=0.1), beta=_randn(g, d, std=0.1),
             Wg=_randn(g, E, d, std=0.2), W1=_randn(g, E, F, d, std=0.2), W3=_randn(g, E, F, d, std=0.2),
             W2=_randn(g, E, d, F, std=0.2))
    dy = _randn(g, n, d)
    ws = lib.alloc_train_workspace(cfg)
    P = n * k
    new = lambda *shape: torch.empty(*shape, device="cuda")
    nws = torch.empty(max(256, lib.moe_layernorm_workspace_size(n, d, "f32")), dtype=torch.uint8,
                      device="cuda")
    a = dict(xn=new(n, d), mean=new(n), rstd=new(n), idx=torch.empty(n, k, dtype=torch.int32,
                                                                    device="cuda"),
             gate=new(n, k), probs=new(n, E), xp=new(P, d), g=new(P, F), u=new(P, F), h=new(P, F),
             yp=new(P, d), y=new(n, d))
    ints = [torch.empty(m, dtype=torch.int32, device="cuda") for m in (E, E + 1, P, P)]

    def forward(p):
        w = lib.make_weights(p)
        lib.moe_layernorm(p["x"], p["gamma"], p["beta"], a["xn"], a["mean"], a["rstd"])
        lib.moe_route(cfg, a["xn"], w, a["idx"], a["gate"], a["probs"], ws)
        lib.moe_dispatch(cfg, a["idx"], a["xn"], *ints, a["xp"], ws)
        lib.moe_expert_ffn_train(cfg, a["xp"], ints[1], w, a["g"], a["u"], a["h"], a["yp"], ws)
        lib.moe_combine(cfg, a["yp"], ints[3], a["gate"], None, a["y"], ws)
        _ok(lib, ws)
        return (a["y"].double() * dy.double()).sum().item(), a["idx"].clone()

    _, idx0 = forward(p)
    w = lib.make_weights(p)
    gr = {key: torch.empty_like(t) for key, t in p.items()}
    dyp, dgate, dxp, dxn = new(P, d), new(n, k), new(P, d), new(n, d)
    lib.moe_combine_backward(cfg, dy, a["yp"], ints[3], a["gate"], dyp, dgate, ws)
    lib.moe_expert_ffn_backward(cfg, a["xp"], ints[1], w, a["g"], a["u"], a["h"], dyp, dxp,
                                lib.make_expert_grads(gr), ws)
    lib.moe_route_backward(cfg, a["xn"], w, None, a["idx"], a["gate"], dgate, None, 0.0, ints[3], dxp,
                           dxn, gr["Wg"], None, ws)
    lib.moe_layernorm_backward(p["x"], p["gamma"], a["mean"], a["rstd"], dxn, gr["x"], gr["gamma"],
                               gr["beta"], nws)
    _ok(lib, ws)
    e = 2.0 ** -6
    for key, t in p.items():
        v = gr[key] / gr[key].norm() * t.norm() * 0.05      # along the gradient: <grad, v> is large
        up, i1 = forward({**p, key: t + e * v})
        down, i2 = forward({**p, key: t - e * v})
        assert torch.equal(i1, idx0) and torch.equal(i2, idx0)   # (the loss is smooth in between)
        want = (gr[key].double() * v.double()).sum().item()
        assert abs((up - down) / (2 * e) - want) <= 2e-2 * abs(want), key


@pytest.mark.parametrize("wanted", ["W1 W3 W2 dx", "W3 dx", "W2 dx", "W2 W1"])
def test_ffn_backward_side_by_side_again_and_again(lib, wanted):
    """Launches that run at the same time, back to back without a wait, followed at once by
    work that overwrites their inputs: the bits of a run with a wait after each call."""
    s = _ffn_inputs((sum(MANY), 264, 520, len(MANY), 1, "bf16", "swiglu", MANY), 5)
    ws = lib.alloc_train_workspace(s["cfg"])
    g, u, h, _y = _train(lib, s, ws)
    gr = {key: t if key in wanted else None for key, t in _grads(s).items()}
    dx = _empty(s, 264) if "dx" in wanted else None
    x2, dy2 = s["x"].flip(0).contiguous(), s["dy"].flip(0).contiguous()
    x, dy = s["x"].clone(), s["dy"].clone()
    w = lib.make_weights(s)

    def back():
        lib.moe_expert_ffn_backward(s["cfg"], x, s["offsets"], w, g, u, h, dy, dx,
                                    lib.make_expert_grads(gr), ws)
        return [t.clone() for t in (dx, *gr.values()) if t is not None]

    want = []
    for a, b in ((s["x"], s["dy"]), (x2, dy2)):
        x.copy_(a), dy.copy_(b)
        torch.cuda.synchronize()
        want.append(back())
        _ok(lib, ws)
    got = []
    for i in range(10):
        x.copy_((s["x"], x2)[i % 2]), dy.copy_((s["dy"], dy2)[i % 2])
        got.append(back())
    _ok(lib, ws)
    for i, ts in enumerate(got):
        for a, b in zip(ts, want[i % 2]):
            assert torch.equal(a, b), i


def test_ffn_backward_side_by_side_in_a_graph(lib):
    s = _ffn_inputs((sum(MANY), 264, 520, len(MANY), 1, "bf16", "swiglu", MANY), 6)
    ws = lib.alloc_train_workspace(s["cfg"])
    g, u, h, _y = _train(lib, s, ws)
    dx, gr, w = _empty(s, 264), _grads(s), lib.make_weights(s)
    outs = (dx, *gr.values())

    def back(stream=None):
        lib.moe_expert_ffn_backward(s["cfg"], s["x"], s["offsets"], w, g, u, h, s["dy"], dx,
                                    lib.make_expert_grads(gr), ws, stream=stream)

    back()
    _ok(lib, ws)
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            back(side)
            kept = [t.clone() for t in outs]        # (reads the results inside the graph)
            for t in outs:
                t.fill_(0)
    for _ in range(3):
        for t in kept:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(kept, want):
            assert torch.equal(a, b)
    _ok(lib, ws)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_in_a_graph_on_another_stream(lib, dtype):
    """The gradients captured on a side stream and replayed give the eager run's bits."""
    s = _ffn_inputs((50, 136, 264, 6, 2, dtype, "swiglu", "even"))
    ws = lib.alloc_train_workspace(s["cfg"])
    w = lib.make_weights(s)
    g, u, h, y = _train(lib, s, ws)
    dx, gr = _empty(s, 136), _grads(s)

    def back(stream=None):
        lib.moe_expert_ffn_backward(s["cfg"], s["x"], s["offsets"], w, g, u, h, s["dy"], dx,
                                    lib.make_expert_grads(gr), ws, stream=stream)

    back()
    _ok(lib, ws)
    want = [t.clone() for t in (dx, *gr.values())]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            back(side)
    for t in (dx, *gr.values()):
        t.fill_(float("nan"))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((dx, *gr.values()), want):
        assert torch.equal(a, b)
