"""The float64 training oracle against autograd and against central differences,
and the C entry points' refusals.  No GPU."""
import ctypes

import pytest
import torch

import moe_synth
from oracle import train_oracle as T

f64 = torch.float64


def _offsets(counts):
    return torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32)


def _rand(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed + sum(s * 31 ** i for i, s in enumerate(shape)))
    return torch.randn(*shape, generator=g, dtype=f64) * scale


def _differences(fn, t, step=1e-5):
    """Central differences of a scalar function of t, element by element."""
    out = torch.zeros_like(t)
    flat, o = t.view(-1), out.view(-1)
    for i in range(flat.numel()):
        keep = float(flat[i])
        flat[i] = keep + step
        up = float(fn())
        flat[i] = keep - step
        down = float(fn())
        flat[i] = keep
        o[i] = (up - down) / (2 * step)
    return out


def _close(a, b, tol):
    assert (a - b).abs().max().item() <= tol * max(1.0, b.abs().max().item()), (a - b).abs().max()


@pytest.mark.parametrize("rows,d", [(1, 3), (5, 17), (7, 64)])
def test_norm_gradient(rows, d):
    x, gamma, beta, dy = (_rand(rows, d), _rand(d, seed=1), _rand(d, seed=2), _rand(rows, d, seed=3))
    y, mean, rstd = T.norm(x, gamma, beta, 1e-5)
    want = torch.nn.functional.layer_norm(x, (d,), gamma, beta, 1e-5)
    _close(y, want, 1e-12)
    dx, dg, db = T.norm_backward(x, gamma, mean, rstd, dy)
    leaves = [t.clone().requires_grad_() for t in (x, gamma, beta)]
    out = torch.nn.functional.layer_norm(leaves[0], (d,), leaves[1], leaves[2], 1e-5)
    for got, ref in zip((dx, dg, db), torch.autograd.grad(out, leaves, dy)):
        _close(got, ref, 1e-11)
    loss = lambda: (T.norm(x, gamma, beta, 1e-5)[0] * dy).sum()
    _close(dx, _differences(loss, x), 1e-6)
    _close(dg, _differences(loss, gamma), 1e-7)


@pytest.mark.parametrize("act", ["swiglu", "relu"])
def test_ffn_gradient(act):
    counts, d, F = [3, 0, 1, 4], 6, 5
    off, P, E = _offsets(counts), sum(counts), len(counts)
    x, dy = _rand(P, d), _rand(P, d, seed=9)
    W1, W2 = _rand(E, F, d, seed=1), _rand(E, d, F, seed=2)
    W3 = _rand(E, F, d, seed=3) if act == "swiglu" else None
    y, g, u, h = T.ffn(x, off, W1, W3, W2)
    dx, dW1, dW3, dW2, _, _ = T.ffn_backward(x, off, W1, W3, W2, g, u, h, dy)
    leaves = [t.clone().requires_grad_() for t in (x, W1, W2) + ((W3,) if W3 is not None else ())]
    out = torch.cat([
        (torch.relu(leaves[0][a:b] @ leaves[1][e].T) if W3 is None else
         torch.nn.functional.silu(leaves[0][a:b] @ leaves[1][e].T) * (leaves[0][a:b] @ leaves[3][e].T))
        @ leaves[2][e].T for e, (a, b) in enumerate(zip(off[:-1].tolist(), off[1:].tolist()))])
    _close(y, out.detach(), 1e-12)
    got = (dx, dW1, dW2) + ((dW3,) if W3 is not None else ())
    for a, b in zip(got, torch.autograd.grad(out, leaves, dy)):
        _close(a, b, 1e-11)
    loss = lambda: (T.ffn(x, off, W1, W3, W2)[0] * dy).sum()
    for a, t in zip(got, (x, W1, W2, W3)):
        _close(a, _differences(loss, t), 1e-6)
    assert dW1[1].abs().max() == 0 and dW2[1].abs().max() == 0     # the expert without rows


def _route(x, Wg, bias, k, gate):
    probs = torch.softmax(x @ Wg.T + bias, 1)
    p, idx = torch.sort(probs, dim=1, descending=True, stable=True)
    p, idx = p[:, :k], idx[:, :k]
    return probs, idx, p / p.sum(1, keepdim=True) if gate == "renorm" else p


@pytest.mark.parametrize("gate,k,aux", [("renorm", 2, 0.0), ("renorm", 3, 0.7), ("top_prob", 1, 0.0),
                                        ("top_prob", 2, 0.4), ("renorm", 5, 0.0)])
def test_router_gradient(gate, k, aux):
    n, d, E = 6, 4, 5
    x, Wg, bias = _rand(n, d), _rand(E, d, seed=1), _rand(E, seed=2)
    dgate, dxp = _rand(n, k, seed=3), _rand(n * k, d, seed=4)
    probs, idx, gates = _route(x, Wg, bias, k, gate)
    f = torch.bincount(idx[:, 0], minlength=E).double() / n if aux else None
    inv = torch.randperm(n * k, generator=torch.Generator().manual_seed(5))
    dl = T.logits_backward(gate, probs, idx, gates, dgate, f, aux)
    dx, dWg, db = T.route_backward(dl, x, Wg, inv, dxp)
    leaves = [t.clone().requires_grad_() for t in (x, Wg, bias)]

    def loss(x, Wg, bias):
        p = torch.softmax(x @ Wg.T + bias, 1)
        c = p.gather(1, idx)
        c = c / c.sum(1, keepdim=True) if gate == "renorm" else c
        out = (c * dgate).sum() + (x.repeat_interleave(k, 0) * dxp[inv]).sum()
        return out + (aux * E * (f * p.mean(0)).sum() if aux else 0)

    for got, ref in zip((dx, dWg, db), torch.autograd.grad(loss(*leaves), leaves)):
        _close(got, ref, 1e-11)
    for got, t in zip((dx, dWg, db), (x, Wg, bias)):
        _close(got, _differences(lambda: loss(x, Wg, bias), t), 1e-6)


def test_combine_gradient():
    n, k, d = 5, 3, 4
    dy, yp, gate = _rand(n, d), _rand(n * k, d, seed=1), _rand(n, k, seed=2)
    inv = torch.randperm(n * k, generator=torch.Generator().manual_seed(6))
    a, b = yp.clone().requires_grad_(), gate.clone().requires_grad_()
    y = (b[:, :, None] * a[inv].view(n, k, d)).sum(1)
    got = T.combine_backward(dy, yp, inv, gate)
    for g, ref in zip(got, torch.autograd.grad(y, (a, b), dy)):
        _close(g, ref, 1e-12)


# ------------------------------------------------------------------- refusals
FAKE = 1 << 20          # a 256-aligned non-null address; never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_layer_moe_gb300 import build
    build.build()
    from mixture_experts_layer_moe_gb300 import moe
    return moe


def _c(lib, **kw):
    base = dict(name="t", n=16, d=64, d_ff=128, E=8, k=2, act_dtype="bf16", weight_dtype="bf16",
                gate="renorm", act="swiglu")
    base.update(kw)
    return lib.make_config(moe_synth.MoEConfig(**base))


def _ws(lib, c):
    out = ctypes.c_size_t(0)
    st = lib.raw_call("moe_train_workspace_size", ctypes.byref(c), ctypes.byref(out))
    return st, out.value


@pytest.mark.parametrize("kw,want", [
    (dict(), 0), (dict(act="relu"), 0), (dict(act_dtype="f32", weight_dtype="f32", d=4, d_ff=4), 0),
    (dict(weight_dtype="mxfp4"), 2), (dict(weight_dtype="nvfp4"), 2), (dict(n=0), 1), (dict(d=60), 2),
    (dict(E=1, k=1, n=1), 0), (dict(d_ff_shared=64), 0)])
def test_train_config_checks(lib, kw, want):
    c = _c(lib, **kw)
    st, size = _ws(lib, c)
    assert st == want, lib.status_string(st)
    if want == 0:
        fwd = ctypes.c_size_t(0)
        assert lib.raw_call("moe_workspace_size", ctypes.byref(c), ctypes.byref(fwd)) == 0
        assert size >= fwd.value


def test_ffn_refusals(lib):
    c = _c(lib)
    _, n = _ws(lib, c)
    w = lib.moe_weights(None, None, FAKE, FAKE, FAKE)
    gr = lib.moe_expert_grads(FAKE, FAKE, FAKE)

    def train(c=c, x=FAKE, off=FAKE, w=w, g=FAKE, u=FAKE, h=FAKE, y=FAKE, ws=FAKE, nb=n):
        return lib.raw_call("moe_expert_ffn_train", ctypes.byref(c), x, off, ctypes.byref(w), g, u, h,
                            y, ws, nb, None)

    def back(c=c, x=FAKE, off=FAKE, w=w, g=FAKE, u=FAKE, h=FAKE, dy=FAKE, dx=FAKE, gr=gr, ws=FAKE,
             nb=n):
        return lib.raw_call("moe_expert_ffn_backward", ctypes.byref(c), x, off, ctypes.byref(w), g, u,
                            h, dy, dx, None if gr is None else ctypes.byref(gr), ws, nb, None)

    for call in (train, back):
        for key in ("x", "off", "g", "u", "h"):
            assert call(**{key: None}) == 1, key
            assert call(**{key: FAKE + 8}) == 1, key
        assert call(ws=None) == 1 and call(ws=FAKE + 16) == 1
        assert call(nb=n - 1) == 3
        assert call(w=lib.moe_weights(None, None, FAKE, None, FAKE)) == 1     # SwiGLU without W3
        assert call(w=lib.moe_weights(None, None, FAKE, FAKE, None)) == 1
        mx = _c(lib, weight_dtype="mxfp4")
        assert call(c=mx) == 2
        relu = _c(lib, act="relu")
        assert call(c=relu, w=lib.moe_weights(None, None, FAKE, None, FAKE)) == 1   # g, u with ReLU
    assert train(y=None) == 1
    assert back(dy=None) == 1 and back(dx=FAKE + 2) == 1 and back(gr=None) == 1
    assert back(gr=lib.moe_expert_grads(FAKE + 8, None, None)) == 1
    relu = _c(lib, act="relu")
    assert back(c=relu, w=lib.moe_weights(None, None, FAKE, None, FAKE), g=None, u=None) == 1  # dW3


def test_combine_and_route_refusals(lib):
    c = _c(lib)
    _, n = _ws(lib, c)

    def comb(dy=FAKE, y=FAKE, inv=FAKE, gate=FAKE, dyp=FAKE, dg=FAKE, ws=FAKE, nb=n, c=c):
        return lib.raw_call("moe_combine_backward", ctypes.byref(c), dy, y, inv, gate, dyp, dg, ws, nb,
                            None)

    for key in ("dy", "y", "inv", "gate", "dyp", "dg"):
        assert comb(**{key: FAKE + 4}) == 1, key
        assert comb(**{key: None}) == 1, key            # y and dg: one without the other
    assert comb(nb=n - 1) == 3 and comb(ws=FAKE + 8) == 1
    w = lib.moe_weights(FAKE)

    def route(c=c, x=FAKE, w=w, p=FAKE, idx=FAKE, gate=FAKE, dg=FAKE, f=None, inv=FAKE, dxp=FAKE,
              dx=FAKE, dWg=FAKE, db=FAKE, ws=FAKE, nb=n):
        return lib.raw_call("moe_route_backward", ctypes.byref(c), x, ctypes.byref(w), p, idx, gate, dg,
                            f, 0.0, inv, dxp, dx, dWg, db, ws, nb, None)

    for key in ("x", "idx", "gate", "dg", "inv", "dxp", "dx"):
        assert route(**{key: None}) == 1, key
    for key in ("x", "p", "idx", "gate", "dg", "f", "inv", "dxp", "dx", "dWg", "db"):
        assert route(**{key: FAKE + 4}) == 1, key
    assert route(w=lib.moe_weights()) == 1 and route(nb=n - 1) == 3
    assert route(f=FAKE, p=None) == 1
    assert route(c=_c(lib, gate="top_prob"), p=None) == 1


def test_norm_refusals(lib):
    def cfg(rows=4, d=10, ldx=0, ldy=0, lddx=0, lddy=0, dtype=1, eps=1e-5, reserved=0):
        return lib.moe_norm_config(rows, ldx, ldy, lddx, lddy, d, dtype, eps, reserved)

    out = ctypes.c_size_t(0)

    def fwd(c=cfg(), x=FAKE, g=FAKE, b=FAKE, y=FAKE, m=FAKE, r=FAKE):
        return lib.raw_call("moe_layernorm", ctypes.byref(c), x, g, b, y, m, r, None)

    def back(c=cfg(), x=FAKE, g=FAKE, m=FAKE, r=FAKE, dy=FAKE, dx=FAKE, dg=FAKE, db=FAKE, ws=FAKE,
             nb=1 << 30):
        return lib.raw_call("moe_layernorm_backward", ctypes.byref(c), x, g, m, r, dy, dx, dg, db, ws,
                            nb, None)

    size = lambda c: lib.raw_call("moe_layernorm_workspace_size", ctypes.byref(c), ctypes.byref(out))
    for bad in (cfg(rows=-1), cfg(d=0), cfg(dtype=2), cfg(eps=-1.0), cfg(eps=float("nan")),
                cfg(ldx=9), cfg(ldy=9), cfg(lddx=9), cfg(lddy=9), cfg(ldx=-1), cfg(ldx=1 << 62),
                cfg(reserved=1)):
        assert size(bad) == 1 and fwd(bad) == 1 and back(bad) == 1
    assert size(cfg(ldx=10, ldy=13)) == 0
    for key in ("x", "g", "y"):
        assert fwd(**{key: None}) == 1 and fwd(**{key: FAKE + 4}) == 1
    assert fwd(m=None) == 1 and fwd(r=None) == 1 and fwd(b=FAKE + 2) == 1 and fwd(m=FAKE + 4) == 1
    for key in ("x", "g", "m", "r", "dy", "dx"):
        assert back(**{key: None}) == 1 and back(**{key: FAKE + 4}) == 1
    assert back(dg=FAKE + 4) == 1 and back(db=FAKE + 8) == 1
    assert back(ws=None) == 1 and back(ws=FAKE + 16) == 1
    big = cfg(rows=4096)
    assert size(big) == 0 and back(big, nb=0) == 3
    assert fwd(cfg(rows=0), x=None, y=None) == 0          # nothing to do, nothing launched


def test_binding_refuses_tensors_it_cannot_pass(lib):
    x = torch.zeros(4, 8)
    v, r = torch.zeros(8), torch.zeros(4)
    for bad in (dict(x=torch.zeros(8, 4).t()), dict(x=x.half()), dict(y=torch.zeros(4, 9)),
                dict(gamma=torch.zeros(7)), dict(gamma=v.bfloat16()), dict(mean=r.double())):
        a = dict(x=x, gamma=v, beta=v, y=x, mean=r, rstd=r, stream=0)
        a.update(bad)
        with pytest.raises(ValueError):
            lib.moe_layernorm(**a)
