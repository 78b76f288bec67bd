"""The float64 oracle of dropout, the block joint and the cross entropy: published generator
vectors, gradients against autograd and against differences."""
import itertools

import numpy as np
import pytest
import torch

from oracle import step_oracle as S

NORMS = ("none", "rms", "layer")


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     "d16cfe09 94fdcceb 5001e420 24126ea1")])
def test_philox_known_answers(counter, key, want):
    """The known-answer vectors that the generator's authors publish for philox4x32, 10 rounds."""
    got = " ".join(f"{int(v):08x}" for v in S.philox4x32_10(counter, key))
    assert got == want


def test_keep_follows_the_place_alone():
    a = S.keep(5, 9, 40, 77, 0.3)
    assert torch.equal(a[:, :16], S.keep(5, 9, 40, 16, 0.3))
    assert torch.equal(a[:7], S.keep(5, 9, 7, 77, 0.3))
    assert not torch.equal(a, S.keep(5, 10, 40, 77, 0.3))
    assert not torch.equal(a, S.keep(6, 9, 40, 77, 0.3))
    # a row's elements are no shifted copy of the next one's
    assert all((a[0] ^ a[i]).any() for i in range(1, 40))


@pytest.mark.parametrize("p", [0.0, 1e-5, 0.1, 0.5, 0.99])
def test_keep_share(p):
    """A binomial share: within six deviations."""
    q = S.threshold(p) / 65536
    k = S.keep(2 ** 63 + 11, 2 ** 40 + 3, 300, 1000, p).double()
    assert abs(k.mean().item() - (1 - q)) <= 6 * np.sqrt(q * (1 - q) / k.numel())


def _case(post, pre, gate, p, seed=0, n=5, d=12):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    params = {}
    if gate:
        params["gate"] = rnd(d)
    for side, kind in (("post", post), ("pre", pre)):
        if kind != "none":
            params[side + "_gamma"] = rnd(d)
        if kind == "layer":
            params[side + "_beta"] = rnd(d)
    rng = torch.tensor([3, 4])
    kw = dict(post=post, pre=pre, scale=0.75, p=p, rng=rng)
    return rnd(n, d), rnd(n, d), params, rnd(n, d), rnd(n, d), kw


def _autograd(x, b, params, dr, dy, post, pre, scale, p, rng, eps=1e-5):
    leaves = {k: v.clone().requires_grad_() for k, v in dict(x=x, b=b, **params).items()}

    def norm(v, kind, side):
        if kind == "none":
            return v
        if kind == "layer":
            v = v - v.mean(1, keepdim=True)
        v = v / torch.sqrt(v.square().mean(1, keepdim=True) + eps) * leaves[side + "_gamma"]
        return v + leaves[side + "_beta"] if kind == "layer" else v

    z = norm(leaves["b"], post, "post") * S.factors(rng, *x.shape, p)
    r = scale * leaves["x"] + (z * leaves["gate"] if "gate" in params else z)
    total = (r * dr).sum()
    if pre != "none":
        total = total + (norm(r, pre, "pre") * dy).sum()
    total.backward()
    return {k: v.grad for k, v in leaves.items()}, total


@pytest.mark.parametrize("post,pre,gate,p",
                         list(itertools.product(NORMS, NORMS, (False, True), (0.0, 0.4))))
def test_join_gradient_against_autograd(post, pre, gate, p):
    x, b, params, dr, dy, kw = _case(post, pre, gate, p)
    r, y, stats, _ = S.join(x, b, params, **kw)
    want, total = _autograd(x, b, params, dr, dy, **kw)
    given = dy if pre != "none" else None
    assert torch.allclose(total, (r * dr).sum() + (0 if y is None else (y * dy).sum()))
    dx, db, g = S.join_backward(b, r, stats, params, dr, given, **kw)
    for name, got in (("x", dx), ("b", db), *((k, g[k]) for k in params)):
        assert torch.allclose(got, want[name], rtol=1e-9, atol=1e-10), name


@pytest.mark.parametrize("post,pre", [("rms", "layer"), ("layer", "rms"), ("none", "rms")])
def test_join_gradient_against_differences(post, pre):
    x, b, params, dr, dy, kw = _case(post, pre, True, 0.3, seed=1)
    r, _, stats, _ = S.join(x, b, params, **kw)
    dx, db, g = S.join_backward(b, r, stats, params, dr, dy, **kw)

    def value(x, b, params):
        r, y, _, _ = S.join(x, b, params, **kw)
        return ((r * dr).sum() + (y * dy).sum()).item()

    h = 1e-5
    gen = torch.Generator().manual_seed(2)
    for name, grad in (("x", dx), ("b", db), *g.items()):
        base = dict(x=x, b=b, params=params)
        if name not in ("x", "b") and name not in params:
            continue
        step = torch.randn(grad.shape, generator=gen, dtype=torch.float64)
        ends = []
        for sign in (1, -1):
            moved = dict(base, params=dict(params))
            if name in ("x", "b"):
                moved[name] = base[name] + sign * h * step
            else:
                moved["params"][name] = params[name] + sign * h * step
            ends.append(value(**moved))
        # the difference is off by the third derivative times h^2
        assert abs((ends[0] - ends[1]) / (2 * h) - (grad * step).sum().item()) < 1e-6, name


@pytest.mark.parametrize("z_loss", [0.0, 0.02])
def test_cross_entropy_gradient(z_loss):
    g = torch.Generator().manual_seed(4)
    x = torch.randn(7, 6, generator=g, dtype=torch.float64, requires_grad=True)
    W = torch.randn(11, 6, generator=g, dtype=torch.float64, requires_grad=True)
    t = torch.tensor([3, -1, 10, 0, 3, -100, 7], dtype=torch.int32)
    dloss = torch.randn(7, generator=g, dtype=torch.float64)
    loss, lse, _ = S.cross_entropy(x, W, t, z_loss)
    assert loss[1] == 0 and loss[5] == 0 and lse[1] == 0
    counted = t >= 0
    logits = x @ W.T
    want = (torch.nn.functional.cross_entropy(logits[counted], t[counted].long(), reduction="none")
            + z_loss * torch.logsumexp(logits[counted], 1) ** 2)
    assert torch.allclose(loss[counted], want)
    (want * dloss[counted]).sum().backward()
    dx, dW, dl = S.cross_entropy_backward(x, W, t, lse, dloss, z_loss)
    assert torch.allclose(dx, x.grad) and torch.allclose(dW, W.grad)
    assert dx[1].abs().max() == 0 and dl[5].abs().max() == 0
    # against differences of the loss
    step, h = torch.randn(11, 6, generator=g, dtype=torch.float64), 1e-5
    ends = [(S.cross_entropy(x, W + s * h * step, t, z_loss)[0] * dloss).sum().item() for s in (1, -1)]
    assert abs((ends[0] - ends[1]) / (2 * h) - (dW * step).sum().item()) < 1e-7
