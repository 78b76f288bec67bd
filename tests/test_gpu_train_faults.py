"""GPU: the training operators on inputs that they have to survive: indexes out of range that
many CTAs meet at once."""
import pytest
import torch

import test_gpu_train as base
from oracle import train_oracle as T

pytestmark = pytest.mark.gpu

lib = base.lib
V, DT = base.V, base.DT


def _routing(n, d, E, k, dtype, seed, gate="renorm"):
    """What a forward pass leaves for moe_route_backward."""
    g = base._gen(seed)
    s = dict(x=base._randn(g, n, d, dtype=dtype), Wg=base._randn(g, E, d, dtype=dtype, std=0.1),
             probs=torch.softmax(base._randn(g, n, E, std=1.5), 1), dgate=base._randn(g, n, k),
             inv=torch.randperm(n * k, generator=g, device="cuda").to(torch.int32),
             dxp=base._randn(g, n * k, d, dtype=dtype))
    p, idx = torch.sort(s["probs"], dim=1, descending=True, stable=True)
    p, s["idx"] = p[:, :k].contiguous(), idx[:, :k].to(torch.int32).contiguous()
    s["gates"] = (p / p.sum(1, keepdim=True) if gate == "renorm" else p).contiguous()
    return s


def _sparse_dx_bound(s, dl, wdx):
    """Error bound of dx where it is one fp32 sum over the token's choices, rounded once
    (route_rows_kernel): a choice's coefficient is off by (k + 4) v of its terms."""
    n, k = s["gates"].shape
    a = {key: s[key].cpu().double().abs() for key in ("gates", "dgate", "Wg", "dxp")}
    total = (a["gates"] * a["dgate"]).sum(1, keepdim=True)
    idx, inv = s["idx"].cpu().long(), s["inv"].cpu().long().view(n, k)
    coef = a["gates"] * (a["dgate"] + total)
    terms = torch.zeros_like(wdx)
    for j in range(k):
        ok = (idx[:, j] >= 0) & (idx[:, j] < s["Wg"].shape[0])
        terms[ok] += coef[ok, j:j + 1] * a["Wg"][idx[ok, j]]
        ok = (inv[:, j] >= 0) & (inv[:, j] < n * k)
        terms[ok] += a["dxp"][inv[ok, j]]
    u = torch.finfo(s["x"].dtype).eps / 2
    e = (3 * k + 8) * V * terms
    return e + u * (wdx.abs() + e)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d,k", [(5000, 2880, 2), (20000, 264, 3)])
def test_route_backward_with_many_bad_indexes(lib, n, d, k, dtype):
    """The fault is recorded while other CTAs of the launch start: each element of dx is right
    or as it was, whichever threads of a CTA saw the status word change."""
    E = 16
    cfg = base._cfg(n, d, 8, E, k, dtype)
    s = _routing(n, d, E, k, dtype, n + d)
    s["idx"][5::97, 0] = E + 7
    s["idx"][11::101, k - 1] = -3
    s["inv"][::131 * k] = n * k
    s["inv"][7::137] = -2
    ws = lib.alloc_train_workspace(cfg)
    w = lib.make_weights(s)
    dl = T.logits_backward("renorm", E, s["idx"], s["gates"], s["dgate"])
    wdx, _, _ = T.route_backward(dl, s["x"], s["Wg"], s["inv"], s["dxp"])
    bound = _sparse_dx_bound(s, dl, wdx)
    for _ in range(20):
        dx = torch.full_like(s["x"], 77.0)
        lib.moe_route_backward(cfg, s["x"], w, None, s["idx"], s["gates"], s["dgate"], None, 0.0,
                               s["inv"], s["dxp"], dx, None, None, ws)
        assert lib.moe_status_check(ws)[0] == 5
        lib.moe_status_clear(ws)
        got = dx.cpu().double()
        right = (got - wdx).abs() <= bound + base.TINY
        assert (right | (got == 77.0)).all()
        assert right.any()


@pytest.mark.parametrize("n,d,E,k", [(700, 2056, 16, 2), (3000, 1032, 40, 8), (200, 128, 8, 3)])
def test_route_backward_of_a_dense_gradient_reports_bad_rows(lib, n, d, E, k):
    """The product that adds the gathered rows skips indexes outside them; the status says so, and
    the next call after the status was cleared is right."""
    cfg = base._cfg(n, d, 8, E, k, "bf16", gate="top_prob")
    s = _routing(n, d, E, k, "bf16", 3, "top_prob")
    ws, w = lib.alloc_train_workspace(cfg), lib.make_weights(s)

    def run(inv):
        dx = torch.full_like(s["x"], 77.0)
        lib.moe_route_backward(cfg, s["x"], w, s["probs"], s["idx"], s["gates"], s["dgate"], None, 0.0,
                               inv, s["dxp"], dx, None, None, ws)
        return dx

    want = run(s["inv"])
    base._ok(lib, ws)
    assert not (want == 77.0).any()
    for at, bad in ((0, -1), (n * k - 1, n * k), (n * k // 2, 2 ** 31 - 1), (7, -2 ** 31)):
        inv = s["inv"].clone()
        inv[at] = bad
        run(inv)
        assert lib.moe_status_check(ws) == (5, at)
        lib.moe_status_clear(ws)
    assert torch.equal(run(s["inv"]), want)
    base._ok(lib, ws)
