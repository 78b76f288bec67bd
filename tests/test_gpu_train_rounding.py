"""GPU: how often the training operators of bf16 layers round, where that differs from the
roundings of their outputs."""
import pytest
import torch

import test_gpu_train as base
from oracle import train_oracle as T

pytestmark = pytest.mark.gpu

lib = base.lib


@pytest.mark.parametrize("n,d,F,E,act", [(1, 2776, 104, 1, "swiglu"), (14, 1000, 64, 3, "swiglu"),
                                         (40, 520, 248, 2, "relu"), (5, 1096, 136, 2, "relu"),
                                         (70, 264, 120, 4, "swiglu"), (2, 8192, 16, 1, "swiglu")])
def test_ffn_backward_with_few_rows_and_a_long_reduction_rounds_once(lib, n, d, F, E, act):
    """dh = dy W2 reduces over d on the tensor cores; dg and du, which only the CUDA cores
    multiply, stay in fp32 (cut and whole reductions)."""
    base.test_ffn_backward_of_small_bf16_layers_rounds_once(lib, n, d, F, E, act)


def test_weight_gradients_of_one_token_have_one_roundings_error(lib):
    """Rounding to bf16 once is off by 2^-8 / sqrt(3) of a binade's lower end in the mean square,
    1.5e-3 to 1.7e-3 of the value over a binade; rounding an operand first makes that sqrt(2) times
    as much, 2.1e-3 or more (the sums' fp32 error is below 1e-5 of the norm here)."""
    s = base._ffn_inputs((1, 2776, 104, 1, 1, "bf16", "swiglu", "even"), 17)
    ws = lib.alloc_train_workspace(s["cfg"])
    g, u, h, _y = base._train(lib, s, ws)
    dx, gr = base._empty(s, 2776), base._grads(s)
    lib.moe_expert_ffn_backward(s["cfg"], s["x"], s["offsets"], lib.make_weights(s), g, u, h,
                                s["dy"], dx, lib.make_expert_grads(gr), ws)
    base._ok(lib, ws)
    _wdx, wW1, wW3, _wW2, _, _ = T.ffn_backward(s["x"], s["offsets"].cpu(), s["W1"], s["W3"], s["W2"],
                                                g, u, h, s["dy"])
    for got, want in ((gr["W1"], wW1), (gr["W3"], wW3)):
        off = ((got.cpu().double() - want).norm() / want.norm()).item()
        assert off <= 1.9e-3, off


# gate rule, n, d, E, k: on the tensor cores (n E d > 2^24), whole and ragged tiles
ROUTE_CASES = [("top_prob", 700, 2056, 16, 2), ("renorm", 1200, 7168, 32, 8),
               ("top_prob", 33, 5000, 128, 5), ("renorm", 4099, 2880, 64, 8)]


@pytest.mark.parametrize("gate,n,d,E,k", ROUTE_CASES)
@pytest.mark.parametrize("rows", [True, False])
def test_dx_of_the_router_is_one_sum_rounded_once(lib, gate, n, d, E, k, rows):
    """dl Wg meets the expert rows in fp32.  The probabilities and the gates' gradients are such
    that dl is a multiple of 2^-8 below 2^-1, so of 8 bits or fewer: exact in bf16 too."""
    cfg = base._cfg(n, d, 8, E, k, "bf16", gate=gate)
    g = base._gen(n + d)
    x, Wg = base._randn(g, n, d, dtype="bf16"), base._randn(g, E, d, dtype="bf16")
    dxp = base._randn(g, n * k, d, dtype="bf16", std=0.1)
    inv = torch.randperm(n * k, generator=g, device="cuda").to(torch.int32)
    idx = torch.rand(n, E, generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
    p = 1.0 / (8 if gate == "renorm" else 16)
    probs = torch.full((n, E), p, device="cuda")
    gates = torch.full((n, k), p, device="cuda")
    dgate = torch.randint(-1, 2, (n, k), generator=g, device="cuda").float()
    dl = T.logits_backward(gate, probs, idx, gates, dgate)
    assert torch.equal(dl, dl.to(torch.bfloat16).double())
    ws = lib.alloc_train_workspace(cfg)
    dx = torch.full_like(x, float("nan"))
    lib.moe_route_backward(cfg, x, lib.make_weights(dict(Wg=Wg)), probs, idx, gates, dgate, None, 0.0,
                           inv if rows else None, dxp if rows else None, dx, None, None, ws)
    base._ok(lib, ws)
    want = (dl.cuda() @ Wg.double()).cpu()
    e = 2 * E * base.V * (dl.abs().cuda() @ Wg.double().abs()).cpu()
    if rows:
        own = dxp[inv.long()].view(n, k, d).double()
        want += own.sum(1).cpu()
        e += (k + 2) * base.V * (own.abs().sum(1).cpu() + (dl.abs().cuda() @ Wg.double().abs()).cpu())
    base._within(dx, want, e + base._u("bf16") * (want.abs() + e), "dx")
