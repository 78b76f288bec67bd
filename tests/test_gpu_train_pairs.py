"""GPU: the tensor-core paths of the training operators on the inputs that
tests/test_gpu_train.py tries on layers small enough for the CUDA cores: segments with NaN and
infinity beside others, offsets that are wrong, rows outside the segments.  And the router's sum
over few choices for rows of more than one CTA's width."""
import pytest
import torch

import test_gpu_train as base
import test_gpu_train_faults as faults
from oracle import train_oracle as T

pytestmark = pytest.mark.gpu

lib = base.lib

# (a layer's reduction above 256 and its weights above 2^19 elements, or its products above 2^24:
# none of its products runs on the CUDA cores)
TAILS = [70, 1, 15, 130, 17, 63, 5, 50]
WIDE = [300, 1, 15, 430, 17, 63, 305, 250]
RUNS = [2061, 17, 2122]
# name: d, F, counts, the segments that go bad
LAYERS = {
    # launches in pairs on shares of the SMs
    "side_by_side": (520, 520, TAILS, (1, 4, 5)),
    "one_after_the_other": (520, 520, WIDE, (1, 4, 5)),
    # the weight gradients' rows in runs
    "runs": (72, 136, RUNS, (1,)),
    # the row products' reductions in ranges (of the up projection and dh, and of the others)
    "cut_over_d": (2104, 520, [20, 1, 13], (1,)),
    "cut_over_d_ff": (520, 2104, [20, 1, 13], (1,)),
}


def _layer(name, act, seed=29):
    d, F, counts, bad = LAYERS[name]
    return base._ffn_inputs((sum(counts), d, F, len(counts), 1, "bf16", act, counts), seed), bad


def _back(lib, s, ws, g, u, h, fill=float("nan")):
    dx, gr = base._empty(s, s["x"].shape[1], fill), base._grads(s)
    lib.moe_expert_ffn_backward(s["cfg"], s["x"], s["offsets"], lib.make_weights(s), g, u, h, s["dy"],
                                dx, lib.make_expert_grads(gr), ws)
    return dx, [t for t in gr.values() if t is not None]


@pytest.mark.parametrize("act", ["swiglu", "relu"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", list(LAYERS))
def test_experts_stay_apart(lib, name, bad, act):
    s, spoilt = _layer(name, act)
    ws = lib.alloc_train_workspace(s["cfg"])
    off = s["offsets"].tolist()

    def run():
        g, u, h, y = base._train(lib, s, ws)
        dx, gr = _back(lib, s, ws, g, u, h)
        base._ok(lib, ws)
        return [y, dx], gr

    rows0, w0 = run()
    assert all(torch.isfinite(t).all() for t in (*rows0, *w0))
    for e in spoilt:
        for key in ("x", "dy"):
            s[key][off[e]:off[e + 1]] = bad
    rows1, w1 = run()
    for e in range(len(off) - 1):
        for which, p, q in zip(("y", "dx"), rows0, rows1):
            p, q = p[off[e]:off[e + 1]], q[off[e]:off[e + 1]]
            if e not in spoilt:
                assert torch.equal(p, q)
            elif which == "y" or act == "swiglu":      # (ReLU: dg = 0 where h > 0 does not hold)
                assert not torch.isfinite(q).all()
        for p, q in zip(w0, w1):
            assert torch.equal(p[e], q[e]) if e not in spoilt else not torch.isfinite(q[e]).all()


@pytest.mark.parametrize("act", ["swiglu", "relu"])
@pytest.mark.parametrize("name", list(LAYERS))
def test_rows_outside_the_segments_stay(lib, name, act):
    """Offsets that begin after the first row and end before the last."""
    s, _ = _layer(name, act)
    F, d = s["W1"].shape[1], s["x"].shape[1]
    P = s["x"].shape[0]
    first, last = 3, P - 6
    s["offsets"] = s["offsets"].clamp(first, last)
    for key in ("x", "dy"):
        s[key][:first] = float("nan")
        s[key][last:] = float("nan")
    ws = lib.alloc_train_workspace(s["cfg"])
    ws[256:] = 255                                       # (NaN wherever scratch is not written)
    gated = act == "swiglu"
    g, u = (base._empty(s, F, 5.0) for _ in range(2)) if gated else (None, None)
    h, y = base._empty(s, F, 5.0), base._empty(s, d, 5.0)
    lib.moe_expert_ffn_train(s["cfg"], s["x"], s["offsets"], lib.make_weights(s), g, u, h, y, ws)
    dx, gr = _back(lib, s, ws, g, u, h, 5.0)
    base._ok(lib, ws)
    for t in (g, u, h, y, dx):
        if t is not None:
            assert (t[:first] == 5.0).all() and (t[last:] == 5.0).all()
            assert torch.isfinite(t[first:last]).all()
    for t in gr:
        assert torch.isfinite(t).all()


def _wrong(off, P):
    """Offsets that go back, end past the rows, begin before them."""
    back, past, before = list(off), list(off), list(off)
    back[1], back[2] = off[2] + 3, off[1]
    past[-1] = P + 1
    before[0] = -1
    return [back, past, before]


@pytest.mark.parametrize("act", ["swiglu", "relu"])
@pytest.mark.parametrize("name", list(LAYERS))
@pytest.mark.parametrize("which", range(3))
def test_wrong_offsets_are_reported(lib, name, act, which):
    s, _ = _layer(name, act)
    ws = lib.alloc_train_workspace(s["cfg"])
    good = s["offsets"]
    g, u, h, y0 = base._train(lib, s, ws)
    dx0, gr0 = _back(lib, s, ws, g, u, h)
    base._ok(lib, ws)
    s["offsets"] = torch.tensor(_wrong(good.tolist(), s["x"].shape[0])[which], dtype=torch.int32,
                                device="cuda")
    *_, h1, y1 = base._train(lib, s, ws)
    assert lib.moe_status_check(ws)[0] == 5
    assert h1.isnan().all() and y1.isnan().all()         # nothing was written
    lib.moe_status_clear(ws)
    dx1, gr1 = _back(lib, s, ws, g, u, h)
    assert lib.moe_status_check(ws)[0] == 5
    assert all(t.isnan().all() for t in (dx1, *gr1))
    lib.moe_status_clear(ws)
    s["offsets"] = good
    *_, y2 = base._train(lib, s, ws)
    dx2, gr2 = _back(lib, s, ws, g, u, h)
    base._ok(lib, ws)
    for a, b in zip((y0, dx0, *gr0), (y2, dx2, *gr2)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d,k", [(1, 7168, 1), (3, 2056, 3), (400, 7168, 2), (330, 2880, 4), (310, 4104, 1)])
@pytest.mark.parametrize("rows", [True, False])
def test_router_sum_over_few_choices_of_wide_rows(lib, n, d, k, dtype, rows):
    """One and two vectors per thread, and several CTAs per token."""
    E = 24
    s = faults._routing(n, d, E, k, dtype, n + d + k)
    cfg = base._cfg(n, d, 8, E, k, dtype)
    ws = lib.alloc_train_workspace(cfg)
    dx = torch.full_like(s["x"], float("nan"))
    lib.moe_route_backward(cfg, s["x"], lib.make_weights(s), None, s["idx"], s["gates"], s["dgate"],
                           None, 0.0, s["inv"] if rows else None, s["dxp"] if rows else None, dx, None,
                           None, ws)
    base._ok(lib, ws)
    dl = T.logits_backward("renorm", E, s["idx"], s["gates"], s["dgate"])
    want, _, _ = T.route_backward(dl, s["x"], s["Wg"], *((s["inv"], s["dxp"]) if rows else ()))
    base._within(dx, want, faults._sparse_dx_bound(s, dl, want), "dx")


@pytest.mark.parametrize("n,d,E,k,gate,aux", [(40, 8200, 64, 40, "renorm", 0.1),
                                              (10, 14336, 256, 8, "top_prob", 0.0),
                                              (300, 264, 256, 17, "renorm", 0.0),
                                              (129, 7168, 32, 1, "top_prob", 0.2),
                                              (1000, 2880, 128, 4, "renorm", 0.1),
                                              (1100, 72, 250, 250, "top_prob", 0.0)])
def test_route_backward_with_the_rows_in_the_products_epilogue(lib, n, d, E, k, gate, aux):
    """Tiles of 64 to 256 columns, one choice to every expert, ragged last rows and columns."""
    base.test_route_backward(lib, n, d, E, k, "bf16", gate, aux)


def test_router_product_with_rows_in_a_graph(lib):
    """Back to back, each call's inputs overwritten at once, and captured: the bits of one call."""
    n, d, E, k = 700, 2056, 16, 2
    cfg = base._cfg(n, d, 8, E, k, "bf16", gate="top_prob")
    s = [faults._routing(n, d, E, k, "bf16", seed, "top_prob") for seed in (1, 2)]
    ws, now = lib.alloc_train_workspace(cfg), {key: t.clone() for key, t in s[0].items()}
    w = lib.make_weights(now)
    dx, dWg, db = torch.empty_like(now["x"]), torch.empty_like(now["Wg"]), torch.empty(E, device="cuda")

    def call(inputs, stream=None):
        for key, t in inputs.items():
            now[key].copy_(t)
        lib.moe_route_backward(cfg, now["x"], w, now["probs"], now["idx"], now["gates"], now["dgate"],
                               None, 0.0, now["inv"], now["dxp"], dx, dWg, db, ws, stream=stream)
        return [t.clone() for t in (dx, dWg, db)]

    want = []
    for inputs in s:
        torch.cuda.synchronize()
        want.append(call(inputs))
        base._ok(lib, ws)
    got = [call(s[i % 2]) for i in range(12)]
    base._ok(lib, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kept = [call(inputs, side) for inputs in s]
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    base._ok(lib, ws)
    for i, ts in enumerate(got + kept):
        for a, b in zip(ts, want[i % 2]):
            assert torch.equal(a, b), i
