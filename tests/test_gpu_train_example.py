"""GPU: the training example runs every operator together and its loss falls."""
import importlib.util
import os

import pytest
import torch

import moe_synth

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from mixture_experts_layer_moe_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("train_step",
                                                  os.path.join(ROOT, "examples", "train_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["renorm", "top_prob"])
def test_loss_falls(example, dtype, gate):
    cfg = moe_synth.MoEConfig("t", 512, 128, 256, 8, 2, dtype, dtype, gate, "swiglu")
    losses = example.train(cfg, steps=30, lr=1.0)
    print(losses[0], losses[-1])
    assert losses[-1] < 0.7 * losses[0], losses


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["renorm", "top_prob"])
def test_a_whole_step_in_a_graph(example, dtype, gate):
    """Forward and backward captured on a side stream: each replay writes the eager bits, also
    after the inputs changed in place."""
    cfg = moe_synth.MoEConfig("t", 200, 136, 264, 8, 2, dtype, dtype, gate, "swiglu")
    block = example.MoEBlock(cfg, 5)
    g = torch.Generator(device="cuda").manual_seed(6)
    dt = block.xn.dtype
    draw = lambda: torch.randn(cfg.n, cfg.d, generator=g, device="cuda").to(dt)
    x, dout = draw(), draw()

    def step():
        y = block.forward(x)
        return y, block.backward(x, dout)

    def snapshot(out):
        return [t.clone() for t in (*out, *block.grad.values())]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        got = snapshot(out)
        want = snapshot(step())
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        x.copy_(draw())
        dout.copy_(draw())
