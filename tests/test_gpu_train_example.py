"""GPU: the training example runs every operator together and its loss falls."""
import importlib.util
import os

import pytest

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
