"""GPU: the small-batch FFN on segment offsets that every CTA of its launch reports: the call
returns, the status says why, and the next call on the same buffers is right again."""
import pytest
import torch

import moe_synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_layer_moe_gb300 import build
    build.build()
    from mixture_experts_layer_moe_gb300 import moe
    assert torch.cuda.is_available()
    return moe


@pytest.mark.parametrize("act", ["relu", "swiglu"])
@pytest.mark.parametrize("bad", [[0, 9, 4, 12, 16, 20, 24, 28, 32], [0, 4, 8, 12, 16, 20, 24, 28, 33],
                                 [-1, 4, 8, 12, 16, 20, 24, 28, 32]])
def test_bad_offsets_of_the_small_batch_ffn(lib, bad, act):
    cfg = moe_synth.CONFIGS["gptoss_decode_mxfp4"].scaled(n=16, d=1024, d_ff=2880, E=8, k=2, act=act)
    inputs = moe_synth.make_inputs(cfg, seed=6, device="cuda")
    w = lib.make_weights(inputs)
    ws = lib.alloc_workspace(cfg)
    P = cfg.n * cfg.k
    x_perm = inputs["x"].repeat_interleave(cfg.k, 0).contiguous()
    good = torch.arange(0, P + 1, P // cfg.E, dtype=torch.int32, device="cuda")
    offsets = torch.tensor(bad, dtype=torch.int32, device="cuda")

    def run(offsets):
        y = torch.full((P, cfg.d), 3.0, dtype=torch.bfloat16, device="cuda")
        lib.moe_expert_ffn(cfg, x_perm, offsets, w, y, ws)
        return y

    want = run(good)
    assert lib.moe_status_check(ws)[0] == 0
    for _ in range(20):
        y = run(offsets)
        assert lib.moe_status_check(ws)[0] == 5
        assert (y == 3.0).all()
        y = run(good)                                   # sticky: nothing is written
        assert lib.moe_status_check(ws)[0] == 5 and (y == 3.0).all()
        lib.moe_status_clear(ws)
    assert torch.equal(run(good), want)
    assert lib.moe_status_check(ws)[0] == 0
