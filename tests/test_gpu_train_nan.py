"""GPU: a NaN in the rows or the weights of a ReLU layer stays visible: max(NaN, 0) is NaN on
every path (CUDA cores, SM pairs, cut reductions) and type, forward and training."""
import pytest
import torch

import test_gpu_train as base

pytestmark = pytest.mark.gpu

lib = base.lib

# n, d, F, E, k, dtype, act, counts: CUDA cores (fp32, small bf16), SM pairs, a cut reduction
CASES = [
    (83, 36, 100, 7, 2, "f32", "relu", "even"),
    (37, 72, 136, 5, 2, "bf16", "relu", "even"),
    (600, 520, 520, 3, 2, "bf16", "relu", "even"),
    (300, 1032, 264, 1, 1, "bf16", "relu", "even"),
    (7, 1096, 136, 1, 1, "bf16", "relu", "even"),
    (300, 136, 1096, 1, 1, "bf16", "relu", "even"),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_relu_keeps_nan(lib, case):
    n, d, F, E, k, dtype, act, _ = case
    s = base._ffn_inputs(case, 23)
    off = s["offsets"].tolist()
    e = max(range(E), key=lambda i: off[i + 1] - off[i])
    row = off[e] + (off[e + 1] - off[e]) // 2
    s["x"][row, d // 2] = float("nan")
    s["W1"][e, 5, d - 1] = float("nan")
    ws = lib.alloc_train_workspace(s["cfg"])
    _g, _u, h, y = base._train(lib, s, ws)
    base._ok(lib, ws)
    want = torch.zeros_like(h, dtype=torch.bool)
    want[row] = True
    want[off[e]:off[e + 1], 5] = True
    assert torch.equal(h.isnan(), want)
    # every output of the expert's rows sums over h[:, 5]
    want = torch.zeros_like(y, dtype=torch.bool)
    want[off[e]:off[e + 1]] = True
    assert torch.equal(y.isnan(), want)
    y2 = torch.empty_like(y)
    lib.moe_expert_ffn(s["cfg"], s["x"], s["offsets"], lib.make_weights(s), y2, ws)
    base._ok(lib, ws)
    assert torch.equal(y2.isnan(), want)
