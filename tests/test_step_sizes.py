"""Sizes that the operators round the layer state and take (no GPU needed)."""
import math

import pytest
import torch


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_layer_moe_gb300 import build
    build.build()
    from mixture_experts_layer_moe_gb300 import moe
    return moe


def _tiles(n, vocab, side):
    return math.ceil(n / side) * math.ceil(vocab / side)


# forwards and gradients that take the most, large and small, few tokens, whole and odd sizes
@pytest.mark.parametrize("n,d,vocab,dtype", [
    (0, 64, 100, "bf16"), (1, 8, 1, "bf16"), (1, 2880, 131072, "bf16"), (149, 7168, 32003, "bf16"),
    (192, 64, 2 ** 24, "bf16"), (300, 64, 200001, "bf16"), (4096, 4096, 131072, "bf16"),
    (131072, 512, 2 ** 20, "bf16"), (2 ** 20, 8, 2 ** 24, "bf16"), (471, 44688, 108510, "bf16"),
    (40, 64, 999, "bf16"), (1, 4, 1, "f32"), (5, 3640, 22803, "f32"), (8, 64, 2 ** 24, "f32"),
    (9, 64, 2 ** 24, "f32"), (256, 128, 4099, "f32"), (1000, 8, 2 ** 23 + 1, "f32"),
    (4096, 4, 2 ** 22, "f32"), (131072, 64, 2 ** 21, "f32"), (2 ** 20, 4, 2 ** 24, "f32")])
def test_cross_entropy_workspace_holds_what_is_stated(moe, n, d, vocab, dtype):
    """The parts that moe.h states, each at its most."""
    f32 = dtype == "f32"
    cores = f32 or (n * vocab * d <= 2 ** 24 and d <= 256)     # (on the CUDA cores)
    few = _tiles(n, vocab, 64) < 152 if f32 else _tiles(n, vocab, 256) < 4864
    copy = n * d * (4 if f32 else 2) + 20 * n
    sums = 8 * n * (8 if few or (cores and not f32) else 4 if f32 else 2) * math.ceil(vocab / 256)
    z = 4 if cores else 2
    piece = min(vocab, max((256 << 20) // (z * (n + 4)), 8192) + 256)
    planes = 4 if n * d >= 2 ** 24 else 152
    gradient = (n + 4) * (piece + 8) * z + planes * n * d * 4 + (40 << 20)
    got = moe.moe_cross_entropy_workspace_size(n, d, vocab, dtype)
    assert got % 256 == 0
    # (every part starts on 256 bytes)
    assert copy + 256 <= got <= copy + max(sums, gradient) + 20 * 256


@pytest.mark.parametrize("size", [2 ** 31, 2 ** 32 + 8])
def test_binding_refuses_sizes_past_32_bits(moe, monkeypatch, size):
    """Cut off to 32 bits, 2^32 + 8 would pass for 8 and most of the result stay unwritten."""
    class Lib:
        def __getattr__(self, name):
            return lambda *a: pytest.fail(f"{name} was reached")

    monkeypatch.setattr(moe, "_lib", Lib())
    meta = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="meta")
    wide, one, ws = meta(1, size), meta(1), meta(16, dtype=torch.uint8)
    rng, none = meta(2, dtype=torch.int64), moe.make_join_grads({})
    v = moe.make_join_params(dict(pre_gamma=meta(size)))
    long, t = meta(size, 8), meta(size, dtype=torch.int32)
    for call in (
            lambda: moe.moe_dropout(wide, wide, 0.1, rng, stream=0),
            lambda: moe.moe_block_join(wide, wide, v, wide, wide, None, post="none", stream=0),
            lambda: moe.moe_block_join_backward(wide, wide, meta(4, 1), v, wide, wide, wide, wide, none,
                                                ws, post="none", stream=0),
            lambda: moe.moe_block_join_workspace_size(1, size, "bf16"),
            lambda: moe.moe_cross_entropy(long, meta(5, 8), t, meta(size), meta(size), ws, stream=0),
            lambda: moe.moe_cross_entropy(meta(1, 8), long, t[:1], one, one, ws, stream=0),
            lambda: moe.moe_cross_entropy_backward(long, meta(5, 8), t, meta(size), meta(size), long,
                                                   None, ws, stream=0),
            lambda: moe.moe_cross_entropy_workspace_size(size, 8, 5, "f32"),
            lambda: moe.moe_cross_entropy_workspace_size(5, 8, size, "f32"),
            lambda: moe.alloc_cross_entropy_workspace(5, size, 5, "f32"),
            lambda: moe.moe_layernorm(wide, meta(size), None, wide, one, one, stream=0),
            lambda: moe.moe_layernorm_workspace_size(1, size, "f32")):
        with pytest.raises(ValueError, match="32 bits"):
            call()
