"""GPU: the ends of the operators' ranges round the layer, against the float64 oracle: rows of any
magnitude, logits far from zero.  Bounds as in test_gpu_step.py, from the arithmetic."""
import pytest
import torch

from oracle import step_oracle as S
from test_gpu_step import (DT, V, _check_join, _check_join_backward, _gen, _join_case, _ok, _randn,
                           _rows, _within)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_layer_moe_gb300 import build
    build.build()
    from mixture_experts_layer_moe_gb300 import moe
    assert torch.cuda.is_available()
    return moe


# -------------------------------------------------- block joint, rows of any magnitude
def _scaled_join_case(rows, d, pad, dtype, post, pre, size):
    """A joint whose rows x, b and r are of this size, and whose gradient dr is of the size of the
    pre norm's, 1 / size."""
    params, x, b, dr, dy, kw = _join_case(rows, d, pad, dtype, post, pre, True, 0.2, 0.75, seed=5)
    if post != "none":
        params["gate"] = params["gate"] * size
    x, b = (_rows(t * size, pad) for t in (x, b))
    return params, x, b, _rows(dr / size, pad), dy, kw


def _check_both(lib, case, eps, pad, dtype):
    params, x, b, dr, dy, kw = case
    r, stats = _check_join(lib, (params, x, b, dr, dy, dict(kw, eps=eps)), pad, dtype)
    _check_join_backward(lib, case, r, stats, pad, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,pad", [(96, 0), (1024, 0), (1001, 3), (4104, 0), (9000, 0)])
@pytest.mark.parametrize("post,pre", [("none", "rms"), ("rms", "rms"), ("layer", "layer"),
                                      ("rms", "none"), ("none", "layer")])
@pytest.mark.parametrize("size,eps", [(1e-16, 0.0), (1e-13, 0.0), (1e12, 1e-5), (1e15, 1e-5),
                                      (1e17, 1e-5)])
def test_join_of_rows_of_any_size(lib, size, eps, post, pre, d, pad, dtype):
    case = _scaled_join_case(19, d, pad, dtype, post, pre, size)
    _check_both(lib, case, eps, pad, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [96, 1001, 9000])
@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("none", "rms"), ("none", "layer")])
def test_join_of_rows_of_zeros_and_a_tiny_eps(lib, post, pre, d, dtype):
    """1 / deviation is 1e15 there: the gradient is finite, in the vectors' too."""
    params, x, b, dr, dy, kw = _join_case(11, d, 0, dtype, post, pre, True, 0.2, 1.0, beta=False)
    x[4], b[4] = 0, 0
    _check_both(lib, (params, x, b, dr, dy, kw), 1e-30, 0, dtype)


# ------------------------------------------------- cross entropy, logits far from zero
# n, d, vocab, dtype: each kernel that forms a token's sums: streams; the CUDA cores' tiles of 32
# and 64; SM pairs, with one block of tokens and several, in one unit and more
FORWARDS = [(3, 64, 4000, "bf16"), (8, 64, 4000, "f32"), (40, 64, 999, "bf16"), (40, 64, 999, "f32"),
            (1000, 64, 4000, "f32"), (40, 512, 4000, "bf16"), (40, 2048, 999, "bf16"),
            (300, 512, 4000, "bf16"), (300, 2048, 999, "bf16")]


@pytest.mark.parametrize("n,d,vocab,dtype", FORWARDS)
def test_cross_entropy_of_a_sure_token_far_from_zero(lib, n, d, vocab, dtype):
    """Logits c - gap, exact in fp32, with one entry at the top and the others 13 and more below: the
    loss is about the others' sum of exponentials, whatever c, and never negative."""
    g = _gen(n + vocab)
    top = 7 * n % vocab
    gap = (104 + torch.randint(148, (vocab,), generator=g, device="cuda")) / 8
    gap[top] = 0
    W, x = torch.zeros(vocab, d, device="cuda"), torch.zeros(n, d, device="cuda")
    W[:, 0], W[:, d - 1] = 23.25, -gap
    x[:, 0] = torch.tensor([128.0, 0.0, -128.0, 1024.0, 16.0], device="cuda").repeat(n)[:n]
    x[:, d - 1] = 1
    W, x = W.to(DT[dtype]), x.to(DT[dtype])
    t = torch.full((n,), top, dtype=torch.int32, device="cuda")
    t[2::3] = torch.arange(len(t[2::3]), device="cuda").to(torch.int32) % vocab
    ws = lib.alloc_cross_entropy_workspace(n, d, vocab, dtype)
    ws[256:] = 0xFF
    loss, lse = (torch.full((n,), float("nan"), device="cuda") for _ in range(2))
    lib.moe_cross_entropy(x, W, t, loss, lse, ws)
    _ok(lib, ws)
    wloss, wlse, logits = S.cross_entropy(x, W, t)
    below = logits.amax(1, keepdim=True) - logits
    # the exponentials but for the top's, which is 1; the fp32 sum; the logarithm and the last sums
    e = ((torch.softmax(logits, 1) * (2 ** -20 + 2 ** -22 * below) * (below > 0)).sum(1)
         + (64 + vocab / 8192) * V)
    at = below.gather(1, t.cpu().long()[:, None])[:, 0]
    _within(loss, wloss, e + 4 * V * (at + wloss), "loss")
    _within(lse, wlse, e + 2 * V * wlse.abs(), "lse")
    assert (loss >= 0).all()


# ------------------------------------------------------------------------- workspaces
@pytest.mark.parametrize("n,d,vocab,dtype", [(4096, 4, 2 ** 22 + 5, "f32"), (1000, 64, 4001, "f32"),
                                             (70, 64, 3001, "f32"), (1000, 64, 4001, "bf16"),
                                             (40, 64, 999, "bf16"), (3, 64, 4001, "f32")])
def test_cross_entropy_stays_in_its_workspace(lib, n, d, vocab, dtype):
    """What lies behind a workspace of the stated size stays, and the sums in it are whole."""
    g = _gen(n + d)
    x, W = _randn(g, n, d, dtype=dtype), _randn(g, vocab, d, dtype=dtype, std=d ** -0.5)
    t = torch.randint(vocab, (n,), generator=g, device="cuda").to(torch.int32)
    size = lib.moe_cross_entropy_workspace_size(n, d, vocab, dtype)
    space = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = space[:size]
    ws[:256] = 0
    loss, lse = (torch.full((n,), float("nan"), device="cuda") for _ in range(2))
    lib.moe_cross_entropy(x, W, t, loss, lse, ws)
    dx, dW = torch.full_like(x, float("nan")), torch.full_like(W, float("nan"))
    lib.moe_cross_entropy_backward(x, W, t, lse, torch.ones_like(lse), dx, dW, ws)
    _ok(lib, ws)
    assert (space[size:] == 0xA5).all()
    assert all(torch.isfinite(v).all() for v in (loss, dx, dW))
    some = torch.arange(0, n, max(1, n // 8), device="cuda")
    logits = x[some].double() @ W.double().T
    want, top = torch.logsumexp(logits, 1), logits.amax(1)
    # |l| <= |x| |W| (norms); exponents of at most the logits' range; the sum; the last roundings
    k = 2 if dtype == "bf16" else 1
    e = (k * d * V * x[some].double().norm(dim=1) * W.double().norm(dim=1).max() + 2 ** -20
         + 2 ** -22 * (top - logits.amin(1)) + (64 + vocab / 8192) * V + 2 * V * (want.abs() + top.abs()))
    assert ((lse[some].double() - want).abs() <= e).all()
