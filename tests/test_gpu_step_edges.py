"""GPU: the ends of the operators' ranges round the layer, against the float64 oracle: rows of any
magnitude.  Bounds as in test_gpu_step.py, from the arithmetic."""
import pytest
import torch

from test_gpu_step import _check_join, _check_join_backward, _join_case, _rows

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
