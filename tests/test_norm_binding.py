"""The layer norm's binding refuses rows that share memory before it calls the library (no GPU
needed: the tensors lie on the host and nothing is launched)."""
import pytest
import torch


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_layer_moe_gb300 import build
    build.build()
    from mixture_experts_layer_moe_gb300 import moe
    return moe


@pytest.fixture()
def calls(moe, monkeypatch):
    """The leading dimensions that reach the library, whose entry points do nothing here."""
    seen = []

    class Lib:
        @staticmethod
        def moe_layernorm(cfg, *a):
            seen.append((cfg._obj.ldx, cfg._obj.ldy))
            return 0

        @staticmethod
        def moe_layernorm_backward(cfg, *a):
            seen.append((cfg._obj.ldx, cfg._obj.lddy, cfg._obj.lddx))
            return 0

    monkeypatch.setattr(moe, "_lib", Lib)
    return seen


def _forward(moe, x, y, d):
    v = torch.ones(d)
    moe.moe_layernorm(x, v, None, y, None, None, stream=0)


def _backward(moe, x, dy, dx, d):
    v, r = torch.ones(d), torch.ones(x.shape[0])
    moe.moe_layernorm_backward(x, v, r, r, dy, dx, None, None, torch.empty(0, dtype=torch.uint8),
                               stream=0)


# one row expanded, one column expanded, windows that slide by less than a row
SHARED = [(lambda: torch.zeros(64).expand(4, 64), 64), (lambda: torch.zeros(1).expand(4, 1), 1),
          (lambda: torch.zeros(1, 1).expand(5, 1), 1),
          (lambda: torch.zeros(67).as_strided((4, 64), (1, 1)), 64),
          (lambda: torch.zeros(67 * 4).as_strided((4, 64), (63, 1)), 64)]


@pytest.mark.parametrize("make,d", SHARED)
def test_rows_that_share_memory_are_refused(moe, calls, make, d):
    bad = make()
    good = torch.zeros(bad.shape[0], d)
    for x, y in ((bad, good), (good, bad)):
        with pytest.raises(ValueError):
            _forward(moe, x, y, d)
    for x, dy, dx in ((bad, good, good), (good, bad, good), (good, good, bad)):
        with pytest.raises(ValueError):
            _backward(moe, x, dy, dx, d)
    assert calls == []


def test_rows_of_their_own_are_passed(moe, calls):
    wide = torch.zeros(4, 67)[:, :64]
    _forward(moe, wide, torch.zeros(4, 64), 64)
    _backward(moe, wide, torch.zeros(4, 64), torch.zeros(4, 65)[:, :64], 64)
    # a single row meets no other: an expanded one is a row like any
    _forward(moe, torch.zeros(64).expand(1, 64), torch.zeros(1, 64), 64)
    _backward(moe, torch.zeros(4, 1), torch.zeros(4, 3)[:, 1:2], torch.zeros(4, 1), 1)
    assert calls == [(67, 64), (67, 64, 65), (64, 64), (1, 3, 1)]
