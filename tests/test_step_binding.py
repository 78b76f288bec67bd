"""What the entry points round the layer refuse before anything is launched: dropout, the block
joint and the cross entropy (no GPU needed)."""
import ctypes

import pytest
import torch

FAKE = 1 << 20          # a 256-aligned non-null address; never dereferenced on the host
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_layer_moe_gb300 import build
    build.build()
    from mixture_experts_layer_moe_gb300 import moe
    return moe


# -------------------------------------------------------------- the C entries
def _dropout(moe, x=FAKE, rng=FAKE, y=FAKE, **kw):
    c = moe.moe_dropout_config(**{**dict(rows=4, d=64, dtype=1, p=0.1), **kw})
    return moe.raw_call("moe_dropout", ctypes.byref(c), x, rng, y, None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(rows=2 ** 32 + 1), UNSUPPORTED), (dict(d=0), INVALID),
    (dict(d=2 ** 30 + 1), UNSUPPORTED), (dict(d=2 ** 31 - 1), UNSUPPORTED),
    (dict(dtype=2), INVALID), (dict(reserved=1), INVALID), (dict(p=-0.1), INVALID),
    (dict(p=1.0), INVALID), (dict(p=0.999999), INVALID), (dict(p=float("nan")), INVALID),
    (dict(ldx=63), INVALID), (dict(ldy=1), INVALID), (dict(ldx=2 ** 62), INVALID),
    (dict(x=None), INVALID), (dict(x=FAKE + 4), INVALID), (dict(y=None), INVALID),
    (dict(y=FAKE + 8), INVALID), (dict(rng=None), INVALID), (dict(rng=FAKE + 4), INVALID),
    (dict(ldx=80), INVALID),        # (y is x, with rows of another distance)
])
def test_dropout_refuses(moe, kw, want):
    assert _dropout(moe, **kw) == want


def test_dropout_of_no_rows(moe):
    assert _dropout(moe, rows=0, x=None, y=None) == 0


def _params(moe, post=1, pre=1, **kw):
    given = dict(gate=None, post_gamma=FAKE if post else None, pre_gamma=FAKE if pre else None)
    return moe.moe_join_params(**{**given, **kw})


def _join(moe, x=FAKE, b=FAKE, rng=None, r=2 * FAKE, y=FAKE, stats=None, vectors={}, **kw):
    c = moe.moe_join_config(**{**dict(rows=4, d=64, dtype=1, post=1, pre=1, eps=1e-5, scale=1.0),
                               **kw})
    w = _params(moe, c.post, c.pre, **vectors)
    return moe.raw_call("moe_block_join", ctypes.byref(c), x, b, ctypes.byref(w), rng, r, y, stats,
                        None)


JOIN_CONFIGS = [
    (dict(rows=-1), INVALID), (dict(rows=2 ** 32 + 1), UNSUPPORTED), (dict(d=0), INVALID),
    (dict(d=2 ** 30 + 1), UNSUPPORTED), (dict(d=2 ** 31 - 1), UNSUPPORTED),
    (dict(dtype=2), INVALID), (dict(reserved=1), INVALID), (dict(post=3), INVALID),
    (dict(pre=-1), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(dropout=1.0), INVALID),
    (dict(dropout=-1.0), INVALID), (dict(dropout=0.5), INVALID),   # (no generator state)
    (dict(vectors=dict(post_gamma=None)), INVALID), (dict(vectors=dict(pre_gamma=None)), INVALID),
    (dict(vectors=dict(post_beta=FAKE)), INVALID), (dict(vectors=dict(pre_beta=FAKE)), INVALID),
    (dict(vectors=dict(gate=FAKE + 2)), INVALID),
    (dict(post=0, vectors=dict(post_gamma=FAKE)), INVALID),
    (dict(post=2, vectors=dict(post_beta=FAKE + 8)), INVALID),
    (dict(rng=FAKE + 4), INVALID), (dict(stats=FAKE + 4), INVALID),
]


@pytest.mark.parametrize("kw,want", JOIN_CONFIGS + [
    (dict(ldx=63), INVALID), (dict(ldb=1), INVALID), (dict(ldr=-8), INVALID),
    (dict(ldy=2 ** 62), INVALID), (dict(x=None), INVALID), (dict(b=FAKE + 2), INVALID),
    (dict(r=None), INVALID), (dict(y=None), INVALID),
    (dict(pre=0), INVALID),                              # (a y without a norm)
    (dict(r=FAKE, ldr=72), INVALID),                     # (r is x, with rows of another distance)
])
def test_join_refuses(moe, kw, want):
    assert _join(moe, **kw) == want


def test_join_of_no_rows(moe):
    assert _join(moe, rows=0, x=None, b=None, r=None, y=None) == 0


def _join_back(moe, b=FAKE, r=FAKE, stats=FAKE, rng=None, dr=FAKE, dy=FAKE, dx=FAKE, db=FAKE,
               vectors={}, grads={}, ws=FAKE, ws_bytes=None, **kw):
    c = moe.moe_join_config(**{**dict(rows=4, d=64, dtype=1, post=1, pre=1, eps=1e-5, scale=1.0),
                               **kw})
    w = _params(moe, c.post, c.pre, **vectors)
    g = moe.moe_join_grads(**grads)
    if ws_bytes is None:
        ws_bytes = moe.moe_block_join_workspace_size(4, 64, "bf16")
    return moe.raw_call("moe_block_join_backward", ctypes.byref(c), b, r, stats, ctypes.byref(w),
                        rng, dr, dy, dx, db, ctypes.byref(g), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(kw, stats=FAKE + 4) if "stats" in kw else kw, w) for kw, w in JOIN_CONFIGS] + [
    (dict(lddx=63), INVALID), (dict(lddb=1), INVALID), (dict(lddr=-8), INVALID),
    (dict(lddy=2 ** 62), INVALID), (dict(b=None), INVALID), (dict(r=None), INVALID),
    (dict(stats=None), INVALID), (dict(dr=FAKE + 2), INVALID), (dict(dy=FAKE + 2), INVALID),
    (dict(dx=FAKE + 2), INVALID), (dict(db=FAKE + 2), INVALID),
    (dict(pre=0, r=None), INVALID),                      # (a dy without a norm)
    (dict(grads=dict(gate=FAKE)), INVALID),              # (no gate)
    (dict(grads=dict(post_beta=FAKE)), INVALID), (dict(grads=dict(pre_beta=FAKE)), INVALID),
    (dict(post=0, b=None, grads=dict(post_gamma=FAKE)), INVALID),
    (dict(post=0, b=None, vectors=dict(gate=FAKE), grads=dict(gate=FAKE)), INVALID),  # (needs b)
    (dict(grads=dict(post_gamma=FAKE + 4)), INVALID),
    (dict(ws=None), INVALID), (dict(ws=FAKE + 16), INVALID), (dict(ws_bytes=1024), WORKSPACE),
])
def test_join_backward_refuses(moe, kw, want):
    assert _join_back(moe, **kw) == want


def _loss(moe, x=FAKE, W=FAKE, t=FAKE, loss=FAKE, lse=FAKE, ws=FAKE, ws_bytes=1 << 34, **kw):
    c = moe.moe_loss_config(**{**dict(n=4, d=64, vocab=100, dtype=1), **kw})
    return moe.raw_call("moe_cross_entropy", ctypes.byref(c), x, W, t, loss, lse, ws, ws_bytes, None)


def _loss_back(moe, x=FAKE, W=FAKE, t=FAKE, lse=FAKE, loss=FAKE, dx=FAKE, dW=FAKE, ws=FAKE,
               ws_bytes=1 << 34, **kw):
    c = moe.moe_loss_config(**{**dict(n=4, d=64, vocab=100, dtype=1), **kw})
    return moe.raw_call("moe_cross_entropy_backward", ctypes.byref(c), x, W, t, lse, loss, dx, dW,
                        ws, ws_bytes, None)


LOSS = [
    (dict(n=-1), INVALID), (dict(n=2 ** 20 + 1), UNSUPPORTED), (dict(d=0), INVALID),
    (dict(d=60), UNSUPPORTED), (dict(d=66, dtype=0), UNSUPPORTED), (dict(vocab=0), INVALID),
    (dict(d=65544), UNSUPPORTED),
    (dict(vocab=2 ** 24 + 1), UNSUPPORTED), (dict(dtype=2), INVALID), (dict(reserved=1), INVALID),
    (dict(z_loss=-1.0), INVALID), (dict(z_loss=float("nan")), INVALID),
    (dict(z_loss=float("inf")), INVALID), (dict(x=None), INVALID), (dict(x=FAKE + 8), INVALID),
    (dict(W=None), INVALID), (dict(W=FAKE + 2), INVALID), (dict(t=None), INVALID),
    (dict(t=FAKE + 4), INVALID), (dict(loss=None), INVALID), (dict(lse=None), INVALID),
    (dict(lse=FAKE + 4), INVALID), (dict(ws=None), INVALID), (dict(ws=FAKE + 16), INVALID),
    (dict(ws_bytes=100), WORKSPACE),
]


@pytest.mark.parametrize("kw,want", LOSS)
def test_cross_entropy_refuses(moe, kw, want):
    assert _loss(moe, **kw) == want
    assert _loss_back(moe, **kw) == want


def test_cross_entropy_backward_refuses(moe):
    assert _loss_back(moe, dx=FAKE + 8) == INVALID
    assert _loss_back(moe, dW=FAKE + 8) == INVALID


def test_cross_entropy_without_work(moe):
    assert _loss(moe, n=0, x=None, t=None, loss=None, lse=None) == 0
    assert _loss_back(moe, n=0, x=None, t=None, lse=None, loss=None, dW=None) == 0
    assert _loss_back(moe, dx=None, dW=None) == 0


@pytest.mark.parametrize("n,d,vocab,dtype", [
    (0, 64, 100, "bf16"), (1, 8, 1, "bf16"), (4096, 4096, 131072, "bf16"),
    (2 ** 20, 8192, 2 ** 18, "bf16"), (2 ** 20, 4, 7, "f32"), (1, 4, 2 ** 24, "f32"),
    (1000, 512, 50021, "f32")])
def test_loss_workspace_stays_below_the_logits(moe, n, d, vocab, dtype):
    """A piece of the logits, the partial sums and a few copies of x: a bound of each."""
    z = 2 if dtype == "bf16" else 4
    got = moe.moe_cross_entropy_workspace_size(n, d, vocab, dtype)
    assert got % 256 == 0
    pieces = 1 + vocab * (n + 8) * 4 // (192 << 20)
    piece = min((n + 8) * vocab * 4, max(256 << 20, 256 * (n + 8) * 4))
    assert got <= (piece + 8 * n * (vocab // 256 + 1) + n * d * z + 64 * n + 65536
                   + (pieces * z + 152 * 4) * n * d)


# --------------------------------------------------------------- the binding
@pytest.fixture()
def silent(moe, monkeypatch):
    """The library's entry points do nothing here; what reached them."""
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append((name, a)) or 0

    monkeypatch.setattr(moe, "_lib", Lib())
    return seen


RNG = torch.tensor([1, 2])
SHARED = [lambda d: torch.zeros(d).expand(4, d),
          lambda d: torch.zeros(4 * d).as_strided((4, d), (d - 1, 1)),
          lambda d: torch.zeros(d, 4).T]


@pytest.mark.parametrize("make", SHARED)
def test_binding_refuses_rows_that_are_not_their_own(moe, silent, make):
    good, bad = torch.zeros(4, 64), make(64)
    v = moe.make_join_params(dict(post_gamma=torch.ones(64), pre_gamma=torch.ones(64)))
    none = moe.make_join_grads({})
    ws, st = torch.zeros(16, dtype=torch.uint8), torch.zeros(4, 4)
    for a in ((bad, good), (good, bad)):
        with pytest.raises(ValueError):
            moe.moe_dropout(*a, 0.1, RNG, stream=0)
    for i in range(4):
        rows = [bad if i == j else good for j in range(4)]
        with pytest.raises(ValueError):
            moe.moe_block_join(*rows[:2], v, *rows[2:], None, stream=0)
    for i in range(6):
        b, r, dr, dy, dx, db = [bad if i == j else good for j in range(6)]
        with pytest.raises(ValueError):
            moe.moe_block_join_backward(b, r, st, v, dr, dy, dx, db, none, ws, stream=0)
    assert silent == []


def test_binding_refuses_other_shapes_and_types(moe, silent):
    x, half = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.moe_dropout(x, half, 0.1, RNG, stream=0)
    with pytest.raises(ValueError):
        moe.moe_dropout(x, x, 0.1, torch.zeros(2), stream=0)
    with pytest.raises(ValueError):
        moe.moe_dropout(x, x, 0.1, torch.zeros(3, dtype=torch.int64), stream=0)
    with pytest.raises(ValueError):
        moe.moe_dropout(x.double(), x.double(), 0.1, RNG, stream=0)
    with pytest.raises(ValueError):
        moe.make_join_params(dict(gamma=torch.ones(64)))
    with pytest.raises(ValueError):
        moe.make_join_params(dict(gate=torch.ones(64), pre_gamma=torch.ones(32)))
    with pytest.raises(ValueError):
        moe.make_join_grads(dict(gate=torch.ones(64, dtype=torch.bfloat16)))
    v = moe.make_join_params(dict(post_gamma=torch.ones(32), pre_gamma=torch.ones(32)))
    with pytest.raises(ValueError):
        moe.moe_block_join(x, x, v, x, x, None, stream=0)
    W, t, f = torch.zeros(10, 64), torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    ws = torch.zeros(16, dtype=torch.uint8)
    for args in ((x, W[:, :32], t, f, f), (x, W.bfloat16(), t, f, f), (x, W, t.long(), f, f),
                 (x, W, t[:3], f, f), (x, W, t, f[:3], f), (x, W, t, f, f.double()),
                 (x.T, W, t, f, f)):
        with pytest.raises(ValueError):
            moe.moe_cross_entropy(*args, ws, stream=0)
    with pytest.raises(ValueError):
        moe.moe_cross_entropy(x, W, t, f, f, ws.float(), stream=0)
    with pytest.raises(ValueError):
        moe.moe_cross_entropy_backward(x, W, t, f, f, x, x, ws, stream=0)
    assert silent == []


def test_binding_passes_rows_of_their_own(moe, silent):
    wide = torch.zeros(4, 70)[:, :64]
    v = moe.make_join_params({})
    moe.moe_block_join(wide, wide, v, torch.zeros(4, 64), None, None, post="none", pre="none",
                       stream=0)
    moe.moe_dropout(torch.zeros(64).expand(1, 64), torch.zeros(1, 64), 0.0, stream=0)
    (name, a), (other, b) = silent
    assert name == "moe_block_join" and (a[0]._obj.ldx, a[0]._obj.ldr) == (70, 64)
    assert other == "moe_dropout" and b[0]._obj.ldx == 64
