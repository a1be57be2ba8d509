"""Layer norm on the CPU: the FP64 definition's gradients against differences,
and the refusals of the entry points, before anything touches a GPU."""
import numpy as np
import pytest
import torch

from lm_head_projection_flce_b200 import build as B
from lm_head_projection_flce_b200 import flce
from oracle import head_ops as HO

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    B.build()
    return flce.load_library()


def test_definition_gradients_match_differences():
    rng = np.random.default_rng(0)
    x, dy = rng.standard_normal((3, 7)) + 0.5, rng.standard_normal((3, 7))
    w, b = rng.standard_normal(7), rng.standard_normal(7)
    dx, dw, db = HO.layer_norm_grad(dy, x, w)
    step = 1e-5

    def diff(a, fn):
        g = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            a[i] += step
            up = fn()
            a[i] -= 2 * step
            g[i] = (up - fn()) / (2 * step)
            a[i] += step
        return g

    loss = lambda: float((dy * HO.layer_norm(x, w, b)[0]).sum())  # noqa: E731
    # central differences are off by step^2 times the third derivative, here below 1e-7
    for got, at in ((dx, x), (dw, w), (db, b)):
        assert np.max(np.abs(got - diff(at, loss))) < 1e-7


def _fwd(lib, **kw):
    a = dict(x=FAKE, dtype=0, n=4, h=64, ldx=64, w=FAKE, b=FAKE, w_dtype=0, eps=1e-5, y=FAKE,
             ldy=64, mean=FAKE, rstd=FAKE)
    a.update(kw)
    return lib.flce_layer_norm_forward(*a.values(), None)


def _bwd(lib, **kw):
    a = dict(dy=FAKE, lddy=64, x=FAKE, dtype=0, n=4, h=64, ldx=64, w=FAKE, w_dtype=0, mean=FAKE,
             rstd=FAKE, dx=FAKE, lddx=64, dw=FAKE, db=FAKE, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return lib.flce_layer_norm_backward(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(n=-1), dict(h=0), dict(ldx=63), dict(dtype=2), dict(w_dtype=2),
                                 dict(x=0), dict(x=FAKE + 1), dict(w=FAKE + 1),
                                 dict(rstd=FAKE + 2)])
def test_bad_arguments_of_both(lib, bad):
    assert _fwd(lib, **bad) == 1
    assert _bwd(lib, **bad) == 1


@pytest.mark.parametrize("bad", [dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                                 dict(y=0), dict(y=FAKE + 1), dict(ldy=3), dict(b=FAKE + 1)])
def test_bad_arguments_forward(lib, bad):
    assert _fwd(lib, **bad) == 1


@pytest.mark.parametrize("bad", [dict(dy=0), dict(lddy=1), dict(lddx=1), dict(dx=FAKE + 1),
                                 dict(dw=FAKE + 1), dict(db=FAKE + 1), dict(mean=0), dict(rstd=0)])
def test_bad_arguments_backward(lib, bad):
    assert _bwd(lib, **bad) == 1


def test_workspace(lib):
    need = lib.flce_layer_norm_workspace_size(4, 64)
    assert need > 0
    assert _bwd(lib, ws=0) == 2
    assert _bwd(lib, ws_bytes=need - 1) == 2
    assert _bwd(lib, ws=FAKE + 8) == 2
    assert lib.flce_layer_norm_workspace_size(-1, 64) == 0
    assert lib.flce_layer_norm_workspace_size(4, 0) == 0
    # the partials are one row per block, not one per token
    assert lib.flce_layer_norm_workspace_size(1 << 20, 4096) < 64 << 20


def test_nothing_to_do(lib):
    assert _fwd(lib, n=0, x=0, y=0) == 0
    assert _bwd(lib, dx=0, dw=0, db=0, ws=0) == 0
    assert _bwd(lib, n=0, dw=0, db=0, ws=0) == 0


def test_binding_refuses(lib):
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        flce.layer_norm(x)
    with pytest.raises(TypeError):
        flce.layer_norm(x.half())
