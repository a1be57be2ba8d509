"""Layer norm refuses outputs that share bytes with inputs or with one another, and takes
ones that only lie among them."""
import pytest
import torch

from lm_head_projection_flce_b200 import build as B
from lm_head_projection_flce_b200 import flce

from gpu_common import gpu_device

N, H = 4, 64
NAMES = ("x", "w", "b", "y", "mean", "rstd", "dy", "dx", "dw", "db", "ws")


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: nothing may be launched")
    B.build()
    return flce.load_library()


def _fwd(lib, **kw):
    a = {name: (i + 1) << 24 for i, name in enumerate(NAMES)} | dict(ldx=H, ldy=H, n=N) | kw
    status = lib.flce_layer_norm_forward(a["x"], 1, a["n"], H, a["ldx"], a["w"], a["b"], 1, 1e-5, a["y"],
                                         a["ldy"], a["mean"], a["rstd"], None)
    assert status in (1, 3, 4)  # not refused: there is no device
    return status == 1


def _bwd(lib, **kw):
    a = {name: (i + 1) << 24 for i, name in enumerate(NAMES)} | dict(ldx=H, lddy=H, lddx=H) | kw
    need = lib.flce_layer_norm_workspace_size(N, H)
    status = lib.flce_layer_norm_backward(a["dy"], a["lddy"], a["x"], 1, N, H, a["ldx"], a["w"], 1, a["mean"],
                                          a["rstd"], a["dx"], a["lddx"], a["dw"], a["db"], a["ws"], need, None)
    assert status in (1, 3, 4)
    return status == 1


def test_forward(lib):
    x, row = 1 << 24, 4 * H
    assert not _fwd(lib)
    for shift in (0, 4, N * row - 4, -4, -(N * row - 4)):
        assert _fwd(lib, y=x + shift), shift
    assert not _fwd(lib, y=x + N * row) and not _fwd(lib, y=x - N * row)
    # two halves of one buffer's rows, and rows one element too close
    assert not _fwd(lib, ldx=2 * H, ldy=2 * H, y=x + row)
    assert _fwd(lib, ldx=2 * H, ldy=2 * H, y=x + row - 4) and _fwd(lib, ldx=2 * H, ldy=2 * H, y=x + row + 4)
    assert not _fwd(lib, ldx=2 * H, ldy=3 * H, y=x + row, n=1) and _fwd(lib, ldx=2 * H, ldy=3 * H, y=x + row)
    for a, b in (("y", "w"), ("y", "b"), ("y", "mean"), ("mean", "rstd"), ("mean", "x"), ("rstd", "b")):
        assert _fwd(lib, **{a: (NAMES.index(b) + 1) << 24}), (a, b)
    assert not _fwd(lib, b=2 << 24)  # weight and bias in one: both are only read
    assert not _fwd(lib, w=None, b=None, mean=None, rstd=None)


def test_backward(lib):
    assert not _bwd(lib)
    assert not _bwd(lib, dy=1 << 24)  # only read
    for a, b in (("dx", "x"), ("dx", "dy"), ("dx", "w"), ("dx", "mean"), ("dw", "w"), ("db", "dw"), ("ws", "dx"),
                 ("ws", "x"), ("dw", "ws"), ("db", "rstd")):
        assert _bwd(lib, **{a: (NAMES.index(b) + 1) << 24}), (a, b)
    assert not _bwd(lib, ldx=2 * H, lddx=2 * H, dx=(1 << 24) + 4 * H)


@pytest.mark.gpu
def test_on_the_gpu():
    dev = gpu_device()
    buf = torch.randn(50, 200, device=dev)
    x = buf[:, :100]
    want = flce.layer_norm_forward(x.clone())
    keep = buf.clone()
    for y in (x, buf[:, 50:150]):
        with pytest.raises(flce.FlceError, match="INVALID_ARG"):
            flce.layer_norm_forward(x, y=y)
    with pytest.raises(flce.FlceError, match="INVALID_ARG"):
        flce.layer_norm_backward(x, x, want[1], want[2], dx=x)
    assert torch.equal(buf, keep)
    y, mean, rstd = flce.layer_norm_forward(x, y=buf[:, 100:])  # the other half of the same rows
    assert torch.equal(y, want[0]) and torch.equal(x, keep[:, :100])
    dx = flce.layer_norm_backward(x, x, mean, rstd, dx=buf[:, 100:], want=("dx",))[0]
    assert torch.equal(dx, flce.layer_norm_backward(x.clone(), x.clone(), mean, rstd, want=("dx",))[0])
