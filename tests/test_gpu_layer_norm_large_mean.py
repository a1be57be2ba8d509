"""Layer norm of rows whose mean is large against their spread, and of constant rows.

The kernels subtract a mean m0 that is an FP32 sum, off by e0 <= K u mean|x| (K: the
roundings a row's sum passes through, u = 2^-24), and take what is left over,
r = mean(x - m0), out of the centred values.  x - m0 has the magnitude of the
spread (plus e0), so its rounding and that of r leave a centred value off by
   c = (K + 2) u (mean|x - mean| + |x - mean| + 2 e0),
whatever the mean.  The variance is mean((x - m0)^2) - r^2: the first term is off by
(K + 4) u of var + r^2, r by (K + 2) u mean|x - m0| and so r^2 by 2 (K + 2) u (var + r^2),
and |r| <= e0, which for rstd is a relative error of (3 K + 10) u (1 + e0^2 rstd^2),
halved by the root, and 4 roundings.  The backward sees the mean rounded to FP32 (u |mean|,
below e0) and takes out what is left in the same way where |mean| is above 16 standard
deviations; below, that moves xhat by 16 u, less than the (K + 2) u spread of c.  The
bounds below are those errors carried through the formula once, doubled."""
import numpy as np
import pytest
import torch

from lm_head_projection_flce_b200 import flce
from oracle import head_ops as HO

from gpu_common import gpu_device

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def _np(t):
    return t.detach().double().cpu().numpy()


def _check(x, dy, w, b, eps, y, mean, rstd, dx, dw, db):
    xd, dyd, wd, bd = _np(x), _np(dy), _np(w), _np(b)
    n, h = xd.shape
    k = max(32, -(-h // 1024)) + 5 + 32
    ry, rm, rr = HO.layer_norm(xd, wd, bd, eps)
    cent = xd - rm[:, None]
    e0 = k * U * np.abs(xd).mean(axis=1, keepdims=True)
    spread = np.abs(cent).mean(axis=1, keepdims=True)
    r = rr[:, None]
    c = (k + 2) * U * (spread + np.abs(cent) + 2 * e0)
    er = (3 * k + 10) * U * (1 + (e0 * r) ** 2) / 2 + 4 * U     # relative error of rstd
    xh = cent * r
    exh = c * r + (er + 3 * U) * np.abs(xh)
    assert np.all(np.abs(_np(mean) - rm) <= 2 * (U * np.abs(rm) + (k + 2) * U * (spread + 2 * e0)[:, 0]))
    assert np.all(np.abs(_np(rstd) - rr) <= 2 * er[:, 0] * rr)
    tol = HALF[y.dtype] * np.abs(ry) + 2 * (exh * np.abs(wd) + 3 * U * (np.abs(xh * wd) + np.abs(bd)))
    assert np.all(np.abs(_np(y) - ry) <= tol)
    rdx, rdw, rdb = HO.layer_norm_grad(dyd, xd, wd, eps)
    g = np.abs(dyd * wd)
    if dx is not None:
        m1, m2 = g.mean(axis=1, keepdims=True), (g * np.abs(xh)).mean(axis=1, keepdims=True)
        # m2 is summed over the values before r is taken out: e0 of them on top
        em2 = (g * exh).mean(axis=1, keepdims=True) + (k + 5) * U * (m2 + e0 * r * m1)
        terms = g + m1 + np.abs(xh) * m2
        err = r * ((k + 3) * U * m1 + np.abs(xh) * em2 + exh * m2 + (2 * er + 8 * U) * terms)
        assert np.all(np.abs(_np(dx) - rdx) <= HALF[dx.dtype] * np.abs(rdx) + 2 * err)
    if dw is not None:
        err = (np.abs(dyd) * exh).sum(axis=0) + (n + 48) * U * np.abs(dyd * xh).sum(axis=0)
        assert np.all(np.abs(_np(dw) - rdw) <= HALF[dw.dtype] * np.abs(rdw) + 2 * err)
    if db is not None:
        err = (n + 48) * U * np.abs(dyd).sum(axis=0)
        assert np.all(np.abs(_np(db) - rdb) <= HALF[db.dtype] * np.abs(rdb) + 2 * err)


def _params(h, seed, dev):
    g = torch.Generator().manual_seed(seed)
    return ((1 + 0.2 * torch.randn(h, generator=g)).to(dev), (0.3 * torch.randn(h, generator=g)).to(dev))


def _run(x, dy, w, b, eps=1e-5):
    y, mean, rstd = flce.layer_norm_forward(x, w, b, eps=eps)
    dx, dw, db = flce.layer_norm_backward(dy, x, mean, rstd, w)
    _check(x, dy, w, b, eps, y, mean, rstd, dx, dw, db)
    only = flce.layer_norm_backward(dy, x, mean, rstd, w, want=("dweight", "dbias"))
    assert torch.equal(only[1], dw) and torch.equal(only[2], db)
    only = flce.layer_norm_backward(dy, x, mean, rstd, w, want=("dbias",))
    assert torch.equal(only[2], db)
    only = flce.layer_norm_backward(dy, x, mean, rstd, w, want=("dx",))
    assert torch.equal(only[0], dx)


# a warp's row, a block's (vectors, single elements), streamed rows of both, long rows
SIZES = [(5, 300), (9, 512), (3, 1001), (4, 4096), (2, 8191), (900, 1040), (700, 4096), (901, 1003), (3, 20001),
         (200, 8200)]


@pytest.mark.parametrize("mean", [100.0, -1000.0, 10000.0])
@pytest.mark.parametrize("n,h", SIZES)
def test_large_mean(dev, n, h, mean):
    g = torch.Generator().manual_seed(n + h)
    x = torch.randn(n, h, generator=g) + mean
    x[0, ::3] += 5.0
    dy = torch.randn(n, h, generator=g)
    _run(x.to(dev), dy.to(dev), *_params(h, h, dev))


@pytest.mark.parametrize("n,h", SIZES)
def test_constant_and_nearly_constant_rows(dev, n, h):
    """No spread, or one unit in the last place of it: eps decides, and y is the bias."""
    g = torch.Generator().manual_seed(h)
    x = torch.full((n, h), 1000.1)
    x[1:, ::2] = torch.nextafter(x[1:, ::2], torch.tensor(2000.0))
    if n > 2:
        x[2] = -3.3e5
    dy = torch.randn(n, h, generator=g)
    _run(x.to(dev), dy.to(dev), *_params(h, h, dev))


@pytest.mark.parametrize("n,h", SIZES)
def test_rows_of_both_kinds(dev, n, h):
    """Large means among ordinary rows."""
    g = torch.Generator().manual_seed(n * h)
    x = torch.randn(n, h, generator=g)
    x[torch.rand(n, generator=g) < 0.2] += 3000.0
    x[n - 1] -= 700.0
    dy = torch.randn(n, h, generator=g)
    _run(x.to(dev), dy.to(dev), *_params(h, h, dev))


@pytest.mark.parametrize("n,h", [(5, 300), (4, 4096), (700, 4096), (3, 20001)])
def test_bf16_rows_of_large_mean(dev, n, h):
    g = torch.Generator().manual_seed(n + h)
    x = (torch.randn(n, h, generator=g) * 3 + 300).to(torch.bfloat16)
    dy = torch.randn(n, h, generator=g).to(torch.bfloat16)
    _run(x.to(dev), dy.to(dev), *_params(h, h, dev))


def test_statistics_of_special_rows(dev):
    """A NaN or an infinity reaches the row's statistics, and no other row."""
    for h in (40, 1001, 9000):
        x = torch.randn(4, h, device=dev) + 1000
        x[1, 7], x[2, 9] = float("nan"), float("inf")
        y, mean, rstd = flce.layer_norm_forward(x)
        assert torch.all(y[1:3].isnan()) and torch.all(rstd[1:3].isnan())
        assert not y[0].isnan().any() and not y[3].isnan().any()
        assert torch.equal(mean.isfinite(), torch.tensor([True, False, False, True], device=dev))
