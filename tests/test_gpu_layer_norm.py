"""Layer norm on the GPU against its FP64 definition.

Bounds.  u = 2^-24 is an FP32 rounding's largest relative error, r half a step
of the output's type.  A row's sum passes through at most K roundings (a
thread's own columns one after the other, 5 shuffles, up to 32 warps), so the
mean is off by K u mean|x| and, with the division and the subtraction, a
centred value by c = (K + 2) u (mean|x| + |x|).  rstd is off by the relative
error of a sum of squares (K + 4 roundings, halved by the root, plus the centred
values' own error) and 3 roundings of its own: below (2 K + 8) u relative, as
long as the row's mean is not large against its spread (here |mean| < 2 std).
Every bound below is those errors carried through the formula once, doubled."""
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


def _roundings(h):
    return max(32, -(-h // 1024)) + 5 + 32


def _inputs(seed, n, h, dtype, w_dtype, dev, ld=None):
    g = torch.Generator().manual_seed(seed)
    full = (torch.randn(n, ld or h, generator=g) * 1.5 + 0.5).to(dtype).to(dev)
    x = full[:, :h]
    dy = torch.randn(n, h, generator=g).to(dtype).to(dev)
    w = (1 + 0.2 * torch.randn(h, generator=g)).to(w_dtype).to(dev)
    b = (0.3 * torch.randn(h, generator=g)).to(w_dtype).to(dev)
    return x, dy, w, b


def _check(x, dy, w, b, eps, y, mean, rstd, dx, dw, db):
    xd, dyd = _np(x), _np(dy)
    n, h = xd.shape
    wd = np.ones(h) if w is None else _np(w)
    bd = np.zeros(h) if b is None else _np(b)
    ry, rm, rr = HO.layer_norm(xd, wd, bd, eps)
    k = _roundings(h)
    ax = np.abs(xd).mean(axis=1, keepdims=True)
    c = (k + 2) * U * (ax + np.abs(xd))                   # error of a centred value
    xh = (xd - rm[:, None]) * rr[:, None]
    exh = c * rr[:, None] + (2 * k + 10) * U * np.abs(xh)  # error of xhat
    assert np.all(np.abs(_np(mean) - rm) <= 2 * (k + 1) * U * ax[:, 0])
    assert np.all(np.abs(_np(rstd) - rr) <= 2 * (2 * k + 8) * U * rr)
    if y is not None:
        tol = HALF[y.dtype] * np.abs(ry) + 2 * (exh * np.abs(wd) + 3 * U * (np.abs(xh * wd) + np.abs(bd)))
        assert np.all(np.abs(_np(y) - ry) <= tol)
    rdx, rdw, rdb = HO.layer_norm_grad(dyd, xd, wd, eps)
    g = np.abs(dyd * wd)
    if dx is not None:
        m1, m2 = g.mean(axis=1, keepdims=True), (g * np.abs(xh)).mean(axis=1, keepdims=True)
        em2 = (g * exh).mean(axis=1, keepdims=True) + (k + 3) * U * m2
        terms = g + m1 + np.abs(xh) * m2
        err = rr[:, None] * ((k + 3) * U * m1 + np.abs(xh) * em2 + exh * m2 + (2 * k + 14) * U * terms)
        assert np.all(np.abs(_np(dx) - rdx) <= HALF[dx.dtype] * np.abs(rdx) + 2 * err)
    # a column's sum over the rows: at most n + 48 roundings in all
    if dw is not None:
        err = (np.abs(dyd) * exh).sum(axis=0) + (n + 48) * U * np.abs(dyd * xh).sum(axis=0)
        assert np.all(np.abs(_np(dw) - rdw) <= HALF[dw.dtype] * np.abs(rdw) + 2 * err)
    if db is not None:
        err = (n + 48) * U * np.abs(dyd).sum(axis=0)
        assert np.all(np.abs(_np(db) - rdb) <= HALF[db.dtype] * np.abs(rdb) + 2 * err)


SIZES = [(1, 1), (3, 2), (5, 7), (64, 256), (2, 257), (7, 510), (33, 1000), (333, 1001), (9, 1380), (17, 2049),
         (4, 4094), (40, 4096), (3, 5376), (2, 8191), (600, 64), (5, 8192), (2, 8200), (3, 20001)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,h", SIZES)
def test_parity(dev, dtype, n, h):
    w_dtype = torch.float32 if (n + h) % 2 else dtype
    x, dy, w, b = _inputs(n * 7 + h, n, h, dtype, w_dtype, dev)
    y, mean, rstd = flce.layer_norm_forward(x, w, b, eps=1e-3)
    dx, dw, db = flce.layer_norm_backward(dy, x, mean, rstd, w)
    assert y.dtype == dx.dtype == dtype and dw.dtype == db.dtype == w_dtype
    _check(x, dy, w, b, 1e-3, y, mean, rstd, dx, dw, db)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,h,ld,off", [(700, 8192, 8192, 0), (5000, 1040, 1040, 0), (6003, 1003, 1003, 3),
                                        (701, 5377, 5380, 1), (700, 4096, 4100, 0), (3001, 2050, 2050, 8)])
def test_more_rows_than_blocks(dev, dtype, n, h, ld, off):
    """Rows streamed through shared memory: aligned, odd, with gaps, starting and ending anywhere."""
    g = torch.Generator(device=dev).manual_seed(n + h)
    flat = torch.randn(2, n * ld + off, generator=g, device=dev) * 1.5 + 0.5
    flat = flat.to(dtype)
    x, dy = (flat[i, off:].view(n, ld)[:, :h] for i in (0, 1))
    w = 1 + 0.2 * torch.randn(h, generator=g, device=dev)
    b = 0.3 * torch.randn(h, generator=g, device=dev)
    y, mean, rstd = flce.layer_norm_forward(x, w, b)
    dx, dw, db = flce.layer_norm_backward(dy, x, mean, rstd, w)
    _check(x, dy, w, b, 1e-5, y, mean, rstd, dx, dw, db)
    only = flce.layer_norm_backward(dy, x, mean, rstd, w, want=("dweight", "dbias"))
    assert torch.equal(only[1], dw) and torch.equal(only[2], db)
    assert flce.get_error(dev) == flce.FLCE_OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("h,ld,off", [(256, 264, 0), (256, 257, 0), (100, 128, 4), (511, 600, 1)])
def test_row_strides_and_gaps(dev, dtype, h, ld, off):
    x, dy, w, b = _inputs(h + ld, 21, h, dtype, dtype, dev, ld=ld + off)
    x = x if off == 0 else torch.nn.functional.pad(x, (off, ld))[:, off:off + h]
    ybuf = torch.full((21, ld), 7.0, dtype=dtype, device=dev)
    dbuf = torch.full((21, ld + 8), 7.0, dtype=dtype, device=dev)
    y, mean, rstd = flce.layer_norm_forward(x, w, b, y=ybuf[:, :h])
    dx, dw, db = flce.layer_norm_backward(dy, x, mean, rstd, w, dx=dbuf[:, :h])
    _check(x, dy, w, b, 1e-5, y, mean, rstd, dx, dw, db)
    assert torch.all(ybuf[:, h:] == 7.0) and torch.all(dbuf[:, h:] == 7.0)


@pytest.mark.parametrize("has_w,has_b", [(False, False), (True, False), (False, True)])
def test_without_weight_or_bias(dev, has_w, has_b):
    x, dy, w, b = _inputs(4, 19, 300, torch.float32, torch.bfloat16, dev)
    w, b = w if has_w else None, b if has_b else None
    y, mean, rstd = flce.layer_norm_forward(x, w, b)
    dx, dw, db = flce.layer_norm_backward(dy, x, mean, rstd, w, param_dtype=torch.bfloat16)
    _check(x, dy, w, b, 1e-5, y, mean, rstd, dx, dw, db)
    only = flce.layer_norm_backward(dy, x, mean, rstd, w, want=("dbias",), param_dtype=torch.bfloat16)
    assert only[0] is None and only[1] is None and torch.equal(only[2], db)
    only = flce.layer_norm_backward(dy, x, mean, rstd, w, want=("dx",))
    assert torch.equal(only[0], dx) and only[1] is None


def test_autograd_shapes_and_shared_input(dev):
    """[B, S, H] with a broadcast upstream gradient; x used twice gets both gradients."""
    x, _, w, b = _inputs(5, 12, 96, torch.float32, torch.float32, dev)
    x3 = x.reshape(3, 4, 96).clone().requires_grad_()
    w, b = w.requires_grad_(), b.requires_grad_()
    (flce.layer_norm(x3, w, b).sum() + flce.layer_norm(x3, w, b).sum()).backward()
    one, two = x3.grad.clone(), w.grad.clone()
    x3.grad = w.grad = b.grad = None
    flce.layer_norm(x3, w, b).sum().backward()
    ones = torch.ones_like(x)
    y, mean, rstd = flce.layer_norm_forward(x, w.detach(), b.detach())
    _check(x, ones, w, b, 1e-5, None, mean, rstd, x3.grad.reshape(12, 96), w.grad, b.grad)
    assert torch.equal(one, 2 * x3.grad) and torch.equal(two, 2 * w.grad)


def test_empty_and_special_rows(dev):
    w = torch.ones(40, device=dev)
    y, mean, rstd = flce.layer_norm_forward(torch.empty(0, 40, device=dev), w, w)
    dx, dw, db = flce.layer_norm_backward(torch.empty(0, 40, device=dev), torch.empty(0, 40, device=dev),
                                          mean, rstd, w)
    assert y.shape == dx.shape == (0, 40) and torch.all(dw == 0) and torch.all(db == 0)
    x = torch.randn(4, 40, device=dev)
    x[0] = 3.0                      # no spread: y is the bias, rstd 1 / sqrt(eps)
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    y, mean, rstd = flce.layer_norm_forward(x, w, 2 * w)
    assert torch.all(y[0] == 2) and torch.all(y[1].isnan()) and torch.all(y[2].isnan())
    assert not y[3].isnan().any()   # rows do not touch one another


def test_deterministic_other_stream_and_graph(dev):
    x, dy, w, b = _inputs(6, 500, 1000, torch.bfloat16, torch.float32, dev)
    y, mean, rstd = flce.layer_norm_forward(x, w, b)
    ref = (y, *flce.layer_norm_backward(dy, x, mean, rstd, w))
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    y2, mean2, rstd2 = flce.layer_norm_forward(x, w, b, stream=side)
    got = (y2, *flce.layer_norm_backward(dy, x, mean2, rstd2, w, stream=side))
    torch.cuda.current_stream(dev).wait_stream(side)
    assert all(torch.equal(a, c) for a, c in zip(ref, got))
    sx, sdy = x.clone(), dy.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gy, gm, gr = flce.layer_norm_forward(sx, w, b)
        grads = flce.layer_norm_backward(sdy, sx, gm, gr, w)
    for seed in (7, 8):
        nx, ndy, _, _ = _inputs(seed, 500, 1000, torch.bfloat16, torch.float32, dev)
        sx.copy_(nx)
        sdy.copy_(ndy)
        graph.replay()
        y, mean, rstd = flce.layer_norm_forward(nx, w, b)
        want = (y, *flce.layer_norm_backward(ndy, nx, mean, rstd, w))
        assert all(torch.equal(a, c) for a, c in zip((gy, *grads), want))


def test_rows_that_must_be_copied(dev):
    """Leading dimensions without one row stride: copied on the stream the kernel runs on."""
    x, _, w, b = _inputs(11, 60, 130, torch.bfloat16, torch.float32, dev)
    t = x.reshape(6, 10, 130).transpose(0, 1)
    want = flce.layer_norm_forward(t.contiguous(), w, b)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    for stream in (None, side):
        got = flce.layer_norm_forward(t, w, b, stream=stream)
        dx, _, _ = flce.layer_norm_backward(t, t, got[1], got[2], w, stream=stream, want=("dx",))
        torch.cuda.synchronize(dev)
        assert all(torch.equal(a, c) for a, c in zip(got, want))
        assert dx.shape == t.shape
    with pytest.raises(ValueError, match="one stride"):
        flce.layer_norm_forward(t.contiguous(), w, b, y=torch.empty_like(x).reshape(6, 10, 130).transpose(0, 1))
    with pytest.raises(ValueError, match="contiguous"):
        flce.layer_norm_forward(torch.empty(130, 60, device=dev).t(), w, b)


def test_no_second_derivative(dev):
    x = torch.randn(3, 64, device=dev, requires_grad=True)
    (g,) = torch.autograd.grad(flce.layer_norm(x).square().sum(), x)
    with pytest.raises(RuntimeError, match="no gradient"):
        torch.autograd.grad(flce.layer_norm(x).square().sum(), x, create_graph=True)


def test_norm_in_front_of_the_loss(dev):
    """fused_linear_cross_entropy with norm_weight / norm_bias equals the two calls."""
    g = torch.Generator().manual_seed(9)
    x = (torch.randn(64, 256, generator=g) * 2).to(torch.bfloat16).to(dev)
    head = (torch.randn(1000, 256, generator=g) * 0.05).to(torch.bfloat16).to(dev)
    labels = torch.randint(0, 1000, (64,), generator=g).to(dev)
    w, b = torch.rand(256, generator=g).to(dev) + 0.5, torch.randn(256, generator=g).to(dev)
    leaves = [t.clone().requires_grad_() for t in (x, head, w, b)]
    loss = flce.fused_linear_cross_entropy(leaves[0], leaves[1], labels, norm_weight=leaves[2],
                                           norm_bias=leaves[3], norm_eps=1e-6)
    loss.backward()
    y, mean, rstd = flce.layer_norm_forward(x, w, b, eps=1e-6)
    l2, lse = flce.forward(y, head, labels)
    dh, dhead = flce.backward(y, head, labels, lse, torch.ones(1, device=dev))
    dx, dw, db = flce.layer_norm_backward(dh, x, mean, rstd, w)
    assert torch.equal(loss.detach(), l2)
    for leaf, want in zip(leaves, (dx, dhead, dw, db)):
        assert torch.equal(leaf.grad, want)
    assert flce.get_error(dev) == flce.FLCE_OK
