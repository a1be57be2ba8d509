"""MXFP4 on the GPU against its FP64 definition.  Codes, scales and dequantised
values are equal bit for bit: dividing by a power of two is exact.  The
product's error is FP32 accumulation: the tensor core adds the H products of
a logit in some order, each partial sum rounded or cut once, so it is off by at
most H 2^-23 sum |products|; the cap adds 8 x 2^-24 relative to its result (tanhf
2 ulp = 4 x 2^-24, its argument two roundings, the product one; tanh' <= 1) and
the output's type half a step."""
import numpy as np
import pytest
import torch

from lm_head_projection_flce_b200 import flce
from oracle import head_ops as HO

from gpu_common import gpu_device

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def _np(t):
    return t.detach().double().cpu().numpy()


def _matrix(seed, r, c, dtype, ld=None):
    """Blocks of very different magnitude, exact ties, zero blocks."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(r, ld or c, generator=g) * torch.exp2(torch.randint(-20, 20, (r, 1), generator=g).float())
    x[::3] = torch.round(x[::3] * 4) / 4
    x[:, 5::97] = 0
    if r > 2:
        x[2] = 0
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("r,c", [(1, 1), (1, 32), (3, 33), (5, 100), (129, 256), (130, 1000), (7, 1001),
                                 (257, 264), (2, 8192), (40, 5376)])
def test_quantise(dev, dtype, r, c):
    x = _matrix(r * 31 + c, r, c, dtype)
    q = flce.mxfp4_quantize(x.to(dev))
    codes, exps, values = HO.mxfp4(_np(x))
    assert np.array_equal(q.element_codes().cpu().numpy(), codes)
    assert np.array_equal(q.block_exponents().cpu().numpy(), exps)
    for out in (torch.bfloat16, torch.float32):
        assert np.array_equal(_np(flce.mxfp4_dequantize(q, out)), values)


def test_special_blocks(dev):
    x = torch.ones(3, 96)
    x[0, 3], x[1, 40], x[2, 95] = float("nan"), float("-inf"), 2.0 ** 127
    x[0, 64:] = 2.0 ** -126          # the smallest normal numbers
    x[1, 64:] = 2.0 ** -133          # subnormal in both types
    for dtype in (torch.bfloat16, torch.float32):
        q = flce.mxfp4_quantize(x.to(dtype).to(dev))
        _, exps, values = HO.mxfp4(_np(x.to(dtype)))
        assert np.array_equal(q.block_exponents().cpu().numpy(), exps)
        assert np.array_equal(_np(flce.mxfp4_dequantize(q, torch.float32)), values, equal_nan=True)
        assert np.array_equal(_np(flce.mxfp4_dequantize(q)), values, equal_nan=True)


@pytest.mark.parametrize("c,ld", [(64, 72), (64, 65), (100, 104)])
def test_row_strides(dev, c, ld):
    full = _matrix(c + ld, 33, c, torch.bfloat16, ld=ld).to(dev)
    q = flce.mxfp4_quantize(full[:, :c])
    assert torch.equal(q.element_codes(), flce.mxfp4_quantize(full[:, :c].contiguous()).element_codes())
    out = torch.full((33, ld), 7.0, dtype=torch.bfloat16, device=dev)
    flce.mxfp4_dequantize(q, out=out[:, :c])
    assert torch.equal(out[:, :c], flce.mxfp4_dequantize(q)) and torch.all(out[:, c:] == 7.0)


def _check_logits(hidden, weight, got, softcap):
    ref, size = HO.mxfp4_logits(_np(hidden), _np(weight), softcap)
    h = hidden.shape[-1]
    tol = HALF[got.dtype] * np.abs(ref) + (h * 2.0 ** -23 * size + 8 * 2.0 ** -24 * np.abs(ref))
    err = np.abs(_np(got) - ref)
    assert np.all(err <= tol), float(np.max(err - tol))


@pytest.mark.parametrize("n", [1, 16, 17, 77, 128, 129, 193, 400])
@pytest.mark.parametrize("h,v,out,cap", [(256, 130, torch.float32, 0.0), (1000, 127, torch.bfloat16, 0.0),
                                         (96, 300, torch.float32, 5.0)])
def test_logits(dev, n, h, v, out, cap):
    g = torch.Generator().manual_seed(n * 1000 + h)
    hidden = torch.randn(n, h, generator=g).to(torch.bfloat16)
    weight = (torch.randn(v, h, generator=g) * 0.3).to(torch.bfloat16)
    head = flce.mxfp4_quantize(weight.to(dev))
    got = flce.mxfp4_logits(hidden.to(dev), head, softcap=cap, dtype=out)
    assert got.shape == (n, v) and got.dtype == out
    _check_logits(hidden, weight, got, cap)
    assert flce.get_error(dev) == flce.FLCE_OK


@pytest.mark.parametrize("h", [1, 31, 32, 33, 64, 65, 128, 129, 160, 200, 255, 257, 480, 520, 2080])
def test_logits_every_tail_of_k(dev, h):
    g = torch.Generator().manual_seed(h)
    hidden, weight = torch.randn(20, h, generator=g), torch.randn(140, h, generator=g)
    got = flce.mxfp4_logits(hidden.to(dev), flce.mxfp4_quantize(weight.to(dev)), dtype=torch.float32)
    _check_logits(hidden, weight, got, 0.0)


@pytest.mark.parametrize("n", [150, 500, 1300])
@pytest.mark.parametrize("v,out", [(20011, torch.float32), (20016, torch.float32), (20012, torch.bfloat16),
                                   (20016, torch.bfloat16), (100, torch.bfloat16)])
def test_logits_many_tiles_per_block(dev, n, v, out):
    """More tiles than SMs: the rings wrap many times; rows of every alignment."""
    g = torch.Generator().manual_seed(3)
    hidden = torch.randn(n, 320, generator=g).to(torch.bfloat16)
    weight = torch.randn(v, 320, generator=g).to(torch.bfloat16)
    got = flce.mxfp4_logits(hidden.to(dev), flce.mxfp4_quantize(weight.to(dev)), dtype=out)
    a = flce.mxfp4_dequantize(flce.mxfp4_quantize(hidden.to(dev)), torch.float32).double()
    w = flce.mxfp4_dequantize(flce.mxfp4_quantize(weight.to(dev)), torch.float32).double()
    tol = HALF[out] * (a @ w.t()).abs() + 320 * 2.0 ** -23 * (a.abs() @ w.abs().t())
    assert torch.all((got.double() - a @ w.t()).abs() <= tol)


def test_logits_padded_vocab_strides_and_shapes(dev):
    g = torch.Generator().manual_seed(4)
    full = torch.randn(6, 72, generator=g).to(dev)
    hidden = full[:, :64].reshape(2, 3, 64)
    weight = torch.randn(200, 64, generator=g).to(dev)
    weight[150:] = float("nan")          # padded rows never reach the result
    head = flce.mxfp4_quantize(weight)
    buf = torch.full((2, 3, 160), 7.0, device=dev)
    got = flce.mxfp4_logits(full[:, :64], head, unpadded_vocab=150, dtype=torch.float32,
                            logits=buf.view(6, 160)[:, :150])
    _check_logits(full[:, :64], weight[:150], got, 0.0)
    assert torch.all(buf.view(6, 160)[:, 150:] == 7.0)
    again = flce.mxfp4_logits(hidden, head, unpadded_vocab=150, dtype=torch.float32)
    assert again.shape == (2, 3, 150) and torch.equal(again.view(6, 150), got)
    assert flce.mxfp4_logits(hidden[:0], head).shape == (0, 3, 200)


def test_logits_special_values(dev):
    hidden, weight = torch.ones(3, 64, device=dev), torch.ones(10, 64, device=dev)
    hidden[1, 40] = float("inf")
    weight[4, 3] = float("nan")
    hidden[2] = 0
    got = flce.mxfp4_logits(hidden, flce.mxfp4_quantize(weight), dtype=torch.float32)
    want = torch.full((3, 10), 64.0, device=dev)
    want[2] = 0
    want[1] = want[:, 4] = float("nan")
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())


def test_graph_and_other_stream(dev):
    g = torch.Generator().manual_seed(5)
    head = flce.mxfp4_quantize(torch.randn(1000, 256, generator=g).to(dev))
    hidden = torch.randn(9, 256, generator=g).to(torch.bfloat16).to(dev)
    ref = flce.mxfp4_logits(hidden, head)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    other = flce.mxfp4_logits(hidden, head, stream=side)
    torch.cuda.current_stream(dev).wait_stream(side)
    assert torch.equal(other, ref)
    x = hidden.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = flce.mxfp4_logits(x, head)
    for seed in (6, 7):
        x.copy_(torch.randn(9, 256, generator=g).to(torch.bfloat16))
        graph.replay()
        assert torch.equal(out, flce.mxfp4_logits(x, head))


def test_loss_of_the_quantised_head(dev):
    """The quantised head spread back to BF16 goes through the fused loss."""
    g = torch.Generator().manual_seed(8)
    hidden = torch.randn(50, 256, generator=g).to(torch.bfloat16).to(dev)
    weight = (torch.randn(1000, 256, generator=g) * 0.1).to(torch.bfloat16).to(dev)
    labels = torch.randint(0, 1000, (50,), generator=g).to(dev)
    q = flce.mxfp4_quantize(weight)
    loss, lse = flce.forward(hidden, flce.mxfp4_dequantize(q), labels)
    w = HO.mxfp4(_np(weight))[2]
    z = _np(hidden) @ w.T
    top = z.max(axis=1)
    ref = top + np.log(np.exp(z - top[:, None]).sum(axis=1))
    assert np.max(np.abs(_np(lse) - ref)) <= 2e-3


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("v,pad", [(v, p) for v in (1, 7, 15, 16, 17, 100, 128, 129, 250, 257, 400)
                                   for p in (0, 1, 3)] + [(384, p) for p in range(16)])
def test_logits_rows_of_every_alignment_and_end(dev, v, pad, out):
    """The many-token kernel's stores: runs that start and end anywhere, nothing beside them."""
    n, h = 200, 64
    g = torch.Generator().manual_seed(v + pad)
    hidden = torch.randn(n, h, generator=g)
    weight = torch.randn(v, h, generator=g)
    head = flce.mxfp4_quantize(weight.to(dev))
    buf = torch.full((n * (v + pad) + 40,), 7.0, dtype=out, device=dev)
    at = pad % 5
    rows = buf[at:at + n * (v + pad)].view(n, v + pad)
    flce.mxfp4_logits(hidden.to(dev), head, dtype=out, logits=rows[:, :v])
    _check_logits(hidden, weight, rows[:, :v], 0.0)
    assert torch.all(rows[:, v:] == 7.0) and torch.all(buf[:at] == 7.0)
    assert torch.all(buf[at + n * (v + pad):] == 7.0)


@pytest.mark.parametrize("n", [3, 300])
@pytest.mark.parametrize("v", [300, 304])
@pytest.mark.parametrize("cap", [1e-3, 0.5, 20.0, 30.0, 1e6])
def test_softcap_small_and_large_values(dev, n, v, cap):
    """The cap's value itself: of the uncapped logits in FP32 it is off by the rounding of a few
    operations (their errors sum to 4 units of 2^-24 on the series' side, 7 beyond: exp2
    and the reciprocal to 2^-22, each times at most 0.35, and four roundings)."""
    g = torch.Generator().manual_seed(n + v)
    hidden = torch.randn(n, 96, generator=g).to(dev)
    weight = torch.randn(v, 96, generator=g) * torch.logspace(-4, 2, v)[:, None]
    head = flce.mxfp4_quantize(weight.to(dev))
    z = flce.mxfp4_logits(hidden, head, dtype=torch.float32).double()
    got = flce.mxfp4_logits(hidden, head, dtype=torch.float32, softcap=cap)
    want = cap * torch.tanh(z / cap)
    err = (got.double() - want).abs()
    assert torch.all(err <= 8 * 2.0 ** -24 * want.abs()), float((err / want.abs()).nan_to_num().max() * 2 ** 24)
    assert torch.equal(got.sign(), z.float().sign())
    low = flce.mxfp4_logits(hidden, head, softcap=cap)
    assert torch.equal(low, got.to(torch.bfloat16))


@pytest.mark.parametrize("n", [3, 300])
def test_softcap_of_nan(dev, n):
    g = torch.Generator().manual_seed(n)
    hidden, weight = torch.randn(n, 64, generator=g), torch.randn(200, 64, generator=g)
    hidden[1, 5] = float("nan")
    weight[150, 40] = float("inf")
    z = flce.mxfp4_logits(hidden.to(dev), flce.mxfp4_quantize(weight.to(dev)), dtype=torch.float32, softcap=5.0)
    bad = torch.zeros(n, 200, dtype=torch.bool, device=dev)
    bad[1], bad[:, 150] = True, True
    assert torch.equal(z.isnan(), bad)
