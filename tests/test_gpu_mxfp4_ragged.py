"""The product with vocabularies that end inside a warp's 32 head rows, more than 32
tokens to each of its lanes: the lanes behind the last row have nothing to store
between the warp-wide loads of the accumulator.

The bound is that of FP32 accumulation: H 2^-23 of the sum of the products' magnitudes."""
import pytest
import torch

from lm_head_projection_flce_b200 import flce

from gpu_common import gpu_device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,v", [(77, 50001), (65, 33), (97, 129), (128, 1003), (161, 95), (192, 20007)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ragged_vocabulary(n, v, dtype):
    dev = gpu_device()
    h = 96
    g = torch.Generator().manual_seed(n + v)
    x, w = torch.randn(n, h, generator=g).to(dev), torch.randn(v, h, generator=g).to(dev)
    head = flce.mxfp4_quantize(w)
    guard = torch.full((n + 1, v + 3), 7.0, dtype=dtype, device=dev)
    z = flce.mxfp4_logits(x, head, dtype=dtype, logits=guard[:n, :v])
    a = flce.mxfp4_dequantize(flce.mxfp4_quantize(x), torch.float32).double()
    b = flce.mxfp4_dequantize(head, torch.float32).double()
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    half = torch.finfo(dtype).eps / 2
    assert torch.all((z.double() - want).abs() <= h * 2.0 ** -23 * size + half * want.abs() + h * 2.0 ** -23 * size * half)
    assert torch.all(guard[n] == 7) and torch.all(guard[:, v:] == 7)
    assert flce.get_error(dev) == flce.FLCE_OK
