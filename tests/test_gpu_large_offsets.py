"""The operators around the head where element offsets pass 2^31: the rows at the
end of a large call equal the same rows in a small one, bit for bit where a row's
arithmetic does not depend on its place."""
import pytest
import torch

from lm_head_projection_flce_b200 import flce

from gpu_common import gpu_device

pytestmark = pytest.mark.gpu
OVER = 1 << 31


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def test_layer_norm(dev):
    h = 8192
    n = OVER // h + 300
    x = torch.empty(n, h, dtype=torch.bfloat16, device=dev)
    x.normal_(generator=torch.Generator(device=dev).manual_seed(1))
    w = torch.linspace(0.5, 1.5, h, device=dev)
    y, mean, rstd = flce.layer_norm_forward(x, w, w)
    ref, rm, rr = flce.layer_norm_forward(x[-300:], w, w)
    # The small call may take another kernel, whose sums round in another order: up to
    # 69 roundings (2^-24) of a mean of |x| below 1 each, twice that relative for rstd,
    # and one BF16 step (2^-7) where the two results round apart.
    assert torch.allclose(y[-300:].float(), ref.float(), rtol=2.0 ** -7, atol=2.0 ** -14)
    assert torch.allclose(mean[-300:], rm, rtol=0, atol=1e-5)
    assert torch.allclose(rstd[-300:], rr, rtol=2e-5, atol=0)
    dx, _, _ = flce.layer_norm_backward(y, x, mean, rstd, w, want=("dx",))
    small, _, _ = flce.layer_norm_backward(y[-300:], x[-300:], mean[-300:], rstd[-300:], w, want=("dx",))
    assert torch.allclose(dx[-300:].float(), small.float(), rtol=2.0 ** -7, atol=2.0 ** -14)


def test_mxfp4(dev):
    h = 8192
    n = OVER // h + 130
    x = torch.empty(n, h, dtype=torch.bfloat16, device=dev)
    x.normal_(generator=torch.Generator(device=dev).manual_seed(2))
    q = flce.mxfp4_quantize(x)
    back = flce.mxfp4_dequantize(q)
    assert torch.equal(back[-130:], flce.mxfp4_dequantize(flce.mxfp4_quantize(x[-130:])))
    del back
    head = flce.mxfp4_quantize(x[:131072, :64].contiguous())
    hidden = x[:OVER // 131072 + 100, 64:128].contiguous()
    z = flce.mxfp4_logits(hidden, head)
    assert z.numel() > OVER
    assert torch.equal(z[-100:], flce.mxfp4_logits(hidden[-100:], head))
    last = flce.mxfp4_quantize(x[131072 - 128:131072, :64].contiguous())
    assert torch.equal(z[:, -128:], flce.mxfp4_logits(hidden, last))


def test_beam_select(dev):
    b, k, v = 300, 32, 262144
    z = torch.empty(b, k, v, dtype=torch.bfloat16, device=dev)
    z.normal_(generator=torch.Generator(device=dev).manual_seed(3))
    s = -torch.rand(b, k, device=dev)
    assert z.numel() > OVER
    got = flce.beam_select(z, s)
    # one item: other segments, so the sums differ in their last bits
    want = flce.beam_select(z[-1:], s[-1:])
    assert torch.equal(got[1][-1:], want[1]) and torch.equal(got[2][-1:], want[2])
    assert torch.allclose(got[0][-1:], want[0], atol=1e-5)


def test_beam_reorder(dev):
    state = torch.empty(1, 2, OVER + 4096, dtype=torch.uint8, device=dev)
    state[0, 0].fill_(1)
    state[0, 1].fill_(2)
    state[0, :, -5:] = torch.tensor([[3], [4]], dtype=torch.uint8, device=dev)
    swap = torch.tensor([[1, 0]], device=dev)
    flce.beam_reorder(state, swap)
    assert state[0, 0, -6:].tolist() == [2, 4, 4, 4, 4, 4] and state[0, 1, -6:].tolist() == [1, 3, 3, 3, 3, 3]
    assert bool((state[0, 0, :-5] == 2).all()) and bool((state[0, 1, :-5] == 1).all())
    out = torch.zeros_like(state)
    flce.beam_reorder(state, swap, out=out)
    assert torch.equal(out[0, 0], state[0, 1]) and torch.equal(out[0, 1], state[0, 0])
