"""Layer norm has no forward-mode derivative: a call that would have to return one says so,
whether or not its arguments require a gradient."""
import pytest
import torch
import torch.autograd.forward_ad as fw

from lm_head_projection_flce_b200 import flce

from gpu_common import gpu_device


def _refused(dev):
    x, w, b = (torch.randn(*s, device=dev) for s in ((3, 8), (8,), (8,)))
    plain = {"x": x, "weight": w, "bias": b}
    with fw.dual_level():
        for name in plain:
            for grad in (False, True):
                args = dict(plain, x=x.clone().requires_grad_(grad))
                args[name] = fw.make_dual(args[name], torch.ones_like(args[name]))
                with pytest.raises(NotImplementedError):
                    flce.layer_norm(**args)
                with torch.no_grad(), pytest.raises(NotImplementedError):
                    flce.layer_norm(**args)
    # the upstream gradient's tangent
    x = x.requires_grad_()
    y = flce.layer_norm(x, w, b)
    with fw.dual_level(), pytest.raises(NotImplementedError, match="forward-mode"):
        torch.autograd.grad(y, x, fw.make_dual(torch.ones_like(y), torch.ones_like(y)))


def test_refused_on_the_host(monkeypatch):
    monkeypatch.setattr(flce, "layer_norm_forward",
                        lambda x, w, b, **kw: (torch.zeros(x.shape), torch.zeros(3), torch.zeros(3)))
    _refused("cpu")


@pytest.mark.gpu
def test_refused():
    dev = gpu_device()
    _refused(dev)
    x = torch.randn(3, 8, device=dev)
    with pytest.raises(RuntimeError):  # torch's own: transforms want another form of the function
        torch.func.jvp(flce.layer_norm, (x,), (torch.ones_like(x),))
    # inside a level, tensors without a tangent go their usual way
    want = flce.layer_norm(x)
    with fw.dual_level():
        assert torch.equal(flce.layer_norm(x), want)
