"""beam_reorder on the GPU: lists that share memory are refused before anything is
launched, and states that interleave without sharing any are moved."""
import pytest
import torch

from lm_head_projection_flce_b200 import flce

from gpu_common import gpu_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def test_refused_lists_are_left_as_they_were(dev):
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(2, 3, 4, 8, generator=g).to(dev) for _ in range(2))
    long = torch.randn(2 * 3 * 32 + 40, generator=g).to(dev)
    part = [long[i:i + 2 * 3 * 32].view(2, 3, 4, 8) for i in (0, 8, 32)]
    parents = torch.tensor([[2, 0, 1], [1, 1, 0]], device=dev)
    before = [t.clone() for t in (k, v, long, parents)]
    for states, out in (([k, v], [v, k]), (part[0], part[1]), (part[1], part[0]), (part[0], part[2]),
                        ([part[0], part[1]], None), ([k, k], None)):
        with pytest.raises(flce.FlceError, match="INVALID_ARG"):
            flce.beam_reorder(states, parents, out=out)
    with pytest.raises(flce.FlceError, match="INVALID_ARG"):  # the parents themselves
        flce.beam_reorder(parents[:, :, None], parents)
    torch.cuda.synchronize(dev)
    assert all(torch.equal(a, b) for a, b in zip((k, v, long, parents), before))
    assert flce.get_error(dev) == flce.FLCE_OK


def test_many_interleaved_states(dev):
    """The layers' keys and values as views of one cache [B, K, layer, 2, T, D], in place and out."""
    g = torch.Generator().manual_seed(2)
    cache = torch.randn(2, 4, 6, 2, 5, 8, generator=g).to(torch.bfloat16).to(dev)
    parents = torch.randint(0, 4, (2, 4), generator=g).to(dev)
    want = cache[torch.arange(2, device=dev)[:, None], parents]
    views = lambda t: [t[:, :, i, j] for i in range(6) for j in range(2)]  # noqa: E731
    out = torch.empty_like(cache)
    flce.beam_reorder(views(cache), parents, out=views(out))
    assert torch.equal(out, want)
    flce.beam_reorder(views(cache), parents)
    assert torch.equal(cache, want)
