"""CapturedBeamStep checks its states, and launches their reordering once, before it captures."""
import pytest
import torch

from lm_head_projection_flce_b200 import flce

from gpu_common import gpu_device

pytestmark = pytest.mark.gpu


def test_states_are_checked_outside_capture(monkeypatch):
    dev = gpu_device()
    head = flce.mxfp4_quantize(torch.randn(100, 64, device=dev))
    hidden, scores = torch.randn(2, 3, 64, device=dev), torch.zeros(2, 3, device=dev)
    good = torch.randn(2, 3, 8, device=dev)
    seen = []
    reorder = flce.beam_reorder

    def spy(*args, **kw):
        seen.append(torch.cuda.is_current_stream_capturing())
        return reorder(*args, **kw)

    monkeypatch.setattr(flce, "beam_reorder", spy)
    for bad in ([good[:1]], [good.transpose(0, 1)], [good, torch.randn(2, 4, 8, device=dev)],
                [good[:, :1].expand(2, 3, 8)], [good, good], [good, good.view(2, 3, 2, 4)[:, :, 1]]):
        seen.clear()
        with pytest.raises((ValueError, flce.FlceError)):
            flce.CapturedBeamStep(hidden, head, scores, states=bad)
        assert seen == [False]
    keep = good.clone()
    seen.clear()
    step = flce.CapturedBeamStep(hidden, head, scores, states=[good])
    assert seen == [False, True] and torch.equal(good, keep)
    _, parents, _ = step.replay()
    assert torch.equal(good, keep[torch.arange(2, device=dev)[:, None], parents])
    # one state instead of a list
    one = keep.clone()
    step = flce.CapturedBeamStep(hidden, head, scores, states=one)
    assert torch.equal(one, keep)
    _, parents, _ = step.replay()
    assert torch.equal(one, keep[torch.arange(2, device=dev)[:, None], parents])
