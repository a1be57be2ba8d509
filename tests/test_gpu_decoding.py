"""The serving operators together: several steps of beam search whose states
follow their beams, with the norm in front and the head in 4 bits, eager and as a
captured step, against the same search in 64 bits on the host.

The logits differ from the 64-bit ones by FP32 rounding (about 1e-6 here) and the
seeded candidates lie further apart, so tokens and parents are equal; a
score gathers at most one such error per step."""
import numpy as np
import pytest
import torch

from lm_head_projection_flce_b200 import flce
from oracle import head_ops as HO

from gpu_common import gpu_device

pytestmark = pytest.mark.gpu
B, K, H, V, STEPS, EOS = 2, 3, 96, 500, 5, 7


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def _np(t):
    return t.detach().double().cpu().numpy()


def _problem(dev):
    g = torch.Generator().manual_seed(17)
    embed = torch.randn(V, H, generator=g)
    mix = torch.randn(H, H, generator=g) / H ** 0.5
    w, b = 1 + 0.1 * torch.randn(H, generator=g), 0.1 * torch.randn(H, generator=g)
    head = torch.randn(V, H, generator=g) * 0.3
    head[EOS] *= 2                                   # some beams end
    start = torch.randn(B, H, generator=g)
    return [t.to(dev) for t in (embed, mix, w, b, head, start)]


def _grid(x):
    """Hidden states on a coarse grid, so that 32 and 64 bits put the same numbers into the norm."""
    return (x * 64).round() / 64


def _search(dev, step):
    embed, mix, w, b, head, start = _problem(dev)
    state = start[:, None, :].repeat(1, K, 1)
    hidden = _grid(state)
    scores = torch.full((B, K), -float("inf"), device=dev)
    scores[:, 0] = 0.0
    done = torch.zeros(B, K, dtype=torch.bool, device=dev)
    history = []
    for _ in range(STEPS):
        scores, parents, tokens = step(hidden, scores, done, state)
        done = done.gather(1, parents) | (tokens == EOS)
        state.copy_(_grid(torch.tanh(state @ mix + embed[tokens])))
        hidden = state.clone()
        history.append((scores.clone(), parents.clone(), tokens.clone(), hidden.clone(), done.clone()))
    return history


def test_decoding_steps_equal_the_search_in_64_bits(dev):
    embed, mix, w, b, head, _ = _problem(dev)
    q = flce.mxfp4_quantize(head)
    inputs = []

    def eager(hidden, scores, done, state):
        inputs.append((hidden.clone(), scores.clone(), done.clone(), state.clone()))
        x = flce.layer_norm(hidden, w, b)
        z = flce.mxfp4_logits(x, q, dtype=torch.float32, softcap=20.0)
        out = flce.beam_select(z, scores, finished=done, eos_token=EOS)
        flce.beam_reorder(state, out[1])
        inputs[-1] += (state.clone(), x.clone())
        return out

    history = _search(dev, eager)
    for (hidden, scores, done, before, after, x), (got_s, got_p, got_t, _, _) in zip(inputs, history):
        y = HO.layer_norm(_np(hidden).reshape(-1, H), _np(w), _np(b))[0]
        assert np.max(np.abs(_np(x).reshape(-1, H) - y)) < 2e-5
        # the norm's FP32 result is what the product quantises
        z = HO.mxfp4_logits(_np(x).reshape(-1, H), _np(head), 20.0)[0].reshape(B, K, V)
        s, p, t = HO.beam_select(z, _np(scores), K, done.cpu().numpy(), EOS)
        assert np.array_equal(got_p.cpu().numpy(), p) and np.array_equal(got_t.cpu().numpy(), t)
        assert np.max(np.abs(_np(got_s) - s)) < 1e-4
        rows = np.arange(B)[:, None]
        assert np.array_equal(_np(after), _np(before)[rows, p])
    assert any(h[4].any() for h in history) and flce.get_error(dev) == flce.FLCE_OK

    # the same search as a captured step, twice from the same start
    first = inputs[0]
    state = first[3].clone()
    step = flce.CapturedBeamStep(first[0], q, first[1], norm_weight=w, norm_bias=b, softcap=20.0,
                                 dtype=torch.float32, finished=first[2], eos_token=EOS, states=[state])
    assert torch.equal(state, first[3])              # capturing runs no step on the states

    def captured(hidden, scores, done, outer):
        state.copy_(outer)
        step.set_inputs(hidden, scores, done)
        out = step.replay()
        outer.copy_(state)
        return out

    for _ in range(2):
        for got, want in zip(_search(dev, captured), history):
            assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_captured_step_refusals(dev):
    q = flce.mxfp4_quantize(torch.randn(100, 64, device=dev))
    hidden, scores = torch.randn(1, 2, 64, device=dev), torch.zeros(1, 2, device=dev)
    with pytest.raises(ValueError, match="num_select"):
        flce.CapturedBeamStep(hidden, q, scores, num_select=3, states=[torch.zeros(1, 2, 4, device=dev)])
    with pytest.raises(ValueError):
        flce.CapturedBeamStep(hidden[0], q, scores)
    step = flce.CapturedBeamStep(hidden, q, scores, num_select=4)
    assert step.replay()[0].shape == (1, 4) and step.logits.shape == (1, 2, 100)
    with pytest.raises(ValueError, match="finished"):
        step.set_inputs(finished=torch.zeros(1, 2, dtype=torch.bool, device=dev))
    with pytest.raises(ValueError, match="shapes"):
        step.set_inputs(hidden=hidden[:, :1])


def test_captured_step_owns_its_inputs(dev):
    """Scores that carry a gradient or lie transposed are copied as plain rows."""
    embed, mix, w, b, head, start = _problem(dev)
    q = flce.mxfp4_quantize(head)
    hidden = _grid(start[:, None, :].repeat(1, K, 1))
    scores = -torch.arange(float(B * K), device=dev).view(K, B).t()
    done = torch.zeros(K, B, dtype=torch.bool, device=dev).t()
    step = flce.CapturedBeamStep(hidden, q, scores.clone().requires_grad_(), finished=done, eos_token=EOS)
    assert not step.scores.requires_grad and step.scores.is_contiguous() and step.finished.is_contiguous()
    step.set_inputs(scores=scores, finished=done)
    want = flce.beam_select(flce.mxfp4_logits(hidden, q), scores.contiguous(), finished=done.contiguous(),
                            eos_token=EOS)
    assert all(torch.equal(x, y) for x, y in zip(step.replay(), want))


def test_training_step_gradients_against_differences(dev):
    """norm -> loss: the gradients of the norm's parameters against differences of the 64-bit loss."""
    g = torch.Generator().manual_seed(23)
    n, h, v = 32, 64, 200
    x = (torch.randn(n, h, generator=g) * 2).to(torch.bfloat16)
    head = (torch.randn(v, h, generator=g) * 0.2).to(torch.bfloat16)
    labels = torch.randint(0, v, (n,), generator=g)
    w, b = 1 + 0.1 * torch.randn(h, generator=g), 0.1 * torch.randn(h, generator=g)
    leaves = [t.to(dev).requires_grad_() for t in (x, w, b)]
    loss = flce.fused_linear_cross_entropy(leaves[0], head.to(dev), labels.to(dev), reduction="mean",
                                           norm_weight=leaves[1], norm_bias=leaves[2])
    loss.backward()
    x64, head64, y = _np(x), _np(head), labels.numpy()

    def ref(w64, b64):
        z = HO.layer_norm(x64, w64, b64)[0] @ head64.T
        top = z.max(axis=1, keepdims=True)
        lse = top[:, 0] + np.log(np.exp(z - top).sum(axis=1))
        return (lse - z[np.arange(n), y]).mean()

    w64, b64 = _np(w), _np(b)
    # The normalised rows, the logit gradients and dhidden are each rounded to BF16 on
    # the way, half a step (2^-8) of terms whose magnitudes sum to `size`; the rows'
    # rounding moves a logit by at most 2^-8 sum |y| |head| and so a probability by
    # twice that relative to itself.
    y_ref = HO.layer_norm(x64, w64, b64)[0]
    p = np.exp(y_ref @ head64.T)
    p /= p.sum(axis=1, keepdims=True)
    p[np.arange(n), y] += 1
    size = p @ np.abs(head64) / n
    xhat = np.abs(HO.layer_norm(x64)[0])
    rel = 2.0 ** -8 * (3 + 2 * (np.abs(y_ref) @ np.abs(head64).T).max())
    for grad, at, bound in ((leaves[1].grad, w64, (size * xhat).sum(axis=0)), (leaves[2].grad, b64, size.sum(axis=0))):
        for i in range(0, h, 7):
            step = 1e-4
            keep = at[i]
            at[i] = keep + step
            up = ref(w64, b64)
            at[i] = keep - step
            diff = (up - ref(w64, b64)) / (2 * step)
            at[i] = keep
            assert abs(float(grad[i]) - diff) <= rel * bound[i]
