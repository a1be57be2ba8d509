"""Beam selection and state reordering on the GPU against their definitions.

Parents and tokens are equal.  A score is FP64 arithmetic rounded once to FP32
(2^-24 of it), on a logsumexp whose sum of exponentials is FP32: each term is
off by the 2-ulp error of the base-2 exponential (2^-22) and its argument's
rounding (2^-23 of |z - max| log2 e, up to 2^-18 for terms 20 below the
maximum, which weigh e^-20), and a thread's sum of up to V / 256 of them by
V / 256 roundings; a relative error of the sum is an absolute one of the score,
so |error| <= 2^-24 |score| + (V / 256 + 16) 2^-23.  Candidates of one
beam are ordered by their logits and equal rows have equal sums, so only
candidates of different beams nearer to one another than that error could
change places; among the seeded inputs here none do."""
import numpy as np
import pytest
import torch

from lm_head_projection_flce_b200 import flce
from oracle import head_ops as HO

from gpu_common import gpu_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def _np(t):
    return t.detach().double().cpu().numpy()


def _inputs(seed, b, k, v, dtype, ld=None):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(b, k, ld or v, generator=g) * 2.5).to(dtype)
    s = -torch.rand(b, k, generator=g) * 10
    return z, s


def _check(dev, z, s, m, finished=None, eos=None, v=None):
    kw = {} if finished is None else dict(finished=finished.to(dev), eos_token=eos)
    got = flce.beam_select(z.to(dev), s.to(dev), num_select=m, unpadded_vocab=v, **kw)
    v = v or z.shape[-1]
    ref = HO.beam_select(_np(z)[..., :v], _np(s), m, None if finished is None else finished.numpy(), eos)
    assert np.array_equal(got[1].cpu().numpy(), ref[1]), (got[1], ref[1])
    assert np.array_equal(got[2].cpu().numpy(), ref[2])
    gs = _np(got[0])
    low = np.isneginf(ref[0])
    assert np.array_equal(np.isneginf(gs), low)
    err = np.abs(gs[~low] - ref[0][~low])
    assert np.all(err <= 2.0 ** -24 * np.abs(ref[0][~low]) + (v / 256 + 16) * 2.0 ** -23)
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b,k,v,m", [(1, 1, 1, 1), (2, 3, 2, 6), (1, 4, 7, 8), (3, 5, 1000, 10), (2, 4, 4097, 4),
                                     (1, 1, 50001, 64), (1, 4, 33333, 4), (70, 8, 1003, 16), (2, 64, 1024, 64),
                                     (1, 16, 20480, 32), (5, 2, 2047, 1)])
def test_select(dev, dtype, b, k, v, m):
    z, s = _inputs(b * 1000 + k + v, b, k, v, dtype)
    _check(dev, z, s, m)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ld", [1001, 1008])
def test_padded_vocab_and_unaligned_rows(dev, dtype, ld):
    z, s = _inputs(ld, 3, 4, 1000, dtype, ld=ld)
    z[..., 997:] = 100.0             # padded tokens would win
    _check(dev, z, s, 8, v=997)
    full = z.to(dev)
    got = flce.beam_select(full[..., :997], s.to(dev))
    want = flce.beam_select(full, s.to(dev), unpadded_vocab=997)
    assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_ties_go_to_the_lowest_index(dev):
    for v in (300, 5000, 20000):
        z = torch.zeros(2, 3, v)
        _check(dev, z, torch.zeros(2, 3), 12)
        z[:, :, v // 2:] = -0.0      # the same value
        z[0, 1, ::7] = 1.0
        z[0, 2, ::7] = 1.0
        _check(dev, z, torch.zeros(2, 3), 12)
    # equal rows at different alignments stay exactly tied
    z, _ = _inputs(3, 1, 1, 5001, torch.bfloat16)
    z = z.expand(1, 6, 5001).contiguous()
    _check(dev, z, torch.zeros(1, 6), 12)


def test_all_large_elements_in_one_thread(dev):
    """Far more elements above the bound than the sorted list holds."""
    for dtype, step in ((torch.float32, 1024), (torch.bfloat16, 2048)):
        z, s = _inputs(11, 1, 1, 400 * step, dtype)
        z = (z / 10).clamp(-1, 1)
        big = torch.randn(400, 8, generator=torch.Generator().manual_seed(1)).abs() * 3 + 2
        z.view(400, step)[:, :8] = big.to(dtype)
        _check(dev, z, s, 5)
        _check(dev, z, s, 64)


def test_dead_finished_and_masked_beams(dev):
    z, s = _inputs(21, 4, 4, 700, torch.float32)
    s[0, 1:] = -float("inf")                       # the first step: one live beam
    s[1] = -float("inf")                           # nothing live
    z[2, 0] = -float("inf")                        # a row whose mask leaves nothing
    z[2, 1, 5:] = -float("inf")                    # ... and one with five tokens left
    z[3] = torch.finfo(torch.float32).min          # masked by the lowest value
    z[3, :, 9] = 0.0
    finished = torch.zeros(4, 4, dtype=torch.bool)
    _check(dev, z, s, 8)
    finished[0, 0] = finished[2, 2] = finished[3, 1] = True
    _check(dev, z, s, 8, finished, 3)
    _check(dev, z, s, 64, finished, 699)
    finished[:] = True
    _check(dev, z, s, 4, finished.to(torch.uint8), 0)


def test_nan_and_infinite_values(dev):
    z, s = _inputs(22, 3, 3, 9000, torch.bfloat16)
    z[0, 1, 8999] = float("nan")
    z[1, 0, 17] = float("inf")
    z[2, 2] = float("nan")
    s[2, 0] = float("nan")
    _check(dev, z, s, 6)


def test_empty_batch(dev):
    out = flce.beam_select(torch.empty(0, 2, 5, device=dev), torch.empty(0, 2, device=dev))
    assert [tuple(t.shape) for t in out] == [(0, 2)] * 3


def test_graph_and_other_stream(dev):
    z, s = _inputs(31, 2, 4, 9999, torch.bfloat16)
    z, s = z.to(dev), s.to(dev)
    ref = flce.beam_select(z, s)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    got = flce.beam_select(z, s, stream=side)
    torch.cuda.current_stream(dev).wait_stream(side)
    assert all(torch.equal(a, c) for a, c in zip(got, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = flce.beam_select(z, s)
    for seed in (32, 33):
        nz, ns = _inputs(seed, 2, 4, 9999, torch.bfloat16)
        z.copy_(nz)
        s.copy_(ns)
        graph.replay()
        assert all(torch.equal(a, c) for a, c in zip(out, flce.beam_select(z, s)))


# ---------------------------------------------------------------- reordering

def _gather(state, parents):
    return state[torch.arange(state.shape[0], device=state.device)[:, None], parents]


@pytest.mark.parametrize("k", [1, 2, 4, 7, 8, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("dtype,tail", [(torch.bfloat16, (3, 40)), (torch.float32, (5,)), (torch.uint8, (7,)),
                                        (torch.bfloat16, (1, 3)), (torch.int64, ()), (torch.float16, (2, 3, 34))])
def test_reorder(dev, k, dtype, tail):
    g = torch.Generator().manual_seed(k)
    state = torch.randint(0, 100, (3, k, *tail), generator=g).to(dtype).to(dev)
    for parents in (torch.randint(0, k, (3, k), generator=g), torch.arange(k).flip(0).expand(3, k).contiguous(),
                    torch.zeros(3, k, dtype=torch.int64)):
        parents = parents.to(dev)
        want = _gather(state, parents)
        out = torch.empty_like(state)
        assert flce.beam_reorder(state, parents, out=out) is out and torch.equal(out, want)
        copy = state.clone()
        assert flce.beam_reorder(copy, parents) is copy and torch.equal(copy, want)


def test_reorder_length_strides_and_many_states(dev):
    g = torch.Generator().manual_seed(5)
    big = torch.randn(2, 4, 2, 3, 50, 16, generator=g).to(torch.bfloat16).to(dev)
    parents = torch.randint(0, 4, (2, 4), generator=g).to(dev)
    # keys and values interleaved in one cache, 33 of 50 positions filled; and 40 small states
    states = [big[:, :, 0], big[:, :, 1]] + [torch.randn(2, 4, 3, 50, 2 + i % 5, generator=g).to(dev)
                                             for i in range(40)]
    before = [t.clone() for t in states]
    want = [torch.cat([_gather(t, parents)[..., :33, :], t[..., 33:, :]], dim=-2) for t in states]
    outs = [torch.full_like(t, 7) for t in states]
    flce.beam_reorder(states, parents, length=33, length_dim=3, out=outs)
    assert all(torch.equal(o[..., :33, :], w[..., :33, :]) and torch.all(o[..., 33:, :] == 7)
               for o, w in zip(outs, want))
    assert all(torch.equal(t, c) for t, c in zip(states, before))
    flce.beam_reorder(states, parents, length=33, length_dim=3)
    assert all(torch.equal(t, w) for t, w in zip(states, want))
    flce.beam_reorder(states, parents, length=0, length_dim=3)
    assert all(torch.equal(t, w) for t, w in zip(states, want))


def test_reorder_bad_parents_keep_their_own_state(dev):
    state = torch.arange(2 * 3 * 4, dtype=torch.float32, device=dev).reshape(2, 3, 4)
    parents = torch.tensor([[2, 3, -1], [1 << 40, 0, 1]], device=dev)
    safe = torch.tensor([[2, 1, 2], [0, 0, 1]], device=dev)
    assert flce.get_error(dev) == flce.FLCE_OK
    got = flce.beam_reorder(state.clone(), parents)
    assert torch.equal(got, _gather(state, safe))
    assert flce.get_error(dev) == flce.FLCE_ERR_BAD_INDEX and flce.get_error(dev) == flce.FLCE_OK


def test_reorder_refusals(dev):
    state = torch.zeros(2, 3, 4, 5, device=dev)
    parents = torch.zeros(2, 3, dtype=torch.int64, device=dev)
    for bad in (lambda: flce.beam_reorder(state.transpose(2, 3), parents),
                lambda: flce.beam_reorder(state[:1], parents),
                lambda: flce.beam_reorder(state, parents, out=state),
                lambda: flce.beam_reorder(state, parents, out=state[:, :, :2]),
                lambda: flce.beam_reorder(state[:, :1].expand(2, 3, 4, 5), parents),
                lambda: flce.beam_reorder(state, parents, length=6, length_dim=3),
                lambda: flce.beam_reorder(state, parents, length=1, length_dim=1),
                lambda: flce.beam_reorder(state, parents[:, ::2])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(flce.FlceError):
        flce.beam_reorder([state, state], parents)       # twice in one call
    assert flce.beam_reorder([], parents) == []
    assert flce.beam_reorder(state[:0], parents[:0]).shape == (0, 3, 4, 5)
    assert flce.beam_reorder(state[:, :, :0], parents).shape == (2, 3, 0, 5)
