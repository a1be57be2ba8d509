"""Beam search on the CPU: the definition on cases worked out by hand, the
refusals of the entry points."""
import ctypes

import numpy as np
import pytest
import torch

from lm_head_projection_flce_b200 import build as B
from lm_head_projection_flce_b200 import flce
from oracle import head_ops as HO

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    B.build()
    return flce.load_library()


def test_definition():
    half = np.log(0.5)
    z = np.zeros((1, 2, 2))
    s, p, t = HO.beam_select(z, np.array([[0.0, 0.0]]), 4)
    assert np.allclose(s, half) and p.tolist() == [[0, 0, 1, 1]] and t.tolist() == [[0, 1, 0, 1]]
    # a dead first beam, a finished second one: its end, then -inf from the lowest index up
    s, p, t = HO.beam_select(z, np.array([[-np.inf, -3.0]]), 3, np.array([[0, 1]]), 1)
    assert s[0, 0] == -3 and (p[0, 0], t[0, 0]) == (1, 1)
    assert np.all(np.isneginf(s[0, 1:])) and p[0, 1:].tolist() == [0, 0] and t[0, 1:].tolist() == [0, 1]


def _select(lib, **kw):
    a = dict(logits=FAKE, dtype=0, batch=2, beams=4, vocab=100, ld=100, scores=FAKE, finished=None, eos=0,
             m=4, out=FAKE, parents=FAKE, tokens=FAKE, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return lib.flce_beam_select(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(beams=0), dict(beams=65), dict(vocab=0), dict(ld=99),
                                 dict(dtype=2), dict(m=0), dict(m=65), dict(beams=1, vocab=3),
                                 dict(vocab=1 << 30, ld=1 << 30), dict(finished=FAKE, eos=-1),
                                 dict(finished=FAKE, eos=100), dict(logits=0), dict(logits=FAKE + 1),
                                 dict(scores=0), dict(scores=FAKE + 2), dict(out=0), dict(parents=0),
                                 dict(parents=FAKE + 4), dict(tokens=FAKE + 4)])
def test_select_bad_arguments(lib, bad):
    assert _select(lib, **bad) == 1


def test_select_workspace(lib):
    size = lib.flce_beam_select_workspace_size
    need = size(2, 4, 100, 4)
    assert _select(lib, ws=0) == 2 and _select(lib, ws_bytes=need - 1) == 2 and _select(lib, ws=FAKE + 8) == 2
    assert _select(lib, batch=0, logits=0, scores=0, ws=0) == 0
    assert size(2, 65, 100, 4) == 0 and size(2, 4, 100, 0) == 0
    assert 0 < size(1, 1, 262144, 64) < 1 << 20


def _state(**kw):
    s = flce.BeamState(FAKE, 2 * FAKE, 64, 16, 64, 16, 1, 0, 16)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _reorder(lib, states, parents=FAKE, batch=2, beams=4):
    arr = (flce.BeamState * len(states))(*states)
    return lib.flce_beam_reorder(ctypes.cast(arr, ctypes.c_void_p), len(states), parents, batch, beams, None)


def test_reorder_bad_arguments(lib):
    bad = [dict(src=None), dict(dst=None), dict(outer=-1), dict(inner=-1), dict(src_batch_stride=-8),
           dict(dst_beam_stride=-8), dict(outer=2, outer_stride=8), dict(dst=FAKE, dst_beam_stride=32),
           dict(outer=1 << 43, outer_stride=16)]
    for kw in bad:
        assert _reorder(lib, [_state(**kw)]) == 1, kw
    assert _reorder(lib, [_state()], parents=0) == 1
    assert _reorder(lib, [_state()], parents=FAKE + 4) == 1
    assert _reorder(lib, [_state()], batch=-1) == 1
    assert _reorder(lib, [_state()], beams=0) == 1
    assert _reorder(lib, [_state()], beams=65) == 1
    assert _reorder(lib, [_state(), _state()]) == 1        # the same state twice
    assert lib.flce_beam_reorder(None, 1, FAKE, 2, 4, None) == 1
    assert lib.flce_beam_reorder(None, 0, FAKE, 2, 4, None) == 0
    assert _reorder(lib, [_state()], batch=0) == 0


def test_state_description_is_nine_words():
    # the binding hands the library an array of 8-byte words
    assert ctypes.sizeof(flce.BeamState) == 72
    assert [getattr(flce.BeamState, n).offset for n, _ in flce.BeamState._fields_] == list(range(0, 72, 8))


def test_error_word_status(lib):
    assert b"parent" in lib.flce_status_string(flce.FLCE_ERR_BAD_INDEX)


def test_binding_refuses():
    z, s = torch.zeros(1, 2, 5), torch.zeros(1, 2)
    with pytest.raises(ValueError, match="CUDA"):
        flce.beam_select(z, s)
    with pytest.raises(TypeError):
        flce.beam_select(z.half(), s)
    with pytest.raises(ValueError, match="CUDA"):
        flce.beam_reorder(torch.zeros(1, 2, 3), torch.zeros(1, 2, dtype=torch.int64))
    with pytest.raises(TypeError):
        flce.beam_reorder(torch.zeros(1, 2, 3), torch.zeros(1, 2))


@pytest.mark.parametrize("stride", [(0, 6, 1), (12, 0, 1), (12, 5, 1), (10, 6, 1), (6, 6, 1), (3, 12, 1)])
def test_binding_refuses_beams_that_share_memory(stride):
    """[2, 2, 6] entries of which two overlap, wholly or in part."""
    with pytest.raises(ValueError, match="share memory"):
        flce._reorder_plan(torch.float32, (2, 2, 6), stride, "d", torch.float32, (2, 2, 6), stride, "d",
                           2, 2, "d", None, 2)


@pytest.mark.parametrize("stride", [(12, 6, 1), (6, 12, 1), (18, 6, 1), (7, 14, 1), (100, 6, 1)])
def test_binding_takes_beams_in_any_order(stride):
    plan = flce._reorder_plan(torch.float32, (2, 2, 6), stride, "d", torch.float32, (2, 2, 6), stride, "d",
                              2, 2, "d", None, 2)
    assert plan == (4 * stride[0], 4 * stride[1], 4 * stride[0], 4 * stride[1], 1, 0, 24)
    # one beam: its stride does not matter
    assert flce._reorder_plan(torch.float32, (2, 1, 6), (6, 0, 1), "d", torch.float32, (2, 1, 6), (6, 0, 1),
                              "d", 2, 1, "d", None, 2) is not None
