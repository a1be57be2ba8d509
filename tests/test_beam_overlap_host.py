"""beam_reorder refuses states that share bytes with what another one reads or writes.

The addresses here are made up, so a call that is not refused must not find a GPU."""
import ctypes
import random

import pytest
import torch

from lm_head_projection_flce_b200 import build as B
from lm_head_projection_flce_b200 import flce

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: nothing may be launched")
BASE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    B.build()
    return flce.load_library()


def _call(lib, states, parents=8, batch=2, beams=3):
    arr = (flce.BeamState * len(states))(*(flce.BeamState(*s) for s in states))
    return lib.flce_beam_reorder(ctypes.cast(arr, ctypes.c_void_p), len(states), parents, batch, beams, None)


def _state(src, dst, beam=64, batch=3 * 64, outer=1, step=0, inner=64, src_strides=None):
    return (src, dst, *(src_strides or (batch, beam)), batch, beam, outer, step, inner)


def _refused(lib, *states, **kw):
    status = _call(lib, states, **kw)
    assert status in (1, 3, 4)  # not refused: there is no device
    return status == 1


K, V, K2, V2 = (BASE + i * 0x1000 for i in range(4))


def test_lists_of_states(lib):
    assert not _refused(lib, _state(K, K), _state(V, V))              # both in place
    assert not _refused(lib, _state(K, K2), _state(V, V2))            # into second buffers
    assert _refused(lib, _state(K, V), _state(V, K))                  # into one another's
    assert _refused(lib, _state(K, K2), _state(V, K))                 # into what the first one reads
    assert _refused(lib, _state(K, K2), _state(V, K2))                # into the same
    assert _refused(lib, _state(K, K), _state(K, K))                  # twice in place
    assert not _refused(lib, _state(K, K2), _state(K, V2))            # one read by two
    assert not _refused(lib, _state(K, K2, src_strides=(0, 0)))       # one beam's state for all


def test_shifted_into_itself(lib):
    for shift in (1, 63, 64, 65, 6 * 64 - 1):
        assert _refused(lib, _state(K, K + shift)), shift
        assert _refused(lib, _state(K + shift, K)), shift
    assert not _refused(lib, _state(K, K + 6 * 64)) and not _refused(lib, _state(K + 6 * 64, K))


def test_parents(lib):
    assert _refused(lib, _state(K, K), parents=K + 8)
    assert _refused(lib, _state(K, K2), parents=K2 + 6 * 64 - 8)
    assert not _refused(lib, _state(K, K2), parents=K)                # only read
    assert not _refused(lib, _state(K, K), parents=K + 6 * 64)
    assert not _refused(lib, _state(K, K), parents=K - 2 * 3 * 8)


def test_interleaved(lib):
    """Keys and values in one buffer: [B, K, 2, inner], and [B, K, outer, 2, inner]."""
    kv = [_state(K + 64 * i, K + 64 * i, beam=128, batch=384) for i in (0, 1)]
    assert not _refused(lib, *kv)
    assert _refused(lib, kv[0], _state(K + 63, K + 63, beam=128, batch=384))
    kv = [_state(K + 16 * i, K + 16 * i, beam=128, batch=384, outer=4, step=32, inner=16) for i in (0, 1)]
    assert not _refused(lib, *kv)
    assert _refused(lib, kv[0], _state(K + 16, K + 16, beam=128, batch=384, outer=4, step=32, inner=17))
    # beams first, batch inside; and a state in the unfilled part of another
    assert not _refused(lib, *(_state(K + 64 * i, K + 64 * i, beam=256, batch=128) for i in (0, 1)))
    assert not _refused(lib, _state(K, K, beam=128, batch=384, inner=40),
                        _state(K + 40, K + 40, beam=128, batch=384, inner=88))


def _bytes(base, batch_stride, beam_stride, outer, step, inner, batch, beams):
    return {base + b * batch_stride + k * beam_stride + o * step + i for b in range(batch) for k in range(beams)
            for o in range(outer) for i in range(inner)}


def test_against_sets_of_bytes(lib):
    rng = random.Random(5)
    seen = [0, 0]
    for _ in range(3000):
        batch, beams = rng.randint(1, 3), rng.randint(1, 3)
        states, reads, writes = [], [], []
        for _ in range(rng.randint(1, 3)):
            inner, outer = rng.randint(1, 4), rng.randint(1, 3)
            step = inner + rng.randint(0, 6)
            strides = [rng.randint(0, 40) for _ in range(4)]
            src, dst = BASE + rng.randint(0, 120), BASE + rng.randint(0, 120)
            if rng.random() < 0.5:
                dst, strides[2:] = src, strides[:2]
            elif rng.random() < 0.5:
                dst += 400
            states.append((src, dst, *strides, outer, step, inner))
            writes.append(_bytes(dst, *strides[2:], outer, step, inner, batch, beams))
            reads.append(set() if src == dst else _bytes(src, *strides[:2], outer, step, inner, batch, beams))
        reads.append(_bytes(8, 0, 0, 1, 0, 8 * batch * beams, 1, 1))
        bad = any(w & r for w in writes for r in reads) or any(
            writes[i] & writes[j] for i in range(len(writes)) for j in range(i)) or any(
            s[0] == s[1] and s[2:4] != s[4:6] for s in states)  # in place means in place
        assert _refused(lib, *states, batch=batch, beams=beams) == bad, (states, batch, beams)
        seen[bad] += 1
    assert min(seen) > 300
