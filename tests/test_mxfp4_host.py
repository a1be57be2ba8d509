"""MXFP4 on the CPU: the definition on values worked out by hand, the sizes and
the refusals of the entry points."""
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
    x = np.zeros((1, 40))
    x[0, 0] = 6.0                   # exponent floor(log2 6) - 2 = 0: unit 1
    # ties go to the even code: 0, 1, 1, 2, 2, 4, 4; above 5 rounds to 6
    x[0, 1:9] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.01]
    x[0, 32] = 7.9                  # same binade as 4: saturates at 6
    codes, exps, values = HO.mxfp4(x)
    assert exps.tolist() == [[127, 127]]
    assert values[0, :9].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -6]
    assert codes[0, 8] == 15 and codes[0, 7] == 6 and values[0, 32] == 6.0
    # a zero block has the smallest scale; the smallest numbers clamp to it
    _, exps, values = HO.mxfp4(np.array([[0.0] * 32 + [2.0 ** -133] * 32 + [np.inf] + [1.0] * 31]))
    assert exps.tolist() == [[0, 0, 255]]
    assert np.all(values[0, :64] == 0) and np.all(np.isnan(values[0, 64:]))


def test_sizes(lib):
    codes, scales = lib.flce_mxfp4_codes_size, lib.flce_mxfp4_scales_size
    assert codes(1, 1) == 16384 and codes(128, 256) == 16384 and codes(129, 257) == 65536
    assert scales(1, 1) == 1024 and scales(128, 256) == 1024 and scales(129, 257) == 4096
    assert codes(0, 8) == 0 and scales(0, 8) == 0
    assert codes(-1, 8) == 0 and scales(4, 0) == 0 and scales(1 << 31, 8) == 0
    assert lib.flce_mxfp4_logits_workspace_size(8, 4096) >= codes(8, 4096) + scales(8, 4096)
    assert lib.flce_mxfp4_logits_workspace_size(-1, 4096) == 0


def _quant(lib, **kw):
    a = dict(x=FAKE, dtype=0, rows=4, cols=64, ld=64, codes=FAKE, scales=FAKE)
    a.update(kw)
    return lib.flce_mxfp4_quantize(*a.values(), None)


def _dequant(lib, **kw):
    a = dict(codes=FAKE, scales=FAKE, rows=4, cols=64, x=FAKE, dtype=0, ld=64)
    a.update(kw)
    return lib.flce_mxfp4_dequantize(*a.values(), None)


@pytest.mark.parametrize("call", [_quant, _dequant])
@pytest.mark.parametrize("bad", [dict(rows=-1), dict(cols=0), dict(ld=63), dict(dtype=2), dict(x=0),
                                 dict(x=FAKE + 1), dict(codes=0), dict(codes=FAKE + 8),
                                 dict(scales=0), dict(scales=FAKE + 4)])
def test_bad_arguments(lib, call, bad):
    assert call(lib, **bad) == 1
    assert call(lib, rows=0, x=0) == 0


def _logits(lib, **kw):
    a = dict(hidden=FAKE, dtype=0, n=4, h=64, ldh=64, codes=FAKE, scales=FAKE, vp=100, v=90, cap=0.0,
             out=FAKE, out_dtype=0, ldo=90, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return lib.flce_mxfp4_logits(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(n=-1), dict(h=0), dict(ldh=63), dict(dtype=5), dict(out_dtype=-1),
                                 dict(vp=0), dict(v=101), dict(cap=-1.0), dict(cap=float("nan")),
                                 dict(cap=float("inf")), dict(cap=1e-45), dict(ldo=89), dict(hidden=0),
                                 dict(hidden=FAKE + 1), dict(codes=0), dict(codes=FAKE + 8),
                                 dict(scales=FAKE + 8), dict(out=0), dict(out=FAKE + 1)])
def test_logits_bad_arguments(lib, bad):
    assert _logits(lib, **bad) == 1


def test_logits_workspace(lib):
    need = lib.flce_mxfp4_logits_workspace_size(4, 64)
    assert _logits(lib, ws=0) == 2 and _logits(lib, ws_bytes=need - 1) == 2
    assert _logits(lib, ws=FAKE + 8) == 2
    assert _logits(lib, n=0, hidden=0, out=0, ws=0) == 0


def test_binding_refuses():
    with pytest.raises(ValueError, match="CUDA"):
        flce.mxfp4_quantize(torch.zeros(4, 64))
    with pytest.raises(TypeError):
        flce.mxfp4_quantize(torch.zeros(4, 64, dtype=torch.float16))
    with pytest.raises(TypeError):
        flce.mxfp4_logits(torch.zeros(4, 64), torch.zeros(100, 64))
