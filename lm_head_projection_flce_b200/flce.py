"""Python binding of libflce.so: argument marshalling only.

Every step of the loss and its gradient runs in the library's CUDA kernels;
this module checks tensors, allocates outputs and workspace with PyTorch (the
caller's device memory) and passes raw pointers and the current CUDA stream
through ctypes.  If the library is missing it raises: there is no fallback.

Entry points mirror include/flce.h:
  forward(hidden, weight, labels, ...)            -> (loss, lse)
  backward(hidden, weight, labels, lse, grad, ...) -> (dhidden, dweight)
  fused_linear_cross_entropy(...)                  autograd-aware convenience
  layer_norm(...)                                  the final norm, autograd-aware
  mxfp4_quantize(...), mxfp4_logits(...)           the head in 4 bits and its product
  beam_select(...), beam_reorder(...)              beam search behind the head
  CapturedStep, CapturedBeamStep                   a training / decoding step as one graph
with the options of the NeMo-AutoModel loss pages
("nemo_automodel.components.loss.linear_ce", FusedLinearCrossEntropy:
ignore_index=-100, logit_softcapping=0, reduction='sum', num_label_tokens;
"nemo_automodel.components.models.inkling2.loss": unpadded_vocab_size and an
FP32 head rounded to BF16).
"""
from __future__ import annotations

import ctypes
import dataclasses
import os

import torch
from torch.autograd import forward_ad

from . import build as _build

LIB_PATH = _build.LIB_PATH

FLCE_OK = 0
FLCE_ERR_BAD_LABEL = 5
FLCE_ERR_TIMEOUT = 6
FLCE_ERR_BAD_INDEX = 7
STATUS = {0: "FLCE_OK", 1: "FLCE_ERR_INVALID_ARG", 2: "FLCE_ERR_WORKSPACE",
          3: "FLCE_ERR_UNSUPPORTED", 4: "FLCE_ERR_CUDA", 5: "FLCE_ERR_BAD_LABEL",
          6: "FLCE_ERR_TIMEOUT", 7: "FLCE_ERR_BAD_INDEX"}
REDUCTIONS = {"sum": 0, "mean": 1, "none": 2}
FLCE_BWD_HEAD_COPY_VALID = 1
FLCE_FUSED_HEAD_CAST = 2
W_DTYPES = {torch.bfloat16: 0, torch.float32: 1}

_c_i64 = ctypes.c_int64
_c_int = ctypes.c_int
_c_ptr = ctypes.c_void_p
_c_size = ctypes.c_size_t

# name -> (restype, argtypes); the exported C ABI of include/flce.h
SIGNATURES = {
    "flce_workspace_size": (_c_size, [_c_i64, _c_i64, _c_i64, _c_i64, _c_int]),
    "flce_workspace_min_size": (_c_size, [_c_i64, _c_i64, _c_i64, _c_i64, _c_int]),
    "flce_workspace_size_ex": (_c_size, [_c_i64, _c_i64, _c_i64, _c_i64, _c_int, ctypes.c_uint]),
    "flce_workspace_min_size_ex": (_c_size, [_c_i64, _c_i64, _c_i64, _c_i64, _c_int,
                                             ctypes.c_uint]),
    "flce_forward": (_c_int, [_c_ptr, _c_ptr, _c_int, _c_ptr, _c_i64, _c_i64, _c_i64, _c_i64,
                              _c_i64, ctypes.c_float, _c_int, _c_i64, _c_ptr, _c_ptr, _c_ptr,
                              _c_size, _c_ptr]),
    "flce_forward_ex": (_c_int, [_c_ptr, _c_ptr, _c_int, _c_ptr, _c_i64, _c_i64, _c_i64,
                                 _c_i64, _c_i64, ctypes.c_float, _c_int, _c_i64, _c_ptr, _c_ptr,
                                 _c_ptr, _c_size, ctypes.c_uint, _c_ptr]),
    "flce_backward": (_c_int, [_c_ptr, _c_ptr, _c_int, _c_ptr, _c_i64, _c_i64, _c_i64, _c_i64,
                               _c_i64, ctypes.c_float, _c_int, _c_i64, _c_ptr, _c_ptr, _c_ptr,
                               _c_ptr, _c_ptr, _c_size, _c_ptr]),
    "flce_backward_ex": (_c_int, [_c_ptr, _c_ptr, _c_int, _c_ptr, _c_i64, _c_i64, _c_i64,
                                  _c_i64, _c_i64, ctypes.c_float, _c_int, _c_i64, _c_ptr,
                                  _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_size, ctypes.c_uint,
                                  _c_ptr]),
    "flce_get_error": (_c_int, [_c_ptr]),
    "flce_status_string": (ctypes.c_char_p, [_c_int]),
    "flce_flops_fwd_bwd": (ctypes.c_double, [_c_i64, _c_i64, _c_i64]),
    "flce_selftest_gemm": (_c_int, [_c_ptr, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_i64, _c_int,
                                    _c_int, _c_ptr]),
    "flce_selftest_wait_timeout": (_c_int, [ctypes.c_uint, _c_ptr]),
    "flce_forward_noalloc": (_c_int, [_c_ptr, _c_ptr, _c_int, _c_ptr, _c_i64, _c_i64, _c_i64,
                                      _c_i64, _c_i64, ctypes.c_float, _c_int, _c_i64, _c_ptr,
                                      _c_ptr, _c_ptr]),
    "flce_ce_workspace_size": (_c_size, [_c_i64]),
    "flce_ce_forward": (_c_int, [_c_ptr, _c_int, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_i64, _c_i64,
                                 _c_int, _c_i64, _c_ptr, _c_ptr, _c_ptr, _c_size, _c_ptr]),
    "flce_ce_backward": (_c_int, [_c_ptr, _c_int, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_i64, _c_i64,
                                  _c_int, _c_i64, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_size, _c_ptr]),
    "flce_layer_norm_workspace_size": (_c_size, [_c_i64, _c_i64]),
    "flce_layer_norm_forward": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_i64, _c_ptr, _c_ptr,
                                         _c_int, ctypes.c_float, _c_ptr, _c_i64, _c_ptr, _c_ptr,
                                         _c_ptr]),
    "flce_layer_norm_backward": (_c_int, [_c_ptr, _c_i64, _c_ptr, _c_int, _c_i64, _c_i64, _c_i64,
                                          _c_ptr, _c_int, _c_ptr, _c_ptr, _c_ptr, _c_i64, _c_ptr,
                                          _c_ptr, _c_ptr, _c_size, _c_ptr]),
    "flce_mxfp4_codes_size": (_c_size, [_c_i64, _c_i64]),
    "flce_mxfp4_scales_size": (_c_size, [_c_i64, _c_i64]),
    "flce_mxfp4_quantize": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_i64, _c_ptr, _c_ptr,
                                     _c_ptr]),
    "flce_mxfp4_dequantize": (_c_int, [_c_ptr, _c_ptr, _c_i64, _c_i64, _c_ptr, _c_int, _c_i64,
                                       _c_ptr]),
    "flce_mxfp4_logits_workspace_size": (_c_size, [_c_i64, _c_i64]),
    "flce_mxfp4_logits": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_i64, _c_ptr, _c_ptr, _c_i64,
                                   _c_i64, ctypes.c_float, _c_ptr, _c_int, _c_i64, _c_ptr, _c_size,
                                   _c_ptr]),
    "flce_beam_select_workspace_size": (_c_size, [_c_i64, _c_i64, _c_i64, _c_i64]),
    "flce_beam_select": (_c_int, [_c_ptr, _c_int, _c_i64, _c_i64, _c_i64, _c_i64, _c_ptr, _c_ptr,
                                  _c_i64, _c_i64, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_size,
                                  _c_ptr]),
    "flce_beam_reorder": (_c_int, [_c_ptr, _c_i64, _c_ptr, _c_i64, _c_i64, _c_ptr]),
    "flce_launch_count": (ctypes.c_ulonglong, []),
    "flce_profile_start": (_c_int, []),
    "flce_profile_stop": (_c_int, [_c_ptr, _c_int, ctypes.POINTER(_c_int)]),
}


class KernelStat(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", ctypes.c_int64),
                ("total_ms", ctypes.c_double), ("flops", ctypes.c_double),
                ("bytes", ctypes.c_double)]


class BeamState(ctypes.Structure):
    _fields_ = [("src", _c_ptr), ("dst", _c_ptr),
                ("src_batch_stride", _c_i64), ("src_beam_stride", _c_i64),
                ("dst_batch_stride", _c_i64), ("dst_beam_stride", _c_i64),
                ("outer", _c_i64), ("outer_stride", _c_i64), ("inner", _c_i64)]


_LIB = None


class FlceError(RuntimeError):
    def __init__(self, where: str, status: int):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


def load_library() -> ctypes.CDLL:
    """Load libflce.so (built in-tree).  Raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m lm_head_projection_flce_b200.build`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


def _check(where: str, status: int) -> None:
    if status != FLCE_OK:
        raise FlceError(where, status)


# The current stream's handle without building a torch.cuda.Stream around it
# (several microseconds of a small call); newer or older builds of torch that
# lack the function take the long way.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(device: torch.device, stream=None) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _current_raw_stream is not None and device.index is not None:
        return _current_raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _elsewhere(device: torch.device, stream) -> bool:
    """True when a call has to make its tensors' device, or `stream`, current first.
    Entry points then call themselves inside `_on`, so that whatever they allocate
    or copy belongs to that stream as well."""
    return stream is not None or device.index != _current_device()


def _on(device: torch.device, stream=None):
    """Context in which `device` and `stream` (None: the device's current stream)
    are current."""
    if stream is None:
        return torch.cuda.device(device)
    if stream.device != device:
        raise ValueError("stream must belong to the tensors' device")
    return torch.cuda.stream(stream)


def _ptr(t: torch.Tensor | None) -> int:
    """Address for a c_void_p argument (0: none, or nothing in it)."""
    return t.data_ptr() if t is not None and t.numel() > 0 else 0


def _vocab(weight: torch.Tensor, unpadded_vocab: int | None) -> int:
    return weight.shape[0] if unpadded_vocab is None or unpadded_vocab <= 0 else int(unpadded_vocab)


def workspace_size(n_tokens: int, hidden: int, padded_vocab: int, unpadded_vocab: int | None,
                   w_dtype: torch.dtype = torch.bfloat16, minimum: bool = False,
                   fused_head_cast: bool = False) -> int:
    lib = load_library()
    fn = lib.flce_workspace_min_size_ex if minimum else lib.flce_workspace_size_ex
    return int(fn(n_tokens, hidden, padded_vocab, unpadded_vocab or 0, W_DTYPES[w_dtype],
                  FLCE_FUSED_HEAD_CAST if fused_head_cast else 0))


def _prepare(hidden, weight, labels):
    if hidden.dtype != torch.bfloat16:
        raise TypeError("hidden must be bf16")
    if weight.dtype not in W_DTYPES:
        raise TypeError("weight must be bf16 or fp32")
    if labels.dtype != torch.int64:
        raise TypeError("labels must be int64")
    h = hidden.shape[-1]
    hid = hidden.reshape(-1, h)
    lab = labels.reshape(-1)
    if hid.shape[0] != lab.shape[0]:
        raise ValueError("hidden and labels disagree on the number of tokens")
    if weight.dim() != 2 or weight.shape[1] != h:
        raise ValueError("weight must be [vocab, hidden]")
    for t in (hid, weight, lab):
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        if t.device != hid.device or t.device.type != "cuda":
            raise ValueError("tensors must be on one CUDA device")
    return hid, lab


def _workspace(ws, need: int, device) -> tuple[torch.Tensor, int]:
    """The workspace tensor and its size in bytes (any dtype; contiguous, on `device`)."""
    if ws is None:
        need = max(need, 16)
        return torch.empty(need, dtype=torch.uint8, device=device), need
    if ws.device != device or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return ws, ws.numel() * ws.element_size()


def _buffer(t, numel: int, dtype, device, name: str) -> torch.Tensor:
    """A caller-supplied buffer the library reads or writes through a raw pointer:
    it must have exactly the expected dtype, size and device, and be contiguous."""
    if t.dtype != dtype or t.numel() != numel or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {numel} elements on "
                         f"{device}")
    return t


def _forward_outputs(loss, lse, n: int, reduction: str, dev):
    loss_n = n if reduction == "none" else 1
    loss = (torch.empty(loss_n, dtype=torch.float32, device=dev) if loss is None
            else _buffer(loss, loss_n, torch.float32, dev, "loss"))
    lse = (torch.empty(n, dtype=torch.float32, device=dev) if lse is None
           else _buffer(lse, n, torch.float32, dev, "lse"))
    return loss, lse


def forward(hidden, weight, labels, *, ignore_index: int = -100, softcap: float = 0.0,
            unpadded_vocab: int | None = None, reduction: str = "sum",
            num_label_tokens: int | None = None, workspace: torch.Tensor | None = None,
            loss: torch.Tensor | None = None, lse: torch.Tensor | None = None,
            fused_head_cast: bool = False, stream=None):
    """Fused projection + cross entropy.  Returns ``(loss, lse)`` (FP32).

    ``fused_head_cast=True`` (flce_forward_ex with FLCE_FUSED_HEAD_CAST): an
    FP32 head is rounded to BF16 inside the GEMM instead of into a V x H BF16
    copy in the workspace; same results, smaller workspace, slower GEMM.
    """
    lib = load_library()
    hid, lab = _prepare(hidden, weight, labels)
    n, h = hid.shape
    vp = weight.shape[0]
    v = _vocab(weight, unpadded_vocab)
    dev = hid.device
    red = REDUCTIONS[reduction]
    loss, lse = _forward_outputs(loss, lse, n, reduction, dev)
    ws, ws_bytes = _workspace(
        workspace, workspace_size(n, h, vp, v, weight.dtype, fused_head_cast=fused_head_cast), dev)
    st = lib.flce_forward_ex(_ptr(hid), _ptr(weight), W_DTYPES[weight.dtype], _ptr(lab), n, h, vp,
                             v, ignore_index, float(softcap), red, int(num_label_tokens or 0),
                             _ptr(loss), _ptr(lse), _ptr(ws), ws_bytes,
                             FLCE_FUSED_HEAD_CAST if fused_head_cast else 0,
                             _stream_handle(dev, stream))
    _check("flce_forward", st)
    return (loss if reduction == "none" else loss.reshape(())), lse


def _grad_loss(grad_loss, n: int, reduction: str, dev) -> torch.Tensor:
    """The upstream gradient as FP32 on the device: [N] for 'none', else one value."""
    grad = torch.as_tensor(grad_loss).reshape(-1).to(device=dev, dtype=torch.float32).contiguous()
    if grad.numel() != (n if reduction == "none" else 1):
        raise ValueError("grad_loss must have one value per token for reduction='none', "
                         "else one value")
    return grad


def backward(hidden, weight, labels, lse, grad_loss, *, ignore_index: int = -100,
             softcap: float = 0.0, unpadded_vocab: int | None = None, reduction: str = "sum",
             num_label_tokens: int | None = None, workspace: torch.Tensor | None = None,
             dhidden: torch.Tensor | None = None, dweight: torch.Tensor | None = None,
             reuse_head_copy: bool = False, fused_head_cast: bool = False, stream=None):
    """Gradients ``(dhidden [.., H] bf16, dweight [Vp, H] in the head's dtype)``.

    ``reuse_head_copy=True`` (flce_backward_ex with FLCE_BWD_HEAD_COPY_VALID):
    for an FP32 head, skip the FP32 -> BF16 cast and use the copy that
    ``forward`` wrote into the same ``workspace`` -- the caller promises that
    the head and that workspace are unchanged since.  Needs ``workspace``;
    ignored for a BF16 head.

    ``fused_head_cast=True`` (FLCE_FUSED_HEAD_CAST): the recompute and
    dhidden GEMMs round an FP32 head to BF16 inside the kernel; no copy is
    read or written.  Not combinable with ``reuse_head_copy``.
    """
    lib = load_library()
    hid, lab = _prepare(hidden, weight, labels)
    n, h = hid.shape
    vp = weight.shape[0]
    v = _vocab(weight, unpadded_vocab)
    dev = hid.device
    red = REDUCTIONS[reduction]
    grad = _grad_loss(grad_loss, n, reduction, dev)
    lse = _buffer(lse, n, torch.float32, dev, "lse")
    dhidden = (torch.empty_like(hid) if dhidden is None
               else _buffer(dhidden, n * h, torch.bfloat16, dev, "dhidden"))
    dweight = (torch.empty_like(weight) if dweight is None
               else _buffer(dweight, weight.numel(), weight.dtype, dev, "dweight"))
    if reuse_head_copy and workspace is None:
        raise ValueError("reuse_head_copy needs the workspace the forward wrote the copy into")
    if reuse_head_copy and fused_head_cast:
        raise ValueError("fused_head_cast writes no head copy to reuse")
    ws, ws_bytes = _workspace(
        workspace, workspace_size(n, h, vp, v, weight.dtype, fused_head_cast=fused_head_cast), dev)
    flags = (FLCE_BWD_HEAD_COPY_VALID if reuse_head_copy else 0) | (
        FLCE_FUSED_HEAD_CAST if fused_head_cast else 0)
    st = lib.flce_backward_ex(_ptr(hid), _ptr(weight), W_DTYPES[weight.dtype], _ptr(lab), n, h,
                              vp, v, ignore_index, float(softcap), red, int(num_label_tokens or 0),
                              _ptr(grad), _ptr(lse), _ptr(dhidden), _ptr(dweight), _ptr(ws),
                              ws_bytes, flags, _stream_handle(dev, stream))
    _check("flce_backward", st)
    return dhidden.reshape(hidden.shape), dweight


def get_error(device=None, stream=None) -> int:
    """Synchronise and read-and-clear the device error word (FLCE_* status)."""
    lib = load_library()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        return int(lib.flce_get_error(_stream_handle(dev, stream)))


def selftest_gemm(a, b, m: int, n: int, k: int, a_mn: bool, b_mn: bool) -> torch.Tensor:
    """D = A . B^T through the library's tensor-core GEMM (tests only)."""
    lib = load_library()
    d = torch.empty(m, n, dtype=torch.float32, device=a.device)
    st = lib.flce_selftest_gemm(_ptr(a), _ptr(b), _ptr(d), m, n, k, int(a_mn), int(b_mn),
                                _stream_handle(a.device))
    _check("flce_selftest_gemm", st)
    return d


def selftest_wait_timeout(timeout_us: int, device=None) -> None:
    lib = load_library()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    _check("flce_selftest_wait_timeout",
           lib.flce_selftest_wait_timeout(timeout_us, _stream_handle(dev)))


class _FusedLinearCE(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, labels, ignore_index, softcap, unpadded_vocab, reduction,
                num_label_tokens, fused_head_cast):
        # An FP32 head's BF16 copy, made by the forward, is kept (in the
        # workspace) for the backward instead of being cast again; autograd's
        # version check refuses a backward after the head changed in place.
        # With fused_head_cast there is no copy and nothing is kept.
        ws = None
        if weight.dtype == torch.float32 and not fused_head_cast:
            hid = hidden.reshape(-1, hidden.shape[-1])
            need = workspace_size(hid.shape[0], hid.shape[1], weight.shape[0],
                                  _vocab(weight, unpadded_vocab), weight.dtype)
            ws = torch.empty(max(need, 16), dtype=torch.uint8, device=hidden.device)
        loss, lse = forward(hidden, weight, labels, ignore_index=ignore_index, softcap=softcap,
                            unpadded_vocab=unpadded_vocab, reduction=reduction,
                            num_label_tokens=num_label_tokens, workspace=ws,
                            fused_head_cast=fused_head_cast)
        ctx.save_for_backward(hidden, weight, labels, lse)
        ctx.workspace = ws
        ctx.opts = (ignore_index, softcap, unpadded_vocab, reduction, num_label_tokens,
                    fused_head_cast)
        return loss

    @staticmethod
    def backward(ctx, grad_out):
        hidden, weight, labels, lse = ctx.saved_tensors
        ii, c, uv, red, nlt, fused = ctx.opts
        ws = ctx.workspace
        ctx.workspace = None
        dh, dw = backward(hidden, weight, labels, lse, grad_out, ignore_index=ii, softcap=c,
                          unpadded_vocab=uv, reduction=red, num_label_tokens=nlt, workspace=ws,
                          reuse_head_copy=ws is not None, fused_head_cast=fused)
        return dh, dw, None, None, None, None, None, None, None


def fused_linear_cross_entropy(hidden, weight, labels, *, ignore_index: int = -100,
                               softcap: float = 0.0, unpadded_vocab: int | None = None,
                               reduction: str = "sum", num_label_tokens: int | None = None,
                               fused_head_cast: bool = False, norm_weight=None, norm_bias=None,
                               norm_eps: float = 1e-5):
    """Autograd-aware loss: gradients flow to ``hidden`` and ``weight``.

    With ``norm_weight`` and / or ``norm_bias`` ([H]), ``hidden`` is what enters
    the final layer norm: it is normalised by ``layer_norm(hidden, norm_weight,
    norm_bias, eps=norm_eps)`` first, and gradients flow to those two as well.

    With an FP32 head the forward's workspace (which holds the head's BF16
    copy, V x H x 2 bytes, and the backward's buffers) is kept until the
    backward runs, so the head is cast once per step; a BF16 head keeps
    nothing between the two.  ``fused_head_cast=True`` rounds an FP32 head
    inside the GEMMs instead: no copy exists and nothing is kept (less memory,
    slower GEMMs, the same results).
    """
    if norm_weight is not None or norm_bias is not None:
        hidden = layer_norm(hidden, norm_weight, norm_bias, eps=norm_eps)
    return _FusedLinearCE.apply(hidden, weight, labels, ignore_index, softcap, unpadded_vocab,
                                reduction, num_label_tokens, fused_head_cast)


class CapturedStep:
    """Forward + backward of the fused loss captured once into a CUDA graph.

    The inputs are static device tensors owned here (``hidden``, ``labels``,
    and the head ``weight`` the caller passes, which must stay alive and keep
    its storage); a step copies new values into them (``set_inputs``) and
    calls ``replay()``, which reruns all of the step's kernel launches as one
    graph launch.  Outputs (``loss``, ``lse``, ``dhidden``, ``dweight``) are static
    too and are overwritten by each replay.  Worth it where a step is short
    enough for launch overhead to show (small batches); the results equal the
    eager calls bit for bit.

    The options, ``num_label_tokens`` included, are host values baked into
    the graph when it is captured: a replay normalises by the count given at
    construction even if ``set_inputs`` brought labels with another number of
    live tokens.  ``set_inputs(..., num_label_tokens=k)`` refuses a ``k`` that
    differs from the captured one; build a new CapturedStep for it.
    An FP32 head is cast to BF16 once per replay (the backward reuses the
    forward's copy).
    """

    def __init__(self, hidden, weight, labels, *, ignore_index: int = -100, softcap: float = 0.0,
                 unpadded_vocab: int | None = None, reduction: str = "sum",
                 num_label_tokens: int | None = None, grad_loss=None):
        hid, lab = _prepare(hidden, weight, labels)
        dev = hid.device
        n, h = hid.shape
        self.hidden = hid.clone()
        self.labels = lab.clone()
        self.weight = weight
        self.kw = dict(ignore_index=ignore_index, softcap=softcap, unpadded_vocab=unpadded_vocab,
                       reduction=reduction, num_label_tokens=num_label_tokens)
        v = _vocab(weight, unpadded_vocab)
        self.workspace = torch.empty(max(workspace_size(n, h, weight.shape[0], v, weight.dtype), 16),
                                     dtype=torch.uint8, device=dev)
        self.loss = torch.empty(n if reduction == "none" else 1, dtype=torch.float32, device=dev)
        self.lse = torch.empty(n, dtype=torch.float32, device=dev)
        self.dhidden = torch.empty_like(self.hidden)
        self.dweight = torch.empty_like(weight)
        g = torch.ones(()) if grad_loss is None else grad_loss
        self.grad = _grad_loss(g, n, reduction, dev).clone()
        stream = torch.cuda.Stream(dev)
        stream.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(stream):
            self._step()          # eager: per-device set-up and launch shapes, outside capture
        torch.cuda.current_stream(dev).wait_stream(stream)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=stream):
            self._step()

    def _step(self):
        forward(self.hidden, self.weight, self.labels, loss=self.loss, lse=self.lse,
                workspace=self.workspace, **self.kw)
        backward(self.hidden, self.weight, self.labels, self.lse, self.grad,
                 dhidden=self.dhidden, dweight=self.dweight, workspace=self.workspace,
                 reuse_head_copy=self.weight.dtype == torch.float32, **self.kw)

    def set_inputs(self, hidden=None, labels=None, num_label_tokens: int | None = None) -> None:
        """Copy new token data into the captured input buffers (same shapes).

        ``num_label_tokens``, if given, must equal the value captured at
        construction (it is fixed inside the graph); anything else raises.
        """
        if num_label_tokens is not None and num_label_tokens != self.kw["num_label_tokens"]:
            raise ValueError(f"num_label_tokens={num_label_tokens} differs from the captured "
                             f"{self.kw['num_label_tokens']}; it is fixed when the graph is "
                             "captured")
        if hidden is not None:
            self.hidden.copy_(hidden.reshape(self.hidden.shape), non_blocking=True)
        if labels is not None:
            self.labels.copy_(labels.reshape(self.labels.shape), non_blocking=True)

    def replay(self):
        """Run forward + backward; returns (loss, dhidden, dweight), static buffers."""
        self.graph.replay()
        loss = self.loss if self.kw["reduction"] == "none" else self.loss.reshape(())
        return loss, self.dhidden, self.dweight


def launch_count() -> int:
    """Kernels the library has launched in this process."""
    return int(load_library().flce_launch_count())


def profile_start() -> None:
    """Bracket every library kernel launch with CUDA events until profile_stop()."""
    _check("flce_profile_start", load_library().flce_profile_start())


def profile_stop() -> dict:
    """Per kernel family: launches, device ms (CUDA events) and algorithmic work."""
    lib = load_library()
    cap = 32
    arr = (KernelStat * cap)()
    count = _c_int(0)
    _check("flce_profile_stop", lib.flce_profile_stop(ctypes.cast(arr, _c_ptr), cap,
                                                       ctypes.byref(count)))
    out = {}
    for i in range(min(count.value, cap)):
        st = arr[i]
        out[st.name.decode()] = {"launches": int(st.launches), "total_ms": float(st.total_ms),
                                 "flops": float(st.flops), "bytes": float(st.bytes)}
    return out


def forward_noalloc(hidden, weight, labels, *, ignore_index: int = -100, softcap: float = 0.0,
                    unpadded_vocab: int | None = None, reduction: str = "sum",
                    num_label_tokens: int | None = None, loss: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, stream=None):
    """flce_forward_noalloc: the forward with the library's fixed 32 MiB device
    scratch instead of a workspace, for callers that cannot provide scratch
    memory.  Only the outputs are allocated here (when not given)."""
    lib = load_library()
    hid, lab = _prepare(hidden, weight, labels)
    n, h = hid.shape
    vp = weight.shape[0]
    v = _vocab(weight, unpadded_vocab)
    dev = hid.device
    loss, lse = _forward_outputs(loss, lse, n, reduction, dev)
    st = lib.flce_forward_noalloc(_ptr(hid), _ptr(weight), W_DTYPES[weight.dtype], _ptr(lab), n,
                                  h, vp, v, ignore_index, float(softcap), REDUCTIONS[reduction],
                                  int(num_label_tokens or 0), _ptr(loss), _ptr(lse),
                                  _stream_handle(dev, stream))
    _check("flce_forward_noalloc", st)
    return (loss if reduction == "none" else loss.reshape(())), lse


# ---------------------------------------------------------------- cross entropy on given logits

def _prepare_logits(logits, labels, mask):
    if logits.dtype not in W_DTYPES:
        raise TypeError("logits must be bf16 or fp32")
    if labels.dtype != torch.int64:
        raise TypeError("labels must be int64")
    v = logits.shape[-1]
    z = logits.reshape(-1, v)
    lab = labels.reshape(-1)
    if z.shape[0] != lab.shape[0]:
        raise ValueError("logits and labels disagree on the number of tokens")
    if z.stride(-1) != 1 or not lab.is_contiguous():
        raise ValueError("logits rows and labels must be contiguous")
    m = None
    if mask is not None:
        m = mask.reshape(-1).to(torch.uint8).contiguous()
        if m.shape[0] != lab.shape[0]:
            raise ValueError("mask must match labels")
    for t in (z, lab) + ((m,) if m is not None else ()):
        if t.device.type != "cuda" or t.device != z.device:
            raise ValueError("tensors must be on one CUDA device")
    return z, lab, m


def ce_forward(logits, labels, *, mask=None, ignore_index: int = -100, reduction: str = "sum",
               num_label_tokens: int | None = None, workspace=None,
               loss: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None):
    """Cross entropy of given logits [..., V] (ChunkedCrossEntropy).  Returns (loss, lse)."""
    lib = load_library()
    z, lab, m = _prepare_logits(logits, labels, mask)
    n, v = z.shape
    dev = z.device
    loss, lse = _forward_outputs(loss, lse, n, reduction, dev)
    ws, ws_bytes = _workspace(workspace, int(lib.flce_ce_workspace_size(n)), dev)
    st = lib.flce_ce_forward(_ptr(z), W_DTYPES[z.dtype], _ptr(lab), _ptr(m), n, v, z.stride(0),
                             ignore_index, REDUCTIONS[reduction], int(num_label_tokens or 0),
                             _ptr(loss), _ptr(lse), _ptr(ws), ws_bytes, _stream_handle(dev, stream))
    _check("flce_ce_forward", st)
    return (loss if reduction == "none" else loss.reshape(())), lse


def ce_backward(logits, labels, lse, grad_loss, *, mask=None, ignore_index: int = -100,
                reduction: str = "sum", num_label_tokens: int | None = None, dlogits=None,
                workspace=None, stream=None):
    """Gradient w.r.t. the logits, in the logits' dtype and shape."""
    lib = load_library()
    z, lab, m = _prepare_logits(logits, labels, mask)
    n, v = z.shape
    dev = z.device
    grad = _grad_loss(grad_loss, n, reduction, dev)
    lse = _buffer(lse, n, torch.float32, dev, "lse")
    if dlogits is None:
        # the kernels write dlogits with the logits' row stride
        dlogits = torch.empty(n, z.stride(0), dtype=z.dtype, device=dev)[:, :v]
    out = dlogits.reshape(n, v)
    if out.dtype != z.dtype or out.device != dev:
        raise ValueError("dlogits must have the logits' dtype and device")
    if out.stride(0) != z.stride(0) or out.stride(1) != 1:
        raise ValueError("dlogits must have the logits' row stride")
    ws, ws_bytes = _workspace(workspace, int(lib.flce_ce_workspace_size(n)), dev)
    st = lib.flce_ce_backward(_ptr(z), W_DTYPES[z.dtype], _ptr(lab), _ptr(m), n, v, z.stride(0),
                              ignore_index, REDUCTIONS[reduction], int(num_label_tokens or 0),
                              _ptr(grad), _ptr(lse), _ptr(out), _ptr(ws), ws_bytes,
                              _stream_handle(dev, stream))
    _check("flce_ce_backward", st)
    return out.reshape(logits.shape)


# ---------------------------------------------------------------- layer norm

def _rows(t, h: int, name: str) -> tuple[torch.Tensor, int, int]:
    """`t` [..., h] as N rows of unit stride: a tensor that starts with the first of
    them, N, and their distance in elements."""
    if t.is_contiguous():
        return t, t.numel() // h, h
    rows = t if t.dim() == 2 else t.reshape(-1, h)
    n = rows.shape[0]
    step, unit = rows.stride()
    if unit != 1 and h > 1:
        raise ValueError(f"{name} rows must be contiguous")
    if n <= 1:
        return rows, n, h
    if step < h:
        raise ValueError(f"{name} rows must not overlap")
    return rows, n, step


def _cuda_tensor(t, dtypes, dev, name: str) -> None:
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {tuple(dtypes)}")
    if not t.is_cuda or (dev is not None and t.device != dev):
        raise ValueError("tensors must be on one CUDA device")


def _result(t, like, shape, dtype, name: str) -> torch.Tensor:
    """The caller's output tensor, checked, or a new one on `like`'s device."""
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    if t.shape != torch.Size(shape) or t.dtype != dtype or t.device != like.device:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {like.device}")
    return t


def _result_rows(t, h: int, name: str) -> tuple[int, int]:
    """Address and row distance of an output, which must be rows of one stride in place."""
    rows, _, ld = _rows(t, h, name)
    if rows is not t and rows.data_ptr() != t.data_ptr():
        raise ValueError(f"{name}'s rows must have one stride")
    return _ptr(rows), ld


def _norm_params(weight, bias, h: int, dev, param_dtype=None) -> torch.dtype:
    """The parameters' common dtype, after checking them."""
    dtype = param_dtype
    for p in (weight, bias):
        if p is None:
            continue
        if dtype is None:
            dtype = p.dtype
        elif p.dtype != dtype:
            raise TypeError("weight, bias and param_dtype must be one dtype")
        if p.dim() != 1 or p.shape[0] != h or not p.is_contiguous():
            raise ValueError("weight and bias must be contiguous [hidden] tensors")
        if p.device != dev:
            raise ValueError("tensors must be on one CUDA device")
    if dtype is None:
        return torch.float32
    if dtype not in W_DTYPES:
        raise TypeError("weight and bias must be bf16 or fp32")
    return dtype


def _norm_input(x) -> None:
    _cuda_tensor(x, W_DTYPES, None, "x")
    if x.dim() == 0 or x.shape[-1] == 0:
        raise ValueError("x must be [..., hidden] with hidden >= 1")


def layer_norm_forward(x, weight=None, bias=None, *, eps: float = 1e-5,
                       y: torch.Tensor | None = None, mean: torch.Tensor | None = None,
                       rstd: torch.Tensor | None = None, stats: bool = True, stream=None):
    """Layer norm over the last dimension (flce_layer_norm_forward).

    ``x`` [..., H] bf16 or fp32 (rows contiguous, any row stride); ``weight`` and
    ``bias`` [H] bf16 or fp32, either may be None.  Returns ``(y, mean, rstd)``:
    y in x's dtype and shape, the row statistics FP32 [N] for the backward
    (``stats=False``: None for statistics that were not given, and not written).
    Outputs given may not share memory with inputs or one another: refused.
    """
    lib = _LIB or load_library()
    _norm_input(x)
    dev = x.device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return layer_norm_forward(x, weight, bias, eps=eps, y=y, mean=mean, rstd=rstd,
                                      stats=stats)
    h = x.shape[-1]
    rows, n, ldx = _rows(x, h, "x")
    w_dtype = _norm_params(weight, bias, h, dev)
    if y is None:
        y = x.new_empty(x.shape)
        out, ldy = y.data_ptr(), h
    else:
        _result(y, x, x.shape, x.dtype, "y")
        out, ldy = _result_rows(y, h, "y")
    if mean is not None:
        _buffer(mean, n, torch.float32, dev, "mean")
    elif stats:
        mean = x.new_empty(n, dtype=torch.float32)
    if rstd is not None:
        _buffer(rstd, n, torch.float32, dev, "rstd")
    elif stats:
        rstd = x.new_empty(n, dtype=torch.float32)
    st = lib.flce_layer_norm_forward(rows.data_ptr(), W_DTYPES[x.dtype], n, h, ldx, _ptr(weight),
                                     _ptr(bias), W_DTYPES[w_dtype], eps, out, ldy, _ptr(mean),
                                     _ptr(rstd), _stream_handle(dev))
    if st != FLCE_OK:
        raise FlceError("flce_layer_norm_forward", st)
    return y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None, *, want=("dx", "dweight", "dbias"),
                        param_dtype: torch.dtype | None = None, dx: torch.Tensor | None = None,
                        dweight: torch.Tensor | None = None, dbias: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, stream=None):
    """Gradients ``(dx, dweight, dbias)`` of layer_norm_forward; None for what is
    not in ``want``.  ``dx`` has x's dtype, the other two the weight's
    (``param_dtype`` where there is no weight; FP32 by default)."""
    lib = _LIB or load_library()
    _norm_input(x)
    dev = x.device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return layer_norm_backward(dy, x, mean, rstd, weight, want=want,
                                       param_dtype=param_dtype, dx=dx, dweight=dweight,
                                       dbias=dbias, workspace=workspace)
    h = x.shape[-1]
    rows, n, ldx = _rows(x, h, "x")
    unknown = set(want) - {"dx", "dweight", "dbias"}
    if unknown:
        raise ValueError(f"unknown gradients {sorted(unknown)}")
    _cuda_tensor(dy, (x.dtype,), dev, "dy")
    if dy.shape != x.shape:
        raise ValueError("dy must have x's shape")
    w_dtype = _norm_params(weight, None, h, dev, param_dtype)
    grads, _, lddy = _rows(dy, h, "dy")
    _buffer(mean, n, torch.float32, dev, "mean")
    _buffer(rstd, n, torch.float32, dev, "rstd")
    lddx = h
    if "dx" in want:
        dx = _result(dx, x, x.shape, x.dtype, "dx")
        _, lddx = _result_rows(dx, h, "dx")
    else:
        dx = None
    if "dweight" in want:
        dweight = (x.new_empty(h, dtype=w_dtype) if dweight is None
                   else _buffer(dweight, h, w_dtype, dev, "dweight"))
    else:
        dweight = None
    if "dbias" in want:
        dbias = (x.new_empty(h, dtype=w_dtype) if dbias is None
                 else _buffer(dbias, h, w_dtype, dev, "dbias"))
    else:
        dbias = None
    _norm_grads(lib, grads, lddy, rows, n, h, ldx, weight, w_dtype, mean, rstd, dx, lddx, dweight,
                dbias, workspace, _stream_handle(dev))
    return dx, dweight, dbias


def _norm_grads(lib, dy, lddy, x, n, h, ldx, weight, w_dtype, mean, rstd, dx, lddx, dweight, dbias,
                workspace, stream) -> None:
    """flce_layer_norm_backward on checked tensors."""
    ws, ws_bytes = None, 0
    if dweight is not None or dbias is not None:
        ws, ws_bytes = _workspace(workspace, lib.flce_layer_norm_workspace_size(n, h), x.device)
    st = lib.flce_layer_norm_backward(_ptr(dy), lddy, _ptr(x), W_DTYPES[x.dtype], n, h, ldx,
                                      _ptr(weight), W_DTYPES[w_dtype], _ptr(mean), _ptr(rstd),
                                      _ptr(dx), lddx, _ptr(dweight), _ptr(dbias), _ptr(ws),
                                      ws_bytes, stream)
    _check("flce_layer_norm_backward", st)


def _has_tangent(*tensors) -> bool:
    """True when one of the tensors carries a forward-mode derivative."""
    if getattr(forward_ad, "_current_level", 0) < 0:  # outside every dual level: none does
        return False
    return any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps=eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.w_dtype = (weight if weight is not None else x if bias is None else bias).dtype
        return y

    @staticmethod
    def backward(ctx, dy):
        if torch.is_grad_enabled():
            raise RuntimeError("layer_norm's gradient has no gradient of its own (create_graph)")
        if _has_tangent(dy):
            raise NotImplementedError("layer_norm's gradient has no forward-mode derivative")
        # What the forward checked is not checked again: this runs in autograd's own
        # thread, where a small call's time is mostly Python.
        x, weight, mean, rstd = ctx.saved_tensors
        dev = x.device
        if _elsewhere(dev, None):
            with _on(dev):
                return _LayerNorm._grads(ctx, dy, x, weight, mean, rstd)
        return _LayerNorm._grads(ctx, dy, x, weight, mean, rstd)

    @staticmethod
    def _grads(ctx, dy, x, weight, mean, rstd):
        need_x, need_w, need_b, _ = ctx.needs_input_grad
        h = x.shape[-1]
        dy = dy.contiguous()  # a gradient that autograd broadcast (a sum's) has rows of stride 0
        rows, n, ldx = _rows(x, h, "x")
        dx = x.new_empty(x.shape) if need_x else None
        dw = x.new_empty(h, dtype=ctx.w_dtype) if need_w else None
        db = x.new_empty(h, dtype=ctx.w_dtype) if need_b else None
        _norm_grads(_LIB, dy, h, rows, n, h, ldx, weight, ctx.w_dtype, mean, rstd, dx, h, dw, db,
                    None, _stream_handle(x.device))
        return dx, dw, db, None


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5):
    """Autograd-aware layer norm over the last dimension: ``(x - mean) * rstd *
    weight + bias``; gradients flow to ``x``, ``weight`` and ``bias``.  Reverse mode and
    once only: tensors with a forward-mode tangent are refused."""
    if not (torch.is_grad_enabled() and (x.requires_grad
                                         or (weight is not None and weight.requires_grad)
                                         or (bias is not None and bias.requires_grad))
            or _has_tangent(x, weight, bias)):
        return layer_norm_forward(x, weight, bias, eps=eps, stats=False)[0]
    return _LayerNorm.apply(x, weight, bias, eps)


# ---------------------------------------------------------------- the head in MXFP4

@dataclasses.dataclass(frozen=True, eq=False)
class Mxfp4:
    """A matrix [rows, cols] in microscaled 4-bit floating point (see include/flce.h):
    ``codes`` uint8, two E2M1 codes per byte, in tiles of 128 rows x 256 columns, and
    ``scales`` uint8, one E8M0 exponent per 32 columns, in tiles of 128 rows x 4
    blocks, both as the tensor core reads them."""

    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int

    def __post_init__(self):
        lib = _LIB or load_library()
        if self.codes.device.type != "cuda":
            raise ValueError("tensors must be on one CUDA device")
        for t, size, name in ((self.codes, lib.flce_mxfp4_codes_size, "codes"),
                              (self.scales, lib.flce_mxfp4_scales_size, "scales")):
            _buffer(t, size(self.rows, self.cols), torch.uint8, self.codes.device, name)

    @property
    def shape(self) -> tuple[int, int]:
        return self.rows, self.cols

    @property
    def device(self) -> torch.device:
        return self.codes.device

    def element_codes(self) -> torch.Tensor:
        """The 4-bit codes (sign and E2M1 index) as uint8 [rows, cols] (a copy in row order)."""
        t = self.codes.view(-(-self.rows // 128), -(-self.cols // 256), 16, 8, 8, 16)
        row = torch.arange(8, device=t.device)[:, None]
        t = t[:, :, :, row, row ^ torch.arange(8, device=t.device)]  # undo the swizzle of a row's 16-byte pieces
        t = t.permute(0, 2, 3, 1, 4, 5).reshape(-(-self.rows // 128) * 128, -1)
        return torch.stack([t & 15, t >> 4], dim=-1).view(t.shape[0], -1)[:self.rows, :self.cols].contiguous()

    def block_exponents(self) -> torch.Tensor:
        """The biased exponents as [rows, ceil(cols / 32)] (a copy in row order)."""
        tiles = -(-self.rows // 128), 2 * -(-self.cols // 256)
        t = self.scales.view(*tiles, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(tiles[0] * 128, -1)
        return t[:self.rows, :-(-self.cols // 32)].contiguous()


def _mxfp4_operand(q: Mxfp4, name: str) -> None:
    if not isinstance(q, Mxfp4):
        raise TypeError(f"{name} must be an Mxfp4 (from mxfp4_quantize)")


def mxfp4_quantize(x, *, out: Mxfp4 | None = None, stream=None) -> Mxfp4:
    """``x`` [rows, cols] (bf16 or fp32, contiguous rows) in MXFP4: per 32 columns the
    power of two 2^(floor(log2 max|x|) - 2), elements rounded to the nearest E2M1
    number (ties to even, saturating).  ``out`` is overwritten if given.  No gradient
    flows through it."""
    lib = _LIB or load_library()
    _cuda_tensor(x, W_DTYPES, None, "x")
    if x.dim() != 2 or x.shape[1] == 0:
        raise ValueError("x must be [rows, cols] with cols >= 1")
    n, h = x.shape
    dev = x.device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return mxfp4_quantize(x, out=out)
    rows, _, ld = _rows(x, h, "x")
    if out is None:
        codes = x.new_empty(lib.flce_mxfp4_codes_size(n, h), dtype=torch.uint8)
        scales = x.new_empty(lib.flce_mxfp4_scales_size(n, h), dtype=torch.uint8)
        out = object.__new__(Mxfp4)  # nothing to check in buffers made here
        out.__dict__.update(codes=codes, scales=scales, rows=n, cols=h)
    else:
        _mxfp4_operand(out, "out")
        if out.shape != (n, h) or out.device != dev:
            raise ValueError("out must have x's shape and device")
    st = lib.flce_mxfp4_quantize(rows.data_ptr(), W_DTYPES[x.dtype], n, h, ld, out.codes.data_ptr(),
                                 out.scales.data_ptr(), _stream_handle(dev))
    _check("flce_mxfp4_quantize", st)
    return out


def mxfp4_dequantize(q: Mxfp4, dtype: torch.dtype = torch.bfloat16, *,
                     out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The numbers ``q`` stands for, [rows, cols] in bf16 or fp32 (both hold them exactly)."""
    lib = _LIB or load_library()
    _mxfp4_operand(q, "q")
    if dtype not in W_DTYPES:
        raise TypeError("dtype must be bf16 or fp32")
    dev = q.device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return mxfp4_dequantize(q, dtype, out=out)
    out = _result(out, q.codes, q.shape, dtype, "out")
    rows, ld = _result_rows(out, q.cols, "out")
    st = lib.flce_mxfp4_dequantize(q.codes.data_ptr(), q.scales.data_ptr(), q.rows, q.cols, rows,
                                   W_DTYPES[dtype], ld, _stream_handle(dev))
    _check("flce_mxfp4_dequantize", st)
    return out


def mxfp4_logits(hidden, head: Mxfp4, *, softcap: float = 0.0, unpadded_vocab: int | None = None,
                 dtype: torch.dtype = torch.bfloat16, logits: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``softcap * tanh(z / softcap)`` (softcap 0: ``z``) of ``z = q(hidden) . head^T``,
    [..., V] in ``dtype``: the hidden states [..., H] (bf16 or fp32) are put into MXFP4
    in the workspace, the product runs on 4-bit tensor cores with FP32 accumulation.
    For serving and evaluation: no gradient flows through it."""
    lib = _LIB or load_library()
    _mxfp4_operand(head, "head")
    _cuda_tensor(hidden, W_DTYPES, head.device, "hidden")
    if dtype not in W_DTYPES:
        raise TypeError("dtype must be bf16 or fp32")
    if hidden.dim() == 0 or hidden.shape[-1] != head.cols:
        raise ValueError("hidden must be [..., H] with the head's H")
    dev, h, vp = hidden.device, head.cols, head.rows
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return mxfp4_logits(hidden, head, softcap=softcap, unpadded_vocab=unpadded_vocab,
                                dtype=dtype, logits=logits, workspace=workspace)
    v = vp if unpadded_vocab is None or unpadded_vocab <= 0 else int(unpadded_vocab)
    rows, n, ldh = _rows(hidden, h, "hidden")
    shape = (*hidden.shape[:-1], v)
    if logits is None:
        logits = hidden.new_empty(shape, dtype=dtype)
        out, ldo = logits.data_ptr(), v
    else:
        _result(logits, hidden, shape, dtype, "logits")
        out, ldo = _result_rows(logits, v, "logits")
    ws, ws_bytes = _workspace(workspace, lib.flce_mxfp4_logits_workspace_size(n, h), dev)
    st = lib.flce_mxfp4_logits(rows.data_ptr(), W_DTYPES[hidden.dtype], n, h, ldh,
                               head.codes.data_ptr(), head.scales.data_ptr(), vp, v, softcap, out,
                               W_DTYPES[dtype], ldo, ws.data_ptr(), ws_bytes, _stream_handle(dev))
    _check("flce_mxfp4_logits", st)
    return logits


# ---------------------------------------------------------------- beam search

def beam_select(logits, scores, *, num_select: int | None = None, finished=None,
                eos_token: int | None = None, unpadded_vocab: int | None = None,
                workspace: torch.Tensor | None = None, stream=None):
    """The ``num_select`` (default: as many as beams) best continuations of each item.

    ``logits`` [B, K, V'] (bf16 or fp32; the first ``unpadded_vocab`` of V' count),
    ``scores`` FP32 [B, K] cumulative log-probabilities; a candidate's score is
    ``scores + log_softmax(logits)``.  A beam whose score is not finite has no
    candidates.  ``finished`` [B, K] (bool or uint8, with ``eos_token``): such a beam
    continues with ``eos_token`` alone, its score unchanged.  Returns ``(scores FP32,
    parents int64, tokens int64)``, each [B, num_select], best first, ties to the lowest
    ``parent * V + token``; where too few candidates are above -inf, the lowest unused
    ones with score -inf.
    """
    lib = _LIB or load_library()
    _cuda_tensor(logits, W_DTYPES, None, "logits")
    if logits.dim() != 3 or 0 in logits.shape[1:]:
        raise ValueError("logits must be [batch, beams, vocab]")
    b, k, vp = logits.shape
    v = vp if unpadded_vocab is None or unpadded_vocab <= 0 else int(unpadded_vocab)
    if v > vp:
        raise ValueError("unpadded_vocab exceeds the logits' vocabulary")
    dev = logits.device
    _cuda_tensor(scores, (torch.float32,), dev, "scores")
    if scores.shape != (b, k) or not scores.is_contiguous():
        raise ValueError("scores must be a contiguous [batch, beams] tensor")
    if (finished is None) != (eos_token is None):
        raise ValueError("finished and eos_token go together")
    m = k if num_select is None else int(num_select)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return beam_select(logits, scores, num_select=num_select, finished=finished,
                               eos_token=eos_token, unpadded_vocab=unpadded_vocab,
                               workspace=workspace)
    rows, _, ld = _rows(logits, vp, "logits")
    done = 0
    if finished is not None:
        _cuda_tensor(finished, (torch.bool, torch.uint8), dev, "finished")
        if finished.shape != (b, k) or not finished.is_contiguous():
            raise ValueError("finished must be a contiguous [batch, beams] tensor")
        done = finished.data_ptr()
    out = scores.new_empty((b, m))
    parents = scores.new_empty((b, m), dtype=torch.int64)
    tokens = torch.empty_like(parents)
    ws, ws_bytes = _workspace(workspace, lib.flce_beam_select_workspace_size(b, k, v, m), dev)
    st = lib.flce_beam_select(rows.data_ptr(), W_DTYPES[logits.dtype], b, k, v, ld,
                              scores.data_ptr(), done, -1 if eos_token is None else int(eos_token),
                              m, out.data_ptr(), parents.data_ptr(), tokens.data_ptr(),
                              ws.data_ptr(), ws_bytes, _stream_handle(dev))
    _check("flce_beam_select", st)
    return out, parents, tokens


def _reorder_plan(dtype, shape, stride, device, to_dtype, to_shape, into, to_device, b: int, k: int,
                  dev, length: int | None, length_dim: int):
    """Strides and pieces of one state's layout in bytes; None where there is nothing to move."""
    if device != dev or to_device != dev:
        raise ValueError("tensors must be on one CUDA device")
    if len(shape) < 2 or shape[0] != b or shape[1] != k:
        raise ValueError("states must be [batch, beams, ...]")
    if to_shape != shape or to_dtype != dtype:
        raise ValueError("out must have the states' shapes and dtypes")
    e = dtype.itemsize
    inner, outer, outer_stride = e, 1, 0
    for i in range(len(shape) - 1, 1, -1):
        n = shape[i]
        if n > 1 and (stride[i] * e != inner or into[i] * e != inner):
            raise ValueError("states must be contiguous behind [batch, beams]")
        inner *= n
    extent = inner
    for step, n in sorted(((into[0] * e, b), (into[1] * e, k))):
        if n > 1:
            if step < extent:
                raise ValueError("a state's beams must not share memory")
            extent += step * (n - 1)
    if length is not None:
        if not 2 <= length_dim < len(shape) or not 0 <= length <= shape[length_dim]:
            raise ValueError("length must lie within the states' length_dim")
        for n in shape[2:length_dim]:
            outer *= n
        outer_stride = inner // outer if outer else 0
        inner = outer_stride // max(shape[length_dim], 1) * length
    if outer * inner * b * k == 0:
        return None
    return (stride[0] * e, stride[1] * e, into[0] * e, into[1] * e, outer, outer_stride, inner)


def beam_reorder(states, parents, *, length: int | None = None, length_dim: int = 2, out=None,
                 stream=None):
    """``state[b, k] <- state[b, parents[b, k]]`` for one state or a list of them.

    Each state is [B, K, ...], any dtype, contiguous behind the first two dimensions.
    With ``length`` only the first ``length`` positions along ``length_dim`` follow (a
    cache filled so far); the others are left as they were.  Without ``out`` the
    states are reordered in place, with no scratch memory; with ``out`` (the same
    structure) they are gathered into it.  Nothing that is written may share memory with
    another state, with what is read or with ``parents``: refused.  ``parents``
    int64 [B, K]; entries outside [0, K) keep the beam's own state and raise
    FLCE_ERR_BAD_INDEX (``get_error``).  Returns what was written.
    """
    lib = _LIB or load_library()
    single = isinstance(states, torch.Tensor)
    srcs = [states] if single else list(states)
    dsts = srcs if out is None else ([out] if isinstance(out, torch.Tensor) else list(out))
    if len(dsts) != len(srcs):
        raise ValueError("out must have as many tensors as states")
    _cuda_tensor(parents, (torch.int64,), None, "parents")
    if parents.dim() != 2 or not parents.is_contiguous():
        raise ValueError("parents must be a contiguous int64 [batch, beams] tensor")
    b, k = parents.shape
    dev = parents.device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return beam_reorder(states, parents, length=length, length_dim=length_dim, out=out)
    live = []
    last = plan = None  # states of one layout (a model's layers) share its checks
    for src, dst in zip(srcs, dsts):
        layout = src.dtype, src.shape, src.stride(), src.device, dst.dtype, dst.shape, dst.stride(), dst.device
        if layout != last:
            last, plan = layout, _reorder_plan(*layout, b, k, dev, length, length_dim)
        if plan is None:
            continue
        at, to = src.data_ptr(), dst.data_ptr()
        if out is not None and at == to:
            raise ValueError("out must not overlap the states; leave it out to reorder in place")
        live += (at, to, *plan)
    # flce_beam_state is nine 8-byte fields
    st = lib.flce_beam_reorder((_c_i64 * len(live))(*live), len(live) // 9, _ptr(parents), b,
                               max(k, 1), _stream_handle(dev))
    _check("flce_beam_reorder", st)
    return dsts[0] if single else dsts


class CapturedBeamStep:
    """One decoding step behind the model, captured once into a CUDA graph: layer norm
    (when ``norm_weight`` or ``norm_bias`` is given), the head's product in MXFP4,
    beam selection and, with ``states``, their reordering in place.

    The inputs are static tensors owned here -- ``hidden`` [B, K, H], ``scores``
    [B, K] and ``finished`` [B, K] when given -- and a step copies new values into
    them (``set_inputs``) and calls ``replay()``, one graph launch instead of a
    handful of small ones.  The head, the norm's parameters and the states are the
    caller's and must keep their storage.  ``replay()`` returns ``(scores, parents,
    tokens)``, [B, num_select], static too and overwritten by each replay; ``logits``
    holds the step's logits.  Results equal the separate calls bit for bit.  The
    options are host values baked into the graph; with ``states``, num_select must be
    K, and every position of a state is reordered.  Replays of one step, or of
    two that share states, must be ordered on one stream.
    """

    def __init__(self, hidden, head: Mxfp4, scores, *, norm_weight=None, norm_bias=None,
                 norm_eps: float = 1e-5, softcap: float = 0.0, unpadded_vocab: int | None = None,
                 num_select: int | None = None, finished=None, eos_token: int | None = None,
                 states=None, dtype: torch.dtype = torch.bfloat16):
        _cuda_tensor(hidden, W_DTYPES, None, "hidden")
        if hidden.dim() != 3:
            raise ValueError("hidden must be [batch, beams, hidden]")
        if states is not None and num_select not in (None, hidden.shape[1]):
            raise ValueError("states follow as many beams as there are: num_select must be beams")
        dev = hidden.device
        self.hidden = hidden.detach().clone(memory_format=torch.contiguous_format)
        self.scores = scores.detach().clone(memory_format=torch.contiguous_format)
        self.finished = (None if finished is None
                         else finished.clone(memory_format=torch.contiguous_format))
        self.head, self.norm, self.states = head, (norm_weight, norm_bias, norm_eps), states
        self.kw = dict(softcap=softcap, unpadded_vocab=unpadded_vocab, dtype=dtype)
        self.select = dict(num_select=num_select, finished=self.finished, eos_token=eos_token)
        stream = torch.cuda.Stream(dev)
        stream.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(stream):
            # Eager: per-device set-up and argument checks, outside capture.  The states are
            # reordered with every beam keeping its own, which moves nothing.
            self._step(reorder=False)
            if states is not None:
                own = torch.arange(hidden.shape[1], device=dev)
                beam_reorder(states, own.repeat(hidden.shape[0], 1))
        torch.cuda.current_stream(dev).wait_stream(stream)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=stream):
            self.logits, self.out = self._step(reorder=True)

    def _step(self, reorder: bool):
        x, (weight, bias, eps) = self.hidden, self.norm
        if weight is not None or bias is not None:
            x = layer_norm_forward(x, weight, bias, eps=eps, stats=False)[0]
        logits = mxfp4_logits(x, self.head, **self.kw)
        out = beam_select(logits, self.scores, **self.select)
        if reorder and self.states is not None:
            beam_reorder(self.states, out[1])
        return logits, out

    def set_inputs(self, hidden=None, scores=None, finished=None) -> None:
        """Copy a step's values into the captured input buffers (same shapes)."""
        for buf, new in ((self.hidden, hidden), (self.scores, scores), (self.finished, finished)):
            if new is not None:
                if buf is None:
                    raise ValueError("the step was captured without finished beams")
                if new.shape != buf.shape:
                    raise ValueError("inputs must have the captured shapes")
                buf.copy_(new, non_blocking=True)

    def replay(self):
        """Run the step; returns (scores, parents, tokens), static buffers."""
        self.graph.replay()
        return self.out
