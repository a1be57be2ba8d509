"""FP64 definitions of the operators around the LM head (test infrastructure):
layer norm with its gradients.  numpy only; shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd) of rows x [N, H]."""
    x = np.asarray(x, np.float64)
    mean = x.sum(axis=1) / x.shape[1]
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).sum(axis=1) / x.shape[1] + eps)
    y = d * rstd[:, None]
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y, mean, rstd


def layer_norm_grad(dy, x, weight=None, eps=1e-5):
    """(dx, dweight, dbias) of sum(dy * layer_norm(x))."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    h = x.shape[1]
    xhat, _, rstd = layer_norm(x, eps=eps)
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    dx = rstd[:, None] * (g - g.sum(axis=1, keepdims=True) / h
                          - xhat * (g * xhat).sum(axis=1, keepdims=True) / h)
    return dx, (dy * xhat).sum(axis=0), dy.sum(axis=0)
