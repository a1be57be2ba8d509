"""FP64 definitions of the operators around the LM head (test infrastructure):
layer norm with its gradients, MXFP4 quantisation and its product, beam
selection.  numpy only; shares no code with the CUDA path."""
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


E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mxfp4(x):
    """(codes [R, C] 0..15, biased exponents [R, ceil(C / 32)], values [R, C]) of x."""
    x = np.asarray(x, np.float64)
    r, c = x.shape
    codes = np.zeros((r, c), np.int64)
    exps = np.zeros((r, -(-c // 32)), np.int64)
    values = np.zeros((r, c))
    for i in range(r):
        for b in range(exps.shape[1]):
            blk = x[i, 32 * b:32 * b + 32]
            if not np.all(np.isfinite(blk)):
                exps[i, b] = 255
                values[i, 32 * b:32 * b + 32] = np.nan
                continue
            top = np.max(np.abs(blk))
            e = max(-127, int(np.frexp(top)[1]) - 3) if top > 0 else -127
            y = np.abs(np.ldexp(blk, -e))
            dist = np.abs(y[:, None] - E2M1[None, :])
            near = dist == dist.min(axis=1, keepdims=True)
            # two equally near neighbours: the even code
            k = np.array([next((j for j in np.flatnonzero(row) if j % 2 == 0), np.flatnonzero(row)[0])
                          for row in near])
            codes[i, 32 * b:32 * b + 32] = k + 8 * np.signbit(blk)
            exps[i, b] = e + 127
            values[i, 32 * b:32 * b + 32] = np.copysign(np.ldexp(E2M1[k], e), blk)
    return codes, exps, values


def mxfp4_logits(hidden, weight, softcap=0.0):
    """cap(Q(hidden) . Q(weight)^T) and sum |products| per logit."""
    a, w = mxfp4(hidden)[2], mxfp4(weight)[2]
    z = a @ w.T
    return (softcap * np.tanh(z / softcap) if softcap > 0 else z), np.abs(a) @ np.abs(w).T


def beam_select(logits, scores, m, finished=None, eos=None):
    """(scores, parents, tokens) [B, m] of the m best continuations."""
    z, s = np.asarray(logits, np.float64), np.asarray(scores, np.float64)
    b, k, v = z.shape
    out = np.zeros((b, m)), np.zeros((b, m), np.int64), np.zeros((b, m), np.int64)
    for i in range(b):
        total = np.full((k, v), -np.inf)
        for j in range(k):
            if not np.isfinite(s[i, j]):
                continue
            if finished is not None and finished[i, j]:
                total[j, eos] = s[i, j]
                continue
            with np.errstate(invalid="ignore", divide="ignore"):
                top = z[i, j].max()
                lse = top + np.log(np.exp(z[i, j] - top).sum())
                t = s[i, j] + z[i, j] - lse
            total[j] = np.where(np.isnan(t), -np.inf, t)
        order = np.argsort(-total.ravel(), kind="stable")[:m]
        out[0][i], out[1][i], out[2][i] = total.ravel()[order], order // v, order % v
    return out
