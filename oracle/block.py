"""fp64 oracle: the operators around the grouped GEMMs -- the norm with the residual's addition,
the router, and a whole expert layer for a few tokens.

TEST INFRASTRUCTURE ONLY (see the package docstring).

* add_rmsnorm: s = x + r, y = s / sqrt(mean(s^2) + eps) * gamma, and its gradients;
* moe_route: choice by key = logit + bias (in fp32, as the library defines it), masked where the
  key is -inf; ties to the lowest expert; weights scale a / Z with a = exp(logit) or
  sigmoid(logit) and Z the sum over all unmasked experts, over the choice, or 1;
* moe_decode: out[t] = sum_j w[t, j] W2_e swiglu(W1_e x_t), with the MX form's activation
  quantized in between.

Loops over tokens and choices, on purpose.
"""
from __future__ import annotations

import numpy as np

from . import mx
from .grouped_gemm import swiglu_fwd


def add_rmsnorm(x, residual, gamma, eps):
    """-> (s, y, rstd) in fp64."""
    s = np.asarray(x, dtype=np.float64) + (0.0 if residual is None else residual)
    rstd = 1.0 / np.sqrt(np.mean(s * s, axis=1) + eps)
    return s, s * rstd[:, None] * gamma, rstd


def add_rmsnorm_bwd(dy, dh, h, gamma, rstd):
    """-> (dx, dgamma) at the saved h and rstd."""
    xh = h * rstd[:, None]
    u = dy * gamma
    dx = rstd[:, None] * (u - xh * np.mean(u * xh, axis=1, keepdims=True))
    return dx + (0.0 if dh is None else dh), np.sum(dy * xh, axis=0)


def _row_scores(x, key, score):
    """a [E] (up to a factor that the normalisation takes out again for softmax), 0 where masked."""
    live = key != -np.inf
    a = np.zeros(len(x))
    if score == "softmax":
        if live.any():
            a[live] = np.exp(x[live] - np.max(x[live]))
    else:
        with np.errstate(over="ignore"):
            a[live] = 1.0 / (1.0 + np.exp(-x[live]))
    return a


def moe_route(logits, bias, k, score, renormalize, scale):
    """logits float32 [T, E] -> (ids [T, k], w [T, k])."""
    x32 = np.asarray(logits, dtype=np.float32)
    T, E = x32.shape
    ids = np.zeros((T, k), dtype=np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        with np.errstate(invalid="ignore"):
            key = x32[t] if bias is None else x32[t] + np.asarray(bias, dtype=np.float32)
        rank = np.where(np.isnan(key), -np.inf, key)
        ids[t] = np.argsort(-rank, kind="stable")[:k]
        if np.isnan(key).any():
            w[t] = np.nan
            continue
        a = _row_scores(x32[t].astype(np.float64), key, score)
        Z = a[ids[t]].sum() if renormalize else a.sum() if score == "softmax" else 1.0
        w[t] = [scale * a[e] / Z if a[e] != 0 else 0.0 for e in ids[t]]
    return ids, w


def moe_route_bwd(logits, bias, ids, dw, score, renormalize, scale):
    """dlogits [T, E] from the Jacobian of w, entry by entry."""
    x32 = np.asarray(logits, dtype=np.float32)
    T, E = x32.shape
    k = ids.shape[1]
    out = np.zeros((T, E))
    for t in range(T):
        key = x32[t] if bias is None else x32[t] + np.asarray(bias, dtype=np.float32)
        if np.isnan(key).any():
            out[t] = np.nan
            continue
        x = x32[t].astype(np.float64)
        a = _row_scores(x, key, score)
        # da_e / dx_e (softmax: the subtracted maximum cancels out of a / Z)
        da = a if score == "softmax" else a * (1.0 - a)
        over = list(ids[t]) if renormalize else list(range(E)) if score == "softmax" else []
        Z = a[over].sum() if over else 1.0
        for j in range(k):
            e = ids[t, j]
            if a[e] == 0:
                continue
            out[t, e] += scale * dw[t, j] * da[e] / Z
            for o in over:
                out[t, o] -= scale * dw[t, j] * a[e] / Z * da[o] / Z
    return out


def moe_decode(x, ids, w, W1, W2, limit=None, fmt=None):
    """x [T, H], W1 [E, 2I, H], W2 [E, H, I] (dequantized for an MX fmt) -> (out [T, H], the largest
    single term of each output's sums, and the sum of the terms' magnitudes)."""
    T, k = ids.shape
    out = np.zeros((T, W2.shape[1]))
    top, mag = np.zeros_like(out), np.zeros_like(out)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if e < 0 or e >= W1.shape[0]:
                continue
            a = swiglu_fwd((W1[e] @ x[t])[None, :], limit)[0]
            if fmt:
                s, c = mx.quantize_blocks(fmt, a.reshape(-1, 32))
                a = (mx.decode(fmt, c) * mx.decode_e8m0(s)[:, None]).reshape(-1)
            wt = 1.0 if w is None else float(w[t, j])
            out[t] += wt * (W2[e] @ a)
            terms = np.abs(wt * W2[e] * a)
            top[t] = np.maximum(top[t], terms.max(axis=1))
            mag[t] += terms.sum(axis=1)
    return out, top, mag
