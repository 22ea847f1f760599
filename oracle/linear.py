"""fp64 oracle: the products with biases (per group, with activation and residual) and the joints
between blocks (norms, gate, dropout, scaled residual), with their gradients.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Activations by their definitions with math.erf and math.exp, one element at a time; the generator of
dropout's mask in Python's integers.
"""
from __future__ import annotations

import math

import numpy as np


def _sigmoid(v):
    return 1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0


def _cdf(v):
    return 0.5 * math.erfc(-v / math.sqrt(2.0))


def act(z, kind, alpha=1.0, offset=0.0, limit=0.0):
    """z [M, N] -> [M, N] or, for swiglu, [M, N / 2]."""
    if kind is None:
        return z
    if kind == "silu":
        return np.vectorize(lambda v: v * _sigmoid(alpha * v), otypes=[float])(z)
    if kind == "gelu":
        return np.vectorize(lambda v: v * _cdf(v), otypes=[float])(z)
    g, u = np.split(z, 2, axis=1)
    if limit > 0:
        g, u = np.minimum(g, limit), np.clip(u, -limit, limit)
    return np.vectorize(lambda a, b: a * _sigmoid(alpha * a) * (b + offset), otypes=[float])(g, u)


def act_bwd(dy, z, kind, alpha=1.0, offset=0.0, limit=0.0):
    """dZ [M, N] from dy, the gradient of act(z)."""
    if kind is None:
        return dy
    if kind == "silu":
        def d(v):
            s = _sigmoid(alpha * v)
            return s + alpha * v * s * _sigmoid(-alpha * v)
        return dy * np.vectorize(d, otypes=[float])(z)
    if kind == "gelu":
        return dy * np.vectorize(lambda v: _cdf(v) + v * math.exp(-v * v / 2) / math.sqrt(2 * math.pi), otypes=[float])(z)
    g, u = np.split(z, 2, axis=1)
    over_g, over_u = np.zeros(g.shape, bool), np.zeros(u.shape, bool)
    if limit > 0:
        over_g, over_u = g > limit, np.abs(u) > limit
        g, u = np.minimum(g, limit), np.clip(u, -limit, limit)
    s = np.vectorize(_sigmoid, otypes=[float])(alpha * g)
    ds = np.vectorize(lambda v: _sigmoid(v) * _sigmoid(-v), otypes=[float])(alpha * g)
    dg = np.where(over_g, 0.0, dy * (u + offset) * (s + alpha * g * ds))
    return np.concatenate([dg, np.where(over_u, 0.0, dy * g * s)], axis=1)


def linear(X, W, lens, bias=None, residual=None, kind=None, **form):
    """-> (Y, Z, the magnitudes |X| |W|^T + |bias| that Z's sums are made of)."""
    M, N = X.shape[0], W.shape[1]
    Z, mag = np.zeros((M, N)), np.zeros((M, N))
    a = 0
    for g, n in enumerate(lens):
        r = slice(a, a + n)
        Z[r], mag[r] = X[r] @ W[g].T, np.abs(X[r]) @ np.abs(W[g]).T
        if bias is not None:
            Z[r], mag[r] = Z[r] + bias[g], mag[r] + np.abs(bias[g])
        a += n
    Y = act(Z, kind, **form)
    return (Y if residual is None else Y + residual), Z, mag


def linear_bwd(dY, Z, lens, kind=None, **form):
    """-> (dZ, dbias [G, N], the sums of |dZ| per group)."""
    dZ = act_bwd(dY, Z, kind, **form)
    db, mag, a = [], [], 0
    for n in lens:
        db.append(dZ[a:a + n].sum(axis=0))
        mag.append(np.abs(dZ[a:a + n]).sum(axis=0))
        a += n
    return dZ, np.array(db), np.array(mag)


def philox4x32(counter, key):
    """Ten rounds of Philox4x32 on four counter words under two key words."""
    x, k = list(counter), list(key)
    for _ in range(10):
        p0, p1 = 0xD2511F53 * x[0], 0xCD9E8D57 * x[2]
        x = [(p1 >> 32) ^ x[1] ^ k[0], p1 & 0xFFFFFFFF, (p0 >> 32) ^ x[3] ^ k[1], p0 & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return x


def keep(R, C, p, rng):
    """Dropout's truth values [R, C] for rng = (seed, offset), 64-bit numbers (signed or not)."""
    if not p:
        return np.ones((R, C), bool)
    seed, off = (int(v) & (2 ** 64 - 1) for v in rng)
    key, hi = (seed & 0xFFFFFFFF, seed >> 32), (off & 0xFFFFFFFF, off >> 32)
    words = [w for i in range((R * C + 3) // 4) for w in philox4x32((i & 0xFFFFFFFF, i >> 32, *hi), key)]
    return (np.array(words[:R * C]) >= math.floor(p * 2 ** 32)).reshape(R, C)


def _branch(x, rstd, gamma_post, gate, mask, p):
    t = x if gamma_post is None else x * rstd[:, None] * gamma_post
    g = 1.0 if gate is None else gate
    return np.where(mask, t / (1 - p), 0.0), g


def join(x, residual, gamma_post, gamma, gate, ra, rb, p, mask, eps):
    """-> (s, y, rstd_post, rstd); gate broadcasts against [R, C] ([R, 1] or [C]) or is None."""
    r1 = 1 / np.sqrt(np.mean(x * x, axis=1) + eps)
    b, g = _branch(x, r1, gamma_post, gate, mask, p)
    s = rb * g * b + (0.0 if residual is None else ra * residual)
    r2 = 1 / np.sqrt(np.mean(s * s, axis=1) + eps)
    return s, None if gamma is None else s * r2[:, None] * gamma, r1, r2


def join_bwd(dy, dh, x, h, r1, r2, gamma_post, gamma, gate, ra, rb, p, mask):
    """-> dict of the gradients, and under "mag" the magnitudes that each one's sums are made of."""
    d = np.zeros_like(x) if dh is None else dh.copy()
    dmag = np.abs(d)
    out, mag = {}, {}
    if gamma is not None:
        hh, u = h * r2[:, None], dy * gamma
        m = np.mean(u * hh, axis=1, keepdims=True)
        d = d + r2[:, None] * (u - hh * m)
        dmag = dmag + r2[:, None] * (np.abs(u) + np.abs(hh) * np.mean(np.abs(u * hh), axis=1, keepdims=True))
        out["dgamma"], mag["dgamma"] = np.sum(dy * hh, axis=0), np.sum(np.abs(dy * hh), axis=0)
    out["dresidual"], mag["dresidual"] = ra * d, np.abs(ra) * dmag
    b, g = _branch(x, r1, gamma_post, gate, mask, p)
    if gate is not None:
        axis = 1 if gate.ndim == 2 else 0
        out["dgate"], mag["dgate"] = rb * np.sum(d * b, axis=axis), abs(rb) * np.sum(dmag * np.abs(b), axis=axis)
    f = rb * g * np.where(mask, 1 / (1 - p), 0.0)
    dt, tmag = f * d, np.abs(f) * dmag
    if gamma_post is not None:
        xh = x * r1[:, None]
        out["dgamma_post"], mag["dgamma_post"] = np.sum(dt * xh, axis=0), np.sum(tmag * np.abs(xh), axis=0)
        w, wmag = dt * gamma_post, tmag * np.abs(gamma_post)
        dt = r1[:, None] * (w - xh * np.mean(w * xh, axis=1, keepdims=True))
        tmag = r1[:, None] * (wmag + np.abs(xh) * np.mean(wmag * np.abs(xh), axis=1, keepdims=True))
    out["dx"], mag["dx"] = dt, tmag
    out["mag"] = mag
    return out
