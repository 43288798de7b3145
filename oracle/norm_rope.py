"""RMS norm, rotary embedding and the fused LM-head loss in fp64 (numpy).

TEST INFRASTRUCTURE ONLY (part of the oracle).

Written from the formulas with the analytic gradients; the gradients are
pinned against finite differences and torch's autograd by
``tests/test_oracle_norm_rope.py``.
"""
from __future__ import annotations

import numpy as np


def angles(positions: np.ndarray, inv_freq, axis=None) -> np.ndarray:
    """positions [axes](...) integers -> angles (...)[rot/2], reduced to a turn
    in integer arithmetic: Python's integers hold position * (inv_freq / 2 pi)
    scaled by 2**64 without rounding."""
    inv_freq = np.asarray(inv_freq, dtype=np.float64)
    axis = np.zeros(len(inv_freq), dtype=int) if axis is None else np.asarray(axis)
    out = np.empty(positions.shape[1:] + (len(inv_freq),))
    for f, w in enumerate(inv_freq):
        turns = int(np.floor(np.longdouble(w) / (2 * np.longdouble(np.pi)) * np.longdouble(2.0) ** 64))
        p = positions[axis[f]].reshape(-1)
        frac = [(int(x) * turns) % (1 << 64) for x in p]
        out[..., f] = np.array([(x - (1 << 64) if x >= 1 << 63 else x) / 2.0 ** 64 for x in frac]).reshape(
            positions.shape[1:]) * 2 * np.pi
    return out


def _pairs(rot: int, interleaved: bool):
    f = np.arange(rot // 2)
    return (2 * f, 2 * f + 1) if interleaved else (f, f + rot // 2)


def rotate(x: np.ndarray, t: np.ndarray, interleaved: bool, back: bool = False) -> np.ndarray:
    """x (...)[H][d] turned by t (...)[rot/2] (the same for every head)."""
    y = x.copy()
    a, b = _pairs(2 * t.shape[-1], interleaved)
    c, s = np.cos(t)[..., None, :], np.sin(t)[..., None, :] * (-1 if back else 1)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def norm_rope(x, w, t, interleaved: bool, eps: float):
    """rotate(w * x / rms(x)); w None: rotate(x)."""
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return rotate(x, t, interleaved)


def norm_rope_bwd(x, w, t, dy, interleaved: bool, eps: float):
    """(dx, dw) of norm_rope; dw None without a norm."""
    g = rotate(dy, t, interleaved, back=True)
    if w is None:
        return g, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xhat = x * r
    dw = (g * xhat).reshape(-1, x.shape[-1]).sum(0)
    wg = w * g
    return r * (wg - xhat * (wg * xhat).mean(-1, keepdims=True)), dw


def linear_ce(h, w, shifted, P: int):
    """hidden [B][N][D], weight [V][D], shifted labels [B][N] -> (per-shard mean
    losses, good counts, total, d total/dh, d total/dw, the logits' gradient
    [B*N][V])."""
    B, N, D = h.shape
    rows, y = h.reshape(-1, D), shifted.reshape(-1)
    good = y != -100
    x = np.zeros((B * N, w.shape[0]))
    x[good] = rows[good] @ w.T
    m = x.max(1, keepdims=True)
    e = np.exp(x - m)
    s = e.sum(1, keepdims=True)
    loss = (np.log(s) + m)[:, 0] - x[np.arange(B * N), np.where(good, y, 0)]
    g = e / s
    g[np.arange(B * N), np.where(good, y, 0)] -= 1.0
    T = max(int(good.sum()), 1)
    g *= good[:, None] / T
    per = (loss * good).reshape(B, P, N // P).sum((0, 2))
    counts = good.reshape(B, P, N // P).sum((0, 2))
    total = per.sum() / T
    clean = np.where(good[:, None], rows, 0.0)
    return per / np.maximum(counts, 1), counts, total, (g @ w).reshape(h.shape), g.T @ clean, g
