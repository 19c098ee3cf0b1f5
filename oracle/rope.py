"""fp64 CPU oracle of the per-head RMS norm with the rotary position, and of its backward.

TEST INFRASTRUCTURE ONLY: shares no code with the GPU path.

For a row x[D] at position p, with weights w (None: no norm):
    n = x * w / sqrt(mean(x^2) + eps)
    the first 2 * len(inv_freq) features of n turned by the angles p * inv_freq[i] in the pairs (i, i + half), or
    (2 i, 2 i + 1) when interleaved, and multiplied by `factor`; the others as they are.
Written with explicit D x D rotation matrices, so that the backward is their transpose.
"""
from __future__ import annotations

import numpy as np


def rotation(D: int, inv_freq, p: int, interleaved: bool, factor: float) -> np.ndarray:
    """The matrix R with y = R n at position p."""
    f = np.asarray(inv_freq, dtype=np.float64)
    half = f.size
    R = np.eye(D)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        t = float(p) * f[i]
        c, s = np.cos(t) * factor, np.sin(t) * factor
        R[a, a], R[a, b], R[b, a], R[b, b] = c, -s, s, c
    return R


def forward(x, positions, inv_freq, weight=None, eps=1e-6, interleaved=False, factor=1.0) -> np.ndarray:
    """x [B, H, S, D], positions [B, S] -> y, float64."""
    x = np.asarray(x, dtype=np.float64)
    B, _, S, D = x.shape
    n = x
    if weight is not None:
        n = x * np.asarray(weight, np.float64) / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    y = np.empty_like(x)
    for b in range(B):
        for s in range(S):
            y[b, :, s] = n[b, :, s] @ rotation(D, inv_freq, int(positions[b][s]), interleaved, factor).T
    return y


def backward(dy, x, positions, inv_freq, weight=None, eps=1e-6, interleaved=False, factor=1.0):
    """(dx, dw): dw is None without weights."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    B, _, S, D = x.shape
    g = np.empty_like(dy)
    for b in range(B):
        for s in range(S):
            g[b, :, s] = dy[b, :, s] @ rotation(D, inv_freq, int(positions[b][s]), interleaved, factor)
    if weight is None:
        return g, None
    w = np.asarray(weight, np.float64)
    ms = (x ** 2).mean(-1, keepdims=True) + eps
    t = g * w
    # n_d = x_d w_d ms^-1/2 and d ms / d x_e = 2 x_e / D
    dx = t * ms ** -0.5 - x * ms ** -1.5 * (t * x).sum(-1, keepdims=True) / D
    return dx, (g * x * ms ** -0.5).sum((0, 1, 2))
