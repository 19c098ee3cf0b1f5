"""CPU oracle of the quantized K/V cache: its blocks, and attention of the newest tokens over it.

TEST INFRASTRUCTURE ONLY: shares no code with the GPU path.

Blocks of 32 features, arithmetic in float32 as the formats are defined, the scale rounded to float16 first:
  q8_0  d = fp16(max|x| / 127), q = clip(round(x / d), -127, 127), value d * q
  q4_0  d = fp16(m / -8) with m the first value of the largest magnitude, b = clip(round(x / d) + 8, 0, 15), value
        d * (b - 8); byte j of a block's 16: feature j in the low, feature j + 16 in the high four bits.
A scale is held to +-65504, a value that is not a number counts as 0, an infinite one as the largest finite number.
"""
from __future__ import annotations

import numpy as np

FLT_MAX = np.finfo(np.float32).max


def quantize(x, fmt: str):
    """(values, scales) of float32 x [..., D]: loops over blocks, one at a time."""
    x = np.asarray(x, np.float32)
    x = np.clip(np.where(np.isnan(x), np.float32(0), x), -FLT_MAX, FLT_MAX)
    lead, D = x.shape[:-1], x.shape[-1]
    rows = x.reshape(-1, D // 32, 32)
    d = np.zeros(rows.shape[:2], np.float16)
    q = np.zeros(rows.shape, np.int64)
    for i, row in enumerate(rows):
        for k, b in enumerate(row):
            m = b[int(np.argmax(np.abs(b)))]
            with np.errstate(over="ignore"):
                top = abs(m) / np.float32(127) if fmt == "q8_0" else m / np.float32(-8)
                d[i, k] = np.float16(np.clip(top, np.float32(-65504), np.float32(65504)))
            step = np.float32(d[i, k])
            lo, hi = (-127, 127) if fmt == "q8_0" else (-8, 7)
            if step != 0:
                with np.errstate(over="ignore"):
                    q[i, k] = np.clip(np.rint(b / step), lo, hi).astype(np.int64)
    d = d.reshape(*lead, D // 32)
    if fmt == "q8_0":
        return q.astype(np.int8).reshape(*lead, D), d
    b = (q + 8).astype(np.uint8)
    return (b[..., :16] | (b[..., 16:] << 4)).reshape(*lead, D // 2), d


def values(q, d) -> np.ndarray:
    """float64 values of a plane (q int8 or uint8, d float16)."""
    q, d = np.asarray(q), np.asarray(d, np.float64)
    if q.dtype == np.uint8:
        b = q.reshape(*q.shape[:-1], -1, 16).astype(np.int64)
        n = np.concatenate([b & 15, b >> 4], -1) - 8
    else:
        n = q.reshape(*q.shape[:-1], -1, 32).astype(np.int64)
    return (n * d[..., None]).reshape(*d.shape[:-1], -1)


def decode(q, k, v, lengths, scale: float, window: int = 0):
    """q [B, Hq, Sq, D], k and v [B, Hkv, S, D] -> (o, lse), float64; hidden keys and keys past a sequence's length are
    never touched (they may hold anything)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    B, Hq, Sq, D = q.shape
    G = Hq // k.shape[1]
    o, lse = np.zeros((B, Hq, Sq, D)), np.zeros((B, Hq, Sq))
    for b in range(B):
        for i in range(Sq):
            pos = int(lengths[b]) - Sq + i
            first = max(0, pos - window) if window > 0 else 0
            if pos < first:
                continue
            for h in range(Hq):
                kk, vv = k[b, h // G, first:pos + 1], v[b, h // G, first:pos + 1]
                s = scale * (kk @ q[b, h, i])
                m = s.max()
                p = np.exp(s - m)
                o[b, h, i] = p @ vv / p.sum()
                lse[b, h, i] = m + np.log(p.sum())
    return o, lse
