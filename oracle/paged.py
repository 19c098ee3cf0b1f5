"""CPU oracle of the paged cache: where keys lie, a chunk of new tokens over them, the weight each key got, and eviction.

TEST INFRASTRUCTURE ONLY: shares no code with the GPU path.

Key j of sequence b is row j % P of page table[b][j // P] of the pool's planes [pages, Hkv, P, ...].
"""
from __future__ import annotations

import numpy as np

from . import set_rows
from .kv_cache import values


def gather(plane, table, keys: int):
    """A pool's plane as each sequence's first `keys` keys, [B, Hkv, keys, ...]; entries that are no page give zeros."""
    plane, table = np.asarray(plane), np.asarray(table)
    pages, Hkv, P = plane.shape[:3]
    out = np.zeros((table.shape[0], Hkv, keys) + plane.shape[3:], plane.dtype)
    for b in range(table.shape[0]):
        for j in range(keys):
            page = int(table[b, j // P])
            if 0 <= page < pages:
                out[b, :, j] = plane[page, :, j % P]
    return out


def held(planes, i: int, rounded: bool) -> np.ndarray:
    """float64 K (i = 0) or V (i = 2) of contiguous planes; rounded: to bf16, nearest even, as the training path has them."""
    x = values(planes[i], planes[i + 1])
    return set_rows.to_bf16_bits(x.astype(np.float32)).astype(np.float64) if rounded else x


def seen_keys(length: int, n: int, i: int, window: int):
    """[first, last + 1) of the keys that token i of n sees."""
    pos = length - n + i
    return (max(0, pos - window) if window > 0 else 0), pos + 1


def prefill(q, k, v, lengths, counts, scale: float, window: int = 0):
    """q [B, Hq, Sq, D], k and v float64 [B, Hkv, S, D] -> (o, lse, size) float64: size is what o would be of |v|. Rows from
    counts[b] on are zeros; hidden keys are never touched."""
    q = np.asarray(q, np.float64)
    B, Hq, Sq, D = q.shape
    G = Hq // k.shape[1]
    o, lse, size = np.zeros((B, Hq, Sq, D)), np.zeros((B, Hq, Sq)), np.zeros((B, Hq, Sq, D))
    for b in range(B):
        for i in range(int(counts[b])):
            a, z = seen_keys(int(lengths[b]), int(counts[b]), i, window)
            if z <= a:
                continue
            for h in range(Hq):
                s = scale * (k[b, h // G, a:z] @ q[b, h, i])
                m = s.max()
                p = np.exp(s - m)
                o[b, h, i] = p @ v[b, h // G, a:z] / p.sum()
                size[b, h, i] = p @ np.abs(v[b, h // G, a:z]) / p.sum()
                lse[b, h, i] = m + np.log(p.sum())
    return o, lse, size


def key_weights(q, k, lse, lengths, counts, scale: float, window: int = 0):
    """(sum of exp(scale q k - lse), how many terms) for every key, [B, Hkv, S]."""
    q = np.asarray(q, np.float64)
    B, Hq, Sq, D = q.shape
    Hkv, S = k.shape[1:3]
    G = Hq // Hkv
    out, terms = np.zeros((B, Hkv, S)), np.zeros((B, Hkv, S), np.int64)
    for b in range(B):
        for i in range(int(counts[b])):
            a, z = seen_keys(int(lengths[b]), int(counts[b]), i, window)
            if z <= a:
                continue
            for h in range(Hq):
                out[b, h // G, a:z] += np.exp(scale * (k[b, h // G, a:z] @ q[b, h, i]) - lse[b, h, i])
                terms[b, h // G, a:z] += 1
    return out, terms


def evict(weights, lengths, keep: int, sinks: int, recent: int):
    """(kept int [B, Hkv, keep], new lengths): one head after the other, by sorting."""
    B, Hkv, _ = weights.shape
    kept = np.full((B, Hkv, keep), -1, np.int64)
    left = np.minimum(np.asarray(lengths), keep)
    for b in range(B):
        n = int(lengths[b])
        for h in range(Hkv):
            if n <= keep:
                stay = list(range(n))
            else:
                middle = range(sinks, n - recent)
                by = sorted(middle, key=lambda j: (np.isnan(weights[b, h, j]), -weights[b, h, j], j))
                stay = sorted(list(range(sinks)) + list(range(n - recent, n)) + by[:keep - sinks - recent])
            kept[b, h, :len(stay)] = stay
    return kept, left
