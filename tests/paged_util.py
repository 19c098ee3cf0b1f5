"""Helpers for the tests of a cache in pages: pools, tables, and the contiguous planes that hold the same."""
from __future__ import annotations

import numpy as np
import torch

from oracle import kv_cache as ref
from oracle import paged


def planes_of(k, v, fmt):
    out = []
    for x in (k, v):
        out += [torch.from_numpy(t).cuda() for t in ref.quantize(x, fmt)]
    return out


def make(B, Hkv, S, D, fmt, P, seed, strong=4.0):
    """(contiguous planes [B, Hkv, S, ...], a pool of pages of P keys that holds the same, its table). Pages lie in an order of the
    seed's; the pool has pages that belong to nobody; room is made up to a multiple of P, and planes are as long."""
    rng = np.random.default_rng(seed)
    M = -(-S // P)
    k, v = (rng.standard_normal((B, Hkv, M * P, D)).astype(np.float32) for _ in range(2))
    k[..., ::29] *= strong
    planes = planes_of(k, v, fmt)
    pool, table = to_pages(planes, P, rng)
    return planes, pool, table


def make_any(B, Hkv, S, D, fmt, P, seed):
    """As make, of numbers and scales that were never quantized: for what only moves or compares them."""
    rng = np.random.default_rng(seed)
    S = -(-S // P) * P
    planes = []
    for _ in range(2):
        q = rng.integers(0, 256, (B, Hkv, S, D // 2), np.uint8) if fmt == "q4_0" else rng.integers(-127, 128, (B, Hkv, S, D), np.int8)
        planes += [torch.from_numpy(q).cuda(), torch.from_numpy(rng.uniform(-0.05, 0.05, (B, Hkv, S, D // 32)).astype(np.float16)).cuda()]
    return planes, *to_pages(planes, P, rng)


def to_pages(planes, P, rng, spare=3):
    B, _, S = planes[0].shape[:3]
    M = S // P
    pages = B * M + spare
    at = torch.from_numpy(rng.permutation(pages)[:B * M].reshape(B, M).astype(np.int32)).cuda()
    pool = []
    for p in planes:
        x = torch.full((pages, p.shape[1], P) + tuple(p.shape[3:]), 3, dtype=p.dtype, device="cuda")
        x[at.long()] = p.unflatten(2, (M, P)).transpose(1, 2)
        pool.append(x)
    return pool, at


def unused(table, lengths, P):
    """The table with entries that are no page wherever no key of a sequence is: none of them is looked at."""
    t = table.clone()
    for b, n in enumerate(lengths):
        t[b, -(-int(n) // P):] = [-1, 1 << 30, -(1 << 31)][b % 3]
    return t


def gathered(plane, table):
    return plane[table.long()].transpose(1, 2).flatten(2, 3)


def queries(B, Hq, Sq, D, seed, layout="bhsd"):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((B, Hq, Sq, D), generator=g).to(torch.bfloat16).cuda()
    return q if layout == "bhsd" else q.transpose(1, 2).contiguous()


def i64(x):
    return None if x is None else torch.tensor(x, dtype=torch.int64, device="cuda")


def numpy_planes(planes):
    return [p.cpu().numpy() for p in planes]


def rounded_kv(planes):
    """float64 K and V as the tensor cores get them."""
    n = numpy_planes(planes)
    return paged.held(n, 0, True), paged.held(n, 2, True)
