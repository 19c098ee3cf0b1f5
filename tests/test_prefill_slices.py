"""fa_prefill where a slice of the list has several tiles of keys: the running sums over tiles, and references that follow the scores in
a later tile than the slice's first, with O already holding products. The list is worked out here as well, so that a case whose
slices are too short for that fails on any machine. Tolerances are those of tests/test_prefill.py."""
import numpy as np
import pytest
import torch

from backward_adapter_gb300 import cache as kv
from backward_adapter_gb300 import fa_train as ft
from tests import paged_util as pu
from tests.test_prefill import check

KEYS, ROWS = 128, 128   # of a tile; a unit has two tiles of rows
SMS = 152


def slices_of(Hq, Hkv, lengths, counts, window, sms):
    """Each slice's parts: (b, unit, first tile of keys, how many) in the order of the list."""
    G, units = Hq // Hkv, []
    for b, (length, n) in enumerate(zip(lengths, counts)):
        for _ in range(Hkv):
            for u in range(-(-n * G // (2 * ROWS))):
                first, last = u * 2 * ROWS // G, (min((u + 1) * 2 * ROWS, n * G) - 1) // G
                begin = max(length - n + first - window, 0) // KEYS if window else 0
                units.append((b, u, begin, max(-(-max(length - n + last + 1, 0) // KEYS), begin + 1)))
    total = sum(u[3] - u[2] for u in units)
    sizes = [total // sms + (i < total % sms) for i in range(sms)]
    out, at, done = [], 0, 0
    for size in sizes:
        parts = []
        while size > 0:
            b, u, begin, end = units[at]
            take = min(size, end - begin - done)
            parts.append((b, u, begin + done, take))
            size, done = size - take, done + take
            if done == end - begin:
                at, done = at + 1, 0
        out.append(parts)
    return out


def moves(Hq, Hkv, lengths, counts, window, sms, rising=False):
    """(the shortest slice's tiles; of the warps of 32 rows and tiles of keys behind their part's first: how many have a row whose
    reference is set there, how many have such in two or more groups of 32 keys). rising: every group of keys moves it."""
    G, some, several, shortest = Hq // Hkv, 0, 0, 1 << 30
    for parts in slices_of(Hq, Hkv, lengths, counts, window, sms):
        shortest = min(shortest, sum(p[3] for p in parts))
        for b, u, begin, tiles in parts:
            live = min(counts[b] * G - u * 2 * ROWS, 2 * ROWS)
            for r0 in range(0, live, 32):
                pos = lengths[b] - counts[b] + (u * 2 * ROWS + np.arange(r0, min(r0 + 32, live))) // G
                lo = np.maximum(pos - window, 0) if window else np.zeros_like(pos)
                for t in range(begin + 1, begin + tiles):
                    if rising:
                        groups = {c for c in range(4) if (pos >= t * KEYS + 32 * c).any() and (lo < t * KEYS + 32 * c + 32).any()}
                    else:
                        f = lo[(lo >= t * KEYS) & (lo < (t + 1) * KEYS) & (lo <= pos)]
                        groups = set(((f - t * KEYS) // 32).tolist())
                    some, several = some + bool(groups), several + (len(groups) > 1)
    return shortest, some, several


def lengths_from(lo, hi, B):
    return [int(x) for x in np.linspace(lo, hi, B)]


# Hq, Hkv, Sq, lengths, counts (None: all), window
ONE_TILE = {   # of rows a key/value head
    "a_short_window": (8, 8, 100, lengths_from(1050, 3400, 64), None, 200),
    "a_window_two_heads": (16, 8, 64, lengths_from(1500, 3400, 24), None, 1024),
    "a_window_some_tokens": (8, 8, 100, lengths_from(4150, 1111, 24), [100 - 4 * i for i in range(24)], 1000),
    "all_keys": (16, 8, 9, lengths_from(1500, 640, 16), [9 - i % 4 for i in range(15)] + [0], 0),
}
TWO_TILES = {
    "a_short_window_250": (8, 8, 250, lengths_from(1050, 2100, 16), None, 200),
    "a_window_two_heads_100": (16, 8, 100, lengths_from(1500, 3400, 16), [100 - 3 * i for i in range(16)], 1024),
    "all_keys_250": (4, 4, 250, lengths_from(1500, 900, 16), [250 - 7 * i for i in range(16)], 0),
    "units_of_both_kinds": (4, 4, 500, lengths_from(1500, 700, 12), [500, 300, 129, 128, 1, 0, 257, 256, 400, 33, 384, 385], 0),
}
CASES = {**ONE_TILE, **TWO_TILES}


@pytest.mark.parametrize("name", list(CASES))
def test_cases_have_several_tiles_in_a_slice(name):
    Hq, Hkv, n, lengths, counts, window = CASES[name]
    shortest, some, several = moves(Hq, Hkv, lengths, [n] * len(lengths) if counts is None else counts, window, SMS)
    assert shortest >= 3
    if window:
        assert some >= 50 and several >= 20, (some, several)
    assert (n * (Hq // Hkv) <= ROWS) == (name in ONE_TILE)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name", list(CASES))
def test_prefill_over_several_tiles_of_a_slice(name, D, fmt):
    Hq, Hkv, n, lengths, counts, window = CASES[name]
    B, cnts = len(lengths), [n] * len(lengths) if counts is None else counts
    assert moves(Hq, Hkv, lengths, cnts, window, torch.cuda.get_device_properties(0).multi_processor_count)[0] >= 3
    planes, pool, table = pu.make_any(B, Hkv, max(lengths), D, fmt, 48, len(name))
    q = pu.queries(B, Hq, n, D, 3)
    blank = lambda: dict(out=torch.zeros_like(q), lse=torch.zeros((B, Hq, n), device="cuda"), window=window)  # noqa: E731
    got = kv.prefill(q, *pool, pu.i64(lengths), pu.i64(counts), table=pu.unused(table, lengths, 48), **blank())
    assert ft.device_status() == 0
    check(q, planes, lengths, cnts, got, window=window)
    for _ in range(3):   # nothing depends on when a product ends
        flat = kv.prefill(q, *planes, pu.i64(lengths), pu.i64(counts), **blank())
        assert torch.equal(flat[0], got[0]) and torch.equal(flat[1], got[1])
    assert ft.device_status() == 0


RISING = {n: (8, 8, lengths_from(1500, 1100, 8), [n] * 8) for n in (20, 130)}   # one tile of rows, and two


@pytest.mark.parametrize("n", list(RISING))
@pytest.mark.parametrize("window", [0, 700])
def test_rising_scores_move_references_in_later_tiles(n, window):
    Hq, Hkv, lengths, counts = RISING[n]
    shortest, some, several = moves(Hq, Hkv, lengths, counts, window, SMS, rising=True)
    assert shortest >= 2 and several >= 200


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("n", list(RISING))
def test_prefill_scores_that_rise_over_several_tiles(n, window, D, fmt):
    """Heads whose scores rise by 26 (more than 2^30) each 32 keys, by 13, by either in turn, now and then by leaps of several
    hundred, that fall, and that rise and fall."""
    Hq, Hkv, lengths, counts = RISING[n]
    B, S = len(lengths), max(lengths)
    rng = np.random.default_rng(n + D)
    j = np.arange(S) * 0.1
    kinds = [j, j / 2, np.where(np.arange(S) // 64 % 2, j, j / 2), np.maximum.accumulate(np.where(rng.random(S) < 0.01, j, 0)), j[::-1],
             np.minimum(j, j[::-1]), np.where(rng.random(S) < 0.02, j, j / 2), np.where(rng.random(S) < 0.3, j, -j)]
    height = np.stack([np.roll(np.stack(kinds), b, 0) for b in range(B)])[..., None]   # [B, Hkv, S, 1], of K's values
    top = 7 if fmt == "q4_0" else 127
    d = np.broadcast_to(height / top, (B, Hkv, S, D // 32)).astype(np.float16)
    number = np.full((B, Hkv, S, D // 2), 0xff, np.uint8) if fmt == "q4_0" else np.full((B, Hkv, S, D), 127, np.int8)
    _, _, v_q, v_d = pu.make_any(B, Hkv, S, D, fmt, 1, 5)[0]
    planes = [torch.from_numpy(number).cuda(), torch.from_numpy(d.copy()).cuda(), v_q, v_d]
    q = (1 + 0.05 * pu.queries(B, Hq, n, D, 4).float()).to(torch.bfloat16)
    got = kv.prefill(q, *planes, pu.i64(lengths), scale=8 / D, window=window)
    assert ft.device_status() == 0
    check(q, planes, lengths, counts, got, scale=8 / D, window=window)
    again = kv.prefill(q, *planes, pu.i64(lengths), scale=8 / D, window=window)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    assert ft.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["a_short_window", "all_keys", "a_short_window_250"])
def test_several_tiles_of_a_slice_on_two_streams_and_in_a_graph(name):
    Hq, Hkv, n, lengths, counts, window = CASES[name]
    B = len(lengths)
    _, pool, table = pu.make_any(B, Hkv, max(lengths), 128, "q4_0", 48, 5)
    qs, lens, cnts = [pu.queries(B, Hq, n, 128, s) for s in (1, 2)], pu.i64(lengths), pu.i64(counts)
    outs = [(torch.zeros_like(q), torch.zeros((B, Hq, n), device="cuda")) for q in qs]
    go = lambda q, o, **kw: kv.prefill(q, *pool, lens, cnts, table=table, window=window, out=o[0], lse=o[1], **kw)  # noqa: E731
    for q, o in zip(qs, outs):
        go(q, o)
    want = [[t.clone() for t in o] for o in outs]
    same = lambda: all(torch.equal(t, w) for o, x in zip(outs, want) for t, w in zip(o, x))  # noqa: E731
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(5):
        for o in outs:
            o[0].zero_()
        torch.cuda.synchronize()
        for s, q, o in zip(streams, qs, outs):
            go(q, o, stream=s)
        torch.cuda.synchronize()
        assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for q, o in zip(qs, outs):
            go(q, o)
    for _ in range(5):
        for o in outs:
            o[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same()
    assert ft.device_status() == 0
