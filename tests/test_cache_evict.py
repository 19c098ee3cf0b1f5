"""Eviction by accumulated weight (fa_cache_evict) against the oracle's sorting: whole numbers and moved bits, so everything is
equal."""
import ctypes

import numpy as np
import pytest
import torch

from backward_adapter_gb300 import build as fbuild
from backward_adapter_gb300 import cache as kv
from backward_adapter_gb300 import fa_train as ft
from oracle import paged
from tests import paged_util as pu


def some_weights(kind, shape, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(shape, generator=g)
    if kind == "spread":
        return torch.exp(40 * w - 20)
    if kind == "ties":
        return (w * 5).floor()
    if kind == "zeros":
        return torch.zeros(shape)
    if kind == "signs":
        w = w - 0.5
        w[..., ::7] = -0.0
        w[..., 3::7] = 0.0
        return w
    if kind == "no_numbers":
        w[..., ::5] = float("nan")
        w[..., 1::5] = float("inf")
        w[..., 2::5] = -float("inf")
        return w
    return w


def expected(planes, w, lengths, keep, sinks, recent):
    kept, left = paged.evict(w.numpy(), lengths, keep, sinks, recent)
    weights = torch.zeros_like(w)
    out = [p.cpu().clone() for p in planes]
    for b in range(w.shape[0]):
        for h in range(w.shape[1]):
            at = torch.from_numpy(kept[b, h, :left[b]])
            weights[b, h, :left[b]] = w[b, h, at]
            for o, p in zip(out, planes):
                o[b, h, :left[b]] = p[b, h].cpu()[at]
    return torch.from_numpy(kept).int(), torch.from_numpy(np.asarray(left)).long(), weights, out


# B, Hkv, S, D, P, W, lengths, keep, sinks, recent
CASES = {
    "one_key": (1, 1, 1, 64, 16, 1, [1], 1, 0, 0),
    "one_of_two": (2, 1, 2, 128, 16, 2, [2, 1], 1, 0, 0),
    "nothing_to_do": (3, 2, 40, 64, 16, 40, [40, 0, 39], 40, 4, 4),
    "more_than_room": (2, 2, 40, 64, 48, 40, [40, 7], 100, 40, 60),
    "half": (2, 3, 100, 128, 16, 100, [100, 51], 50, 0, 0),
    "sinks_and_recent": (2, 2, 300, 64, 48, 333, [300, 299], 77, 4, 33),
    "only_sinks_and_recent": (1, 2, 300, 128, 16, 300, [300], 40, 9, 31),
    "all_recent": (1, 1, 200, 64, 16, 200, [190], 50, 0, 50),
    "all_sinks": (1, 1, 200, 64, 16, 200, [190], 50, 50, 0),
    "all_but_one": (2, 2, 130, 128, 112, 130, [130, 129], 129, 1, 1),
    "one_left": (1, 2, 500, 64, 16, 500, [500], 1, 0, 0),
    "clusters": (1, 2, 5000, 128, 64, 5000, [5000], 1300, 4, 100),
    "large_clusters": (1, 1, 20000, 64, 128, 20000, [19999], 4001, 16, 1000),
    "more_than_cached": (1, 1, 100000, 64, 256, 100000, [99999], 60000, 4, 77),
    "more_than_a_large_cluster_caches": (1, 1, 180000, 64, 256, 180000, [179999], 90000, 4, 77),
    "many_heads": (40, 4, 100, 64, 16, 100, [1 + (13 * i) % 100 for i in range(40)], 30, 2, 5),
}


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("kind", ["even", "spread", "ties", "zeros", "signs", "no_numbers"])
@pytest.mark.parametrize("name", list(CASES))
def test_evict_against_the_oracle(name, kind, fmt):
    B, Hkv, S, D, P, W, lengths, keep, sinks, recent = CASES[name]
    if S > 10000 and kind in ("even", "signs"):
        pytest.skip("the oracle's sorting is slow")
    planes, pool, table = pu.make_any(B, Hkv, S, D, fmt, P, len(name))
    w = some_weights(kind, (B, Hkv, W), 5)
    kept, left, weights, moved = expected(planes, w, lengths, keep, sinks, recent)
    same = lambda a, b: torch.equal(a.cpu().view(torch.int32), b.view(torch.int32))  # noqa: E731

    def check(got, wo, planes_after, what):
        assert torch.equal(got[0].cpu(), kept) and torch.equal(got[1].cpu(), left), what
        assert same(wo, weights), what
        for a, b in zip(planes_after, moved):
            for s, n in enumerate(left.tolist()):
                assert torch.equal(a[s, :, :n].cpu(), b[s, :, :n]), what
                assert torch.equal(a[s, :, n:].cpu(), b[s, :, n:]), what + ": the rows behind"
    kw = dict(sinks=sinks, recent=recent)
    # into other pages: those moved from stay as they are
    rng = np.random.default_rng(1)
    more = -(-min(keep, 2 * S) // P)
    big = [torch.cat([p, torch.full((B * more + 2,) + tuple(p.shape[1:]), 9, dtype=p.dtype, device="cuda")]) for p in pool]
    before = [p.clone() for p in big]
    at = torch.from_numpy((pool[0].shape[0] + rng.permutation(B * more + 2)[:B * more]).reshape(B, more).astype(np.int32)).cuda()
    if more * P >= keep:
        dev, wo = w.cuda(), torch.full((B, Hkv, W), 3.0, device="cuda")
        got = kv.cache_evict(*big, dev, pu.i64(lengths), keep, table=pu.unused(table, lengths, P), table_out=at, weights_out=wo, **kw)
        assert same(dev, w) and ft.device_status() == 0
        assert torch.equal(got[0].cpu(), kept) and torch.equal(got[1].cpu(), left) and same(wo, weights)
        for a, b, m in zip(big, before, moved):
            n0 = pool[0].shape[0]
            assert torch.equal(a[:n0], b[:n0])
            there, was = pu.gathered(a, at), pu.gathered(b, at)
            for s, n in enumerate(left.tolist()):
                assert torch.equal(there[s, :, :n].cpu(), m[s, :, :n]) and torch.equal(there[s, :, n:], was[s, :, n:])
    # in the same pages, and without any
    dev = w.cuda()
    check(kv.cache_evict(*pool, dev, pu.i64(lengths), keep, table=pu.unused(table, lengths, P), **kw), dev,
          [pu.gathered(p, table) for p in pool], "pages")
    dev = w.cuda()
    check(kv.cache_evict(*planes, dev, pu.i64(lengths), keep, **kw), dev, planes, "planes")
    assert ft.device_status() == 0


@pytest.mark.gpu
def test_evict_reports_what_it_cannot_use():
    planes, pool, table = pu.make_any(3, 1, 64, 64, "q4_0", 16, 2)
    w = some_weights("even", (3, 1, 48), 1)
    dev = w.cuda()
    got = kv.cache_evict(*planes, dev, pu.i64([64, -5, 30]), 20)
    assert ft.device_status() == 0x40000000 | 952
    kept, left, _, _ = expected(planes, w, [48, 0, 30], 20, 0, 0)   # as many keys as there are weights
    assert torch.equal(got[0].cpu(), kept) and torch.equal(got[1].cpu(), left)
    # keys of a page that is none are zeros, and places in one are not written
    bad, other = table.clone(), table[:, [3, 2]].clone()
    bad[0, 0] = -1
    other[1, 1] = 1 << 20
    before = [p.clone() for p in pool]
    kv.cache_evict(*pool, w.cuda(), pu.i64([40, 40, 40]), 20, sinks=20, table=bad, table_out=other)
    assert ft.device_status() == 0x40000000 | 953
    for p, was in zip(pool, before):
        a = pu.gathered(was, table)
        none = 0x88 if p.dtype == torch.uint8 else 0
        assert bool((p[table[0, 3]] == none).all()) and torch.equal(p[table[0, 2]][:, :4], a[0, :, 16:20])
        assert torch.equal(p[table[1, 3]], a[1, :, :16]) and torch.equal(p[table[1, 2]], was[table[1, 2]])


@pytest.mark.gpu
def test_evict_in_a_graph_and_on_a_stream():
    planes, pool, table = pu.make_any(2, 2, 256, 128, "q8_0", 16, 2)
    first = [p.clone() for p in pool]
    w = some_weights("ties", (2, 2, 256), 1).cuda()
    lens, out = pu.i64([250, 100]), pu.i64([0, 0])
    kept = torch.zeros((2, 2, 60), dtype=torch.int32, device="cuda")
    dev = w.clone()
    want = kv.cache_evict(*pool, dev, lens, 60, recent=7, table=table)
    wanted = [p.clone() for p in pool]
    graph = torch.cuda.CUDAGraph()
    dev = w.clone()
    with torch.cuda.graph(graph):
        kv.cache_evict(*pool, dev, lens, 60, recent=7, table=table, kept=kept, lengths_out=out)
    for _ in range(2):
        for p, f in zip(pool, first):
            p.copy_(f)
        dev.copy_(w)
        kept.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept, want[0]) and torch.equal(out, want[1]) and all(torch.equal(a, b) for a, b in zip(pool, wanted))
    side = torch.cuda.Stream()
    for p, f in zip(pool, first):
        p.copy_(f)
    dev.copy_(w)
    side.wait_stream(torch.cuda.current_stream())
    got = kv.cache_evict(*pool, dev, lens, 60, recent=7, table=table, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and all(torch.equal(a, b) for a, b in zip(pool, wanted))


F = 1 << 40


def test_c_abi_refuses_evict():
    fbuild.build()
    lib, R = ft.load_library(), ctypes.byref

    def go(keep=20, sinks=0, recent=0, reserved=0, to=None, pages=True, w=6 * F, W=64, n=7 * F, wo=6 * F, kept=8 * F, out=9 * F, **kw):
        c = ft.FaCache(kw.get("B", 9), 2, kw.get("S", 16), 64, ft.FA_KV_Q4_0, 0, kw.get("k_q", F), 2 * F, 3 * F, 4 * F)
        t = ft.FaPages(5 * F, 4, 2, 4)
        return lib.fa_cache_evict(R(ft.FaEvictParams(keep, sinks, recent, reserved)), R(c), R(t) if pages else None,
                                  R(to) if to is not None else None, w, W, n, wo, kept, out, None)
    assert go(keep=0) == 1 and go(keep=(1 << 24) + 1) == 1 and go(sinks=-1) == 1 and go(recent=-1) == 1 and go(sinks=11, recent=10) == 1
    assert go(reserved=1) == 1 and go(sinks=0x7fffffff, recent=0x7fffffff) == 1 and go(W=0) == 1 and go(W=1 << 31) == 1
    assert go(w=None) == 1 and go(wo=None) == 1 and go(kept=None) == 1 and go(n=None) == 1 and go(out=None) == 1 and go(w=6 * F + 8) == 1
    assert go(n=7 * F + 4) == 1 and go(out=9 * F + 4) == 1 and go(out=7 * F) == 1 and go(wo=6 * F + 16) == 1 and go(kept=6 * F) == 1
    assert go(kept=F) == 1 and go(wo=3 * F) == 1 and go(kept=5 * F) == 1 and go(k_q=None) == 1 and go(S=24) == 1 and go(out=8 * F) == 1
    assert go(to=ft.FaPages(10 * F, 1, 2, 1)) == 1 and go(to=ft.FaPages(10 * F, 4, 3, 4)) == 1 and go(to=ft.FaPages(None, 4, 2, 4)) == 1
    assert go(to=ft.FaPages(10 * F, 4, 9, 4), pages=False) == 1 and go(to=ft.FaPages(8 * F, 4, 2, 4)) == 1
    c = ft.FaCache(9, 2, 16, 64, ft.FA_KV_Q4_0, 0, F, 2 * F, 3 * F, 4 * F)
    assert lib.fa_cache_evict(None, R(c), None, None, 6 * F, 64, 7 * F, 6 * F, 8 * F, 9 * F, None) == 1


def test_binding_refuses_evict(monkeypatch):
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt)  # noqa: E731
    pool = (z(9, 2, 16, 64, dt=torch.int8), z(9, 2, 16, 2, dt=torch.float16)) * 2
    w, n, table = z(2, 2, 64), z(2, dt=torch.int64), z(2, 4, dt=torch.int32)
    ran = []
    monkeypatch.setattr(ft, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(ft, "_launch", lambda device, call, *a: ran.append(a))
    go = lambda **kw: kv.cache_evict(*pool, **{**dict(weights=w, lengths=n, keep=20, table=table, stream=0), **kw})  # noqa: E731
    kept, left = go()
    assert kept.shape == (2, 2, 20) and kept.dtype == torch.int32 and left.shape == (2,) and left.dtype == torch.int64
    for kw, exc in [(dict(weights=w[:, :1]), ValueError), (dict(weights=w.double()), TypeError), (dict(weights_out=z(2, 2, 63)), ValueError),
                    (dict(lengths=n.int()), TypeError), (dict(keep=0), ValueError), (dict(keep=-7), ValueError), (dict(table_out=z(3, 4, dt=torch.int32)), ValueError),
                    (dict(table_out=table.long()), TypeError), (dict(kept=z(2, 2, 21, dt=torch.int32)), ValueError),
                    (dict(kept=z(2, 2, 20)), ValueError), (dict(lengths_out=z(3, dt=torch.int64)), ValueError)]:
        with pytest.raises(exc):
            go(**kw)
    with pytest.raises(ValueError):
        kv.cache_evict(*pool, z(9, 2, 16), z(9, dt=torch.int64), 5, table_out=table, stream=0)
    assert len(ran) == 1
