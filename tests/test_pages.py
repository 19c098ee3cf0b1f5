"""A quantized cache in pages: what is written, read and attended to through a table is, bit for bit, what one contiguous window
per sequence gives (whose own tests hold the values to the oracle)."""
import ctypes

import numpy as np
import pytest
import torch

from backward_adapter_gb300 import build as fbuild
from backward_adapter_gb300 import cache as kv
from backward_adapter_gb300 import fa_train as ft
from oracle import paged
from tests import paged_util as pu

FORMATS = ["q8_0", "q4_0"]


def same(pool, table, planes, what=""):
    for i, (p, want) in enumerate(zip(pool, planes)):
        assert torch.equal(pu.gathered(p, table), want), (what, i)


def test_oracle_gather():
    plane = np.arange(5 * 2 * 16 * 3).reshape(5, 2, 16, 3)
    got = paged.gather(plane, np.array([[4, 0], [2, 9]]), 20)
    assert np.array_equal(got[0, 1, 17], plane[0, 1, 1]) and np.array_equal(got[0, 0, 15], plane[4, 0, 15])
    assert np.array_equal(got[1, 1, 3], plane[2, 1, 3]) and not got[1, :, 16:].any()


# B, Hkv, S, D, P, rows, begin (int or one each), count, layout
WRITES = {
    "one_row": (1, 1, 16, 64, 16, 1, 5, None, "bhsd"),
    "a_token_each": (5, 2, 100, 128, 16, 1, [0, 15, 16, 63, 99], None, "bhsd"),
    "over_pages": (2, 3, 96, 64, 48, 70, [3, 26], None, "bshd"),
    "ragged": (3, 2, 300, 128, 112, 130, [0, 111, 170], [130, 0, 77], "bhsd"),
    "many_rows": (2, 4, 1000, 128, 64, 900, 33, None, "bshd"),
}


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", list(WRITES))
def test_write_and_read(name, dtype, fmt):
    B, Hkv, S, D, P, n, begin, count, layout = WRITES[name]
    planes, pool, table = pu.make_any(B, Hkv, S, D, fmt, P, 7)
    before = [p.clone() for p in pool]
    g = torch.Generator().manual_seed(1)
    shape = (B, Hkv, n, D) if layout == "bhsd" else (B, n, Hkv, D)
    k, v = (torch.randn(shape, generator=g).to(dtype).cuda() for _ in range(2))
    at = pu.i64(begin) if isinstance(begin, list) else begin
    kv.cache_write(k, v, *planes, at, pu.i64(count), layout=layout)
    kv.cache_write(k, v, *pool, at, pu.i64(count), table=table, layout=layout)
    assert ft.device_status() == 0
    same(pool, table, planes, name)
    spare = [p for p in range(pool[0].shape[0]) if p not in table.flatten().tolist()]
    for a, b in zip(pool, before):
        assert torch.equal(a[spare], b[spare])   # nobody's pages
    room = planes[0].shape[2]
    for out in (torch.bfloat16, torch.float32):
        for first, rows in ((0, room), (room // 3, room // 2), (room - 1, 1), (5, 0)):
            got = kv.cache_read(*pool, first, rows, table=table, dtype=out, layout=layout)
            want = kv.cache_read(*planes, first, rows, dtype=out, layout=layout)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # each sequence from a place of its own, in pages and in one piece; rows behind the end are zeros, and reported
    firsts = [(7 * b) % room for b in range(B)]
    rows = room - max(firsts)
    for args, kw in ((pool, dict(table=table)), (planes, {})):
        got = kv.cache_read(*args, pu.i64(firsts), rows, layout=layout, **kw)
        assert ft.device_status() == 0
        for b, f in enumerate(firsts):
            want = kv.cache_read(*(p[b:b + 1].contiguous() for p in planes), f, rows, layout=layout)
            assert torch.equal(got[0][b], want[0][0]) and torch.equal(got[1][b], want[1][0])
        got = kv.cache_read(*args, pu.i64([room - 2] * B), 5, **kw)
        assert ft.device_status() == 0x40000000 | 951
        want = kv.cache_read(*planes, room - 2, 2)
        assert torch.equal(got[0][:, :, :2], want[0]) and not bool(got[0][:, :, 2:].any()) and not bool(got[1][:, :, 2:].any())


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_entries_that_are_no_page(fmt):
    planes, pool, table = pu.make_any(2, 2, 64, 64, fmt, 16, 3)
    bad = table.clone()
    bad[0, 1], bad[1, 3] = -1, pool[0].shape[0]
    k = torch.ones((2, 2, 64, 64), dtype=torch.bfloat16, device="cuda")
    before = [p.clone() for p in pool]
    kv.cache_write(k, k, *pool, 0, table=bad)
    assert ft.device_status() == 0x40000000 | 953
    keep = [table[0, 1].item(), table[1, 3].item()]
    for p, b in zip(pool, before):
        assert torch.equal(p[keep], b[keep])
    got = kv.cache_read(*pool, table=bad)
    assert ft.device_status() == 0x40000000 | 953
    want = torch.ones_like(got[0])
    want[0, :, 16:32], want[1, :, 48:] = 0, 0
    assert float((got[0] - want).abs().max()) < 2.0 ** -6 and torch.equal(got[0] == 0, want == 0)
    # attention: as zeros
    zero = [pu.gathered(p, table).contiguous() for p in pool]
    for i in range(4):
        none = 0x88 if zero[i].dtype == torch.uint8 else 0
        zero[i][0, :, 16:32], zero[i][1, :, 48:] = none, none
    q = pu.queries(2, 4, 2, 64, 5)
    want = kv.decode(q, *zero, pu.i64([64, 61]))
    got = kv.decode(q, *pool, pu.i64([64, 61]), table=bad)
    assert ft.device_status() == 0x40000000 | 953
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# B, Hq, Hkv, S, D, Sq, P, lengths (None: all), window
DECODES = {
    "one_key": (1, 1, 1, 1, 64, 1, 16, [1], 0),
    "empty": (3, 4, 2, 70, 128, 1, 16, [0, 17, 0], 0),
    "edges": (8, 4, 1, 200, 128, 1, 16, [15, 16, 17, 31, 32, 33, 48, 199], 0),
    "odd_pages": (3, 6, 2, 400, 64, 1, 48, [399, 95, 97], 0),
    "draft": (2, 8, 2, 300, 128, 5, 112, [3, 300], 0),
    "wide_group": (1, 40, 1, 150, 64, 3, 16, [150], 0),
    "window": (2, 4, 2, 900, 64, 2, 64, [900, 70], 100),
    "all_keys": (2, 8, 8, 256, 128, 1, 256, None, 0),
    "split": (2, 8, 2, 5000, 128, 1, 64, [4999, 1200], 0),
    "long_in_small_pages": (1, 16, 4, 20000, 64, 1, 16, [19990], 0),
    "many": (200, 8, 2, 700, 128, 1, 32, [1 + (37 * i) % 700 for i in range(200)], 0),
    "more_than_listed": (1100, 2, 1, 40, 64, 1, 16, [(7 * i) % 41 for i in range(1100)], 0),
}


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", list(DECODES))
def test_decode(name, fmt):
    B, Hq, Hkv, S, D, Sq, P, lengths, window = DECODES[name]
    planes, pool, table = pu.make_any(B, Hkv, S, D, fmt, P, 11)
    for layout in ("bhsd", "bshd"):
        q = pu.queries(B, Hq, Sq, D, 5, layout)
        want = kv.decode(q, *planes, pu.i64(lengths), window=window, layout=layout)
        t = table if lengths is None else pu.unused(table, lengths, P)
        got = kv.decode(q, *pool, pu.i64(lengths), table=t, window=window, layout=layout)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert ft.device_status() == 0


@pytest.mark.gpu
def test_tables_that_share_pages_and_lie_in_larger_ones():
    planes, pool, table = pu.make_any(3, 2, 128, 128, "q4_0", 16, 2)
    shared = table.clone()
    shared[1, :4] = table[0, :4]   # a common beginning
    large = torch.full((6, 20), -5, dtype=torch.int32, device="cuda")
    large[::2, 7:15] = shared
    view = large[::2, 7:15]
    assert view.stride() == (40, 1)
    flat = [pu.gathered(p, shared).contiguous() for p in pool]
    q = pu.queries(3, 8, 4, 128, 1)
    for got, want in ((kv.decode(q, *pool, table=view), kv.decode(q, *flat)),
                      (kv.prefill(q, *pool, table=view), kv.prefill(q, *flat)),
                      (kv.cache_read(*pool, table=view), kv.cache_read(*flat))):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    one = kv.decode(q[:1], *pool, table=view[:1])   # one sequence: the stride is not looked at
    assert torch.equal(one[0], kv.decode(q[:1], *(f[:1] for f in flat))[0])
    assert ft.device_status() == 0


@pytest.mark.gpu
def test_pools_beyond_32_bits():
    """Pages whose bytes lie behind 2^32, and whose number of rows passes 2^31 elements."""
    Hkv, P, D = 8, 128, 128
    pages = (1 << 32) // (Hkv * P * D) + 9   # 2^32 numbers of q8_0 and some
    pool = list(kv.new_cache(pages, Hkv, P, D, "q8_0"))
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((2, Hkv, 200, D), generator=g, device="cuda", dtype=torch.float32).bfloat16() for _ in range(2))
    table = torch.tensor([[pages - 1, 3], [pages - 5, pages - 2]], dtype=torch.int32, device="cuda")
    kv.cache_write(k, v, *pool, 0, table=table)
    small = kv.new_cache(2, Hkv, 256, D, "q8_0")
    kv.cache_write(k, v, *small, 0)
    lens = pu.i64([200, 131])
    q = pu.queries(2, 16, 4, D, 3)
    for got, want in ((kv.cache_read(*pool, 0, 200, table=table), kv.cache_read(*small, 0, 200)),
                      (kv.decode(q, *pool, lens, table=table), kv.decode(q, *small, lens)),
                      (kv.prefill(q, *pool, lens, table=table), kv.prefill(q, *small, lens))):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    w = torch.rand((2, Hkv, 256), generator=g, device="cuda")
    got, want = ([*kv.cache_evict(*c, w.clone(), lens, 70, recent=9, **kw)] for c, kw in ((pool, dict(table=table)), (small, {})))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got, want = kv.cache_read(*pool, 0, 70, table=table), kv.cache_read(*small, 0, 70)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert ft.device_status() == 0


F = 1 << 40


@pytest.mark.parametrize("field,value", [("B", 0), ("B", 65536), ("M", 0), ("M", (1 << 20) + 1), ("stride", 3), ("table", None),
                                         ("table", F + 2), ("page", 24), ("page", 8)])
def test_c_abi_refuses_tables(field, value):
    fbuild.build()
    lib, R = ft.load_library(), ctypes.byref
    t = dict(table=5 * F, stride=4, B=2, M=4)
    if field != "page":
        t[field] = value
    c = ft.FaCache(9, 2, value if field == "page" else 16, 64, ft.FA_KV_Q8_0, 0, F, 2 * F, 3 * F, 4 * F)
    t = ft.FaPages(**t)
    v = [ft.FaView(i * F, 1 << 20, 64, 1 << 10) for i in (6, 7)]
    assert lib.fa_cache_write_pages(R(c), R(t), R(v[0]), R(v[1]), ft.FA_BF16, 5, None, 0, None, None) == 1
    assert lib.fa_cache_read_pages(R(c), R(t), None, 0, 5, ft.FA_BF16, R(v[0]), R(v[1]), None) == 1
    p = ft.FaDecodeParams(4, 1, 0, 0, 0.1, 0)
    assert lib.fa_decode_pages_workspace_size(R(p), R(c), R(t)) == 0
    assert lib.fa_decode_pages(R(p), 6 * F, R(c), R(t), None, 7 * F, 8 * F, 9 * F, 1 << 33, None) == 1


def test_c_abi_refuses_buffers_of_pages():
    fbuild.build()
    lib, R = ft.load_library(), ctypes.byref
    c = ft.FaCache(1 << 20, 2, 16, 64, ft.FA_KV_Q8_0, 0, F, 2 * F, 3 * F, 4 * F)   # more pages than a cache has sequences
    t = ft.FaPages(5 * F, 4, 2, 4)
    v = lambda at: ft.FaView(at, 1 << 13, 64, 1 << 10)  # noqa: E731
    w = lambda n=5, k=6 * F, x=7 * F, at=None, first=0, count=None: lib.fa_cache_write_pages(  # noqa: E731
        R(c), R(t), R(v(k)), R(v(x)), ft.FA_BF16, n, at, first, count, None)
    assert w(n=0) == ft.FA_OK
    assert w(n=-1) == 1 and w(n=65) == 1 and w(first=60) == 1 and w(first=-1) == 1 and w(k=F) == 1 and w(k=None) == 1
    assert w(at=8 * F + 4) == 1 and w(count=8 * F + 1) == 1 and w(at=F) == 1 and w(count=4 * F) == 1
    r = lambda n=5, k=6 * F, x=7 * F, at=None, first=0: lib.fa_cache_read_pages(  # noqa: E731
        R(c), R(t), at, first, n, ft.FA_BF16, R(v(k)), R(v(x)), None)
    assert r(n=0) == ft.FA_OK
    assert r(n=-1) == 1 and r(first=60) == 1 and r(first=-1) == 1 and r(k=F) == 1 and r(k=5 * F) == 1 and r(at=8 * F + 4) == 1
    assert r(at=6 * F) == 1 and r(x=6 * F) == 1
    p = ft.FaDecodeParams(4, 1, 0, 0, 0.1, 0)
    d = lambda o=7 * F, lse=8 * F, n=None: lib.fa_decode_pages(R(p), 6 * F, R(c), R(t), n, o, lse, 9 * F, 1 << 33, None)  # noqa: E731
    assert d(o=5 * F) == 1 and d(lse=5 * F) == 1 and d(n=7 * F) == 1 and d(n=10 * F + 2) == 1
    c.B = 65536   # without a table these are sequences
    assert lib.fa_cache_write_pages(R(c), None, R(v(6 * F)), R(v(7 * F)), ft.FA_BF16, 5, None, 0, None, None) == 1


def test_binding_refuses_tables(monkeypatch):
    z = lambda *s, dt=torch.int8: torch.zeros(s, dtype=dt)  # noqa: E731
    pool = (z(9, 2, 16, 64), z(9, 2, 16, 2, dt=torch.float16)) * 2
    k, n, table = z(2, 2, 5, 64, dt=torch.bfloat16), z(2, dt=torch.int64), z(2, 4, dt=torch.int32)
    ran = []
    monkeypatch.setattr(ft, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(ft, "_rows", lambda t, layout: (0, 0, 0, 0))
    monkeypatch.setattr(ft, "_launch", lambda device, call, *a: ran.append(a))
    write = lambda **kw: kv.cache_write(**{**dict(k=k, v=k, k_q=pool[0], k_d=pool[1], v_q=pool[2], v_d=pool[3],  # noqa: E731
                                                  begin=n, table=table, stream=0), **kw})
    read = lambda **kw: kv.cache_read(*pool, **{**dict(begin=0, n_rows=5, table=table, stream=0), **kw})  # noqa: E731
    read()
    read(begin=n)
    assert read(n_rows=None)[0].shape == (2, 2, 64, 64)
    count = len(ran)
    for call, kw, exc in [(write, dict(table=table.long()), TypeError), (write, dict(table=table[0]), ValueError),
                          (write, dict(table=z(3, 4, dt=torch.int32)), ValueError), (read, dict(begin=n.int()), TypeError), (read, dict(begin=60), ValueError), (read, dict(begin=n, n_rows=None), ValueError),
                          (read, dict(begin=n, n_rows=-1), ValueError), (read, dict(begin=n[:1]), ValueError),
                          (read, dict(table=z(4, 2, dt=torch.int32).T), ValueError)]:
        with pytest.raises(exc):
            call(**kw)
    assert len(ran) == count
