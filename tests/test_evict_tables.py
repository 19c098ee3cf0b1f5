"""The table that eviction moves to (fa_cache_evict) in the memory of the one it moves from: the same table is in place, columns of their
own are other pages, and entries in common are refused."""
import ctypes

import pytest
import torch

from backward_adapter_gb300 import build as fbuild
from backward_adapter_gb300 import cache as kv
from backward_adapter_gb300 import fa_train as ft
from tests import paged_util as pu

F = 1 << 40


@pytest.mark.parametrize("at,stride,M", [(1, 4, 3), (1, 4, 2), (2, 4, 2), (4, 4, 2), (-1, 4, 2), (-3, 4, 4), (3, 9, 2), (0, 9, 2), (8, 2, 2), (-2, 3, 2), (11, 40, 2),
                                         (-30, 30, 2)])
def test_c_abi_refuses_tables_that_share_entries(at, stride, M):
    fbuild.build()
    lib, R = ft.load_library(), ctypes.byref
    c = ft.FaCache(9, 2, 16, 64, ft.FA_KV_Q4_0, 0, F, 2 * F, 3 * F, 4 * F)
    pages, to = ft.FaPages(5 * F, 4, 3, 4), ft.FaPages(5 * F + 4 * at, stride, 3, M)
    p = ft.FaEvictParams(20, 0, 0, 0)
    assert lib.fa_cache_evict(R(p), R(c), R(pages), R(to), 6 * F, 64, 7 * F, 6 * F, 8 * F, 9 * F, None) == ft.FA_ERR_INVALID_ARG
    assert b"share entries" in lib.fa_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("columns", [32, 9])
def test_the_same_table_again_is_in_place(columns, fmt):
    """Many keys, so that rows that moved too early would be seen."""
    B, Hkv, P, keep = 3, 4, 16, 130
    planes, pool, table = pu.make_any(B, Hkv, 32 * P, 128, fmt, P, 7)
    w = torch.rand((B, Hkv, 32 * P), generator=torch.Generator().manual_seed(1)).cuda()
    lens = pu.i64([512, 301, 90])
    twin, wt = [p.clone() for p in pool], w.clone()
    want = kv.cache_evict(*twin, wt, lens, keep, sinks=2, recent=9, table=table)
    got = kv.cache_evict(*pool, w, lens, keep, sinks=2, recent=9, table=table, table_out=table[:, :columns])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(w, wt)
    assert all(torch.equal(a, b) for a, b in zip(pool, twin))
    assert ft.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 3])
def test_columns_of_one_tensor_are_two_tables(B):
    Hkv, P, keep = 2, 32, 100
    planes, pool, table = pu.make_any(B, Hkv, 8 * P, 64, "q8_0", P, 3)
    w = torch.rand((B, Hkv, 8 * P), generator=torch.Generator().manual_seed(1)).cuda()
    lens = pu.i64([120, 70, 128][:B])   # four pages
    a, b = table[:, :4], table[:, 4:]
    before = [p.clone() for p in pool]
    twin, wt = [p.clone() for p in pool], w.clone()
    want = kv.cache_evict(*twin, wt, lens, keep, recent=9, table=a.clone(), table_out=b.clone())
    got = kv.cache_evict(*pool, w, lens, keep, recent=9, table=a, table_out=b)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(w, wt)
    assert all(torch.equal(x, y) for x, y in zip(pool, twin))
    assert all(torch.equal(pu.gathered(x, a), pu.gathered(y, a)) for x, y in zip(pool, before))
    for bad in (table[:, 3:7], table[:, 1:5]):
        with pytest.raises(ft.FaError, match="share entries"):
            kv.cache_evict(*pool, w, lens, keep, table=a, table_out=bad)
    assert ft.device_status() == 0


@pytest.mark.parametrize("keep", [(1 << 24) + 1, 1 << 31, 1 << 60])
def test_more_keys_to_keep_than_a_cache_holds_are_refused_before_memory_is_asked_for(keep, monkeypatch):
    planes = (torch.zeros(2, 2, 16, 64, dtype=torch.int8), torch.zeros(2, 2, 16, 2, dtype=torch.float16)) * 2

    def memory(*a):
        raise AssertionError("memory")
    monkeypatch.setattr(ft, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(ft, "_empty", memory)
    with pytest.raises(ValueError, match="keep"):
        kv.cache_evict(*planes, torch.zeros(2, 2, 16), torch.zeros(2, dtype=torch.int64), keep, stream=0)
