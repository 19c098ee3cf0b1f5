"""What the calls without a page table do on the host before the launch: nothing of what only a table needs."""
import pytest
import torch

from backward_adapter_gb300 import build as fbuild
from backward_adapter_gb300 import cache as kv
from backward_adapter_gb300 import fa_train as ft


@pytest.mark.parametrize("name", ["read", "decode", "prefill", "weights", "evict"])
def test_calls_without_a_table_do_not_look_for_one(name, monkeypatch):
    fbuild.build()
    z = lambda *s, dt=torch.int8: torch.zeros(s, dtype=dt)  # noqa: E731
    planes = (z(2, 2, 48, 64), z(2, 2, 48, 2, dt=torch.float16)) * 2
    q, lse, n = z(2, 4, 5, 64, dt=torch.bfloat16), z(2, 4, 5, dt=torch.float32), z(2, dt=torch.int64)
    ran = []

    def table(*a):
        raise AssertionError("there is no table")
    monkeypatch.setattr(kv, "_paged", table)
    monkeypatch.setattr(kv, "_window", table)   # the window is a 32-bit number as it is
    monkeypatch.setattr(ft, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(ft, "_rows", lambda t, layout: (0, 0, 0, 0))
    monkeypatch.setattr(ft, "_launch", lambda device, call, *a: ran.append(a))
    {"read": lambda: kv.cache_read(*planes, 3, stream=0),
     "decode": lambda: kv.decode(q, *planes, n, window=9, stream=0),
     "prefill": lambda: kv.prefill(q, *planes, n, n, window=9, stream=0),
     "weights": lambda: kv.cache_weights(q, lse, *planes[:2], n, n, window=9, stream=0),
     "evict": lambda: kv.cache_evict(*planes, z(2, 2, 48, dt=torch.float32), n, 9, stream=0)}[name]()
    assert len(ran) == 1


@pytest.mark.parametrize("window", [-1, -(1 << 40), 1 << 31, 1 << 40])
def test_windows_that_are_no_32_bit_numbers(window, monkeypatch):
    fbuild.build()
    planes = (torch.zeros(2, 2, 48, 64, dtype=torch.int8), torch.zeros(2, 2, 48, 2, dtype=torch.float16)) * 2
    q, seen = torch.zeros(2, 4, 5, 64, dtype=torch.bfloat16), []
    call = kv._DecodeCall
    monkeypatch.setattr(kv, "_DecodeCall", lambda *a: seen.append(a[12]) or call(*a))
    monkeypatch.setattr(ft, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(ft, "_launch", lambda device, call, *a: None)
    for f in (kv.decode, kv.prefill):
        f(q, *planes, window=window, stream=0)
    kv.cache_weights(q, torch.zeros(2, 4, 5), *planes[:2], window=window, stream=0)
    assert seen == [-1 if window < 0 else 0x7fffffff] * 3
