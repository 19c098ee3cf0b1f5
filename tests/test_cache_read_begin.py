"""cache_read's begin in a tensor of one element is a number, as an int is, where it cannot be one of each sequence's own, int64 [B] on
the device with n_rows."""
import pytest
import torch

from backward_adapter_gb300 import build as fbuild
from backward_adapter_gb300 import cache as kv
from backward_adapter_gb300 import fa_train as ft
from tests import paged_util as pu


def _planes(B, device="cpu"):
    return kv.new_cache(B, 2, 48, 64, "q8_0", device=device)


@pytest.mark.parametrize("B", [1, 3])
@pytest.mark.parametrize("begin", [torch.tensor(7), torch.tensor([7]), torch.tensor(7, dtype=torch.int32), torch.tensor([7], dtype=torch.int32)],
                         ids=["0d", "1d", "0d_int32", "1d_int32"])
def test_a_number_in_a_tensor(B, begin, monkeypatch):
    fbuild.build()
    calls = []
    monkeypatch.setattr(ft, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(ft, "_rows", lambda t, layout: (0, 0, 0, 0))
    monkeypatch.setattr(ft, "_launch", lambda device, call, *a: calls.append((a[2] is None, a[3], a[4])))
    assert kv.cache_read(*_planes(B), begin, stream=0)[0].shape == (B, 2, 41, 64)
    if begin.dim() == 0 or begin.dtype != torch.int64:
        kv.cache_read(*_planes(B), begin, 5, stream=0)
        assert calls == [(True, 7, 41), (True, 7, 5)]
        with pytest.raises(ValueError):
            kv.cache_read(*_planes(B), begin, 42, stream=0)
    elif B == 1:   # the one sequence's own
        kv.cache_read(*_planes(B), begin, 5, stream=0)
        assert calls == [(True, 7, 41), (False, 0, 5)]
    for bad, n in ((torch.zeros(B + 1, dtype=torch.int64), 5), (torch.zeros(2, dtype=torch.int64), None)):
        with pytest.raises(ValueError):
            kv.cache_read(*_planes(B), bad, n, stream=0)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 3])
def test_a_number_on_the_device(B):
    planes, pool, table = pu.make_any(B, 2, 48, 64, "q4_0", 16, 1)
    want = kv.cache_read(*planes, 7)
    for begin in (torch.tensor(7), torch.tensor([7]), torch.tensor(7).cuda(), torch.tensor([7]).cuda()):
        for args, kw in ((planes, {}), (pool, dict(table=table))):
            for n in (None, 41) if B == 1 or begin.dim() == 0 or not begin.is_cuda else (None,):
                got = kv.cache_read(*args, begin, n, **kw)
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert ft.device_status() == 0
