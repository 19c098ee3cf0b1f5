"""Calls on a cache that are too large for one launch are refused as such, before anything is launched."""
import ctypes

import pytest
import torch

from backward_adapter_gb300 import build as fbuild
from backward_adapter_gb300 import cache as kv
from backward_adapter_gb300 import fa_train as ft


@pytest.mark.parametrize("fmt", [ft.FA_KV_Q8_0, ft.FA_KV_Q4_0])
def test_rows_beyond_31_bits_are_refused(fmt):
    fbuild.build()
    lib, R, F, n = ft.load_library(), ctypes.byref, 1 << 42, 1 << 23
    c = ft.FaCache(256, 1, n, 64, fmt, 0, F, 2 * F, 3 * F, 4 * F)
    k, v = (ft.FaView(i * F, n * 64, 64, n * 64) for i in (5, 6))
    for st in (lib.fa_cache_write(R(c), R(k), R(v), ft.FA_BF16, n, None, 0, None, None),
               lib.fa_cache_read(R(c), 0, n, ft.FA_BF16, R(k), R(v), None)):
        assert st == ft.FA_ERR_UNSUPPORTED and b"too many rows" in lib.fa_last_error()


def test_planes_beyond_31_bits_are_refused():
    """A dimension that a 32-bit number does not hold is not taken for its lower bits."""
    one = torch.zeros(1, dtype=torch.uint8)
    n = (1 << 32) + 5
    planes = (one.expand(1, 1, n, 32), torch.zeros(1, dtype=torch.float16).expand(1, 1, n, 2)) * 2
    for call in (lambda: kv.cache_read(*planes, 0, 3), lambda: kv.decode(torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16), *planes)):
        with pytest.raises(ValueError, match="below 2\\^31"):
            call()


@pytest.mark.gpu
def test_broadcast_rows_beyond_32_bits_are_refused():
    planes = kv.new_cache(1, 1, 8, 64, "q4_0")
    before = [t.clone() for t in planes]
    x = torch.ones((1, 1, 1, 64), device="cuda")
    for n in ((1 << 24) + 1, 1 << 31, (1 << 32) + 3):
        with pytest.raises(ft.FaError, match="n_rows"):
            kv.cache_write(x.expand(1, 1, n, 64), x.expand(1, 1, n, 64), *planes, 0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(planes, before))
