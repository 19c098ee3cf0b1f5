"""Calls on a cache that are too large for one launch are refused as such, before anything is launched."""
import ctypes

import pytest

from backward_adapter_gb300 import build as fbuild
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
