"""Pages that a window hides from every token: any page of the pool may stand in the table for them, whatever it holds."""
import pytest
import torch

from backward_adapter_gb300 import cache as kv
from backward_adapter_gb300 import fa_train as ft
from tests import paged_util as pu


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 48])
@pytest.mark.parametrize("window", [1, 50, 300])
@pytest.mark.parametrize("Sq", [1, 5, 40, 200])
def test_any_page_will_do_before_a_window(Sq, window, P, D, fmt):
    Hq, Hkv, lengths = 4, 2, [1000, 977, 512, 544, 400, 301, 17, 0] + [700 + i for i in range(16)]
    B = len(lengths)
    planes, pool, table = pu.make_any(B, Hkv, max(lengths), D, fmt, P, 3)
    spare = next(p for p in range(pool[0].shape[0]) if p not in set(table.flatten().tolist()))
    for i, bad in ((1, float("nan")), (3, float("inf"))):
        pool[i][spare] = bad
    q, lens = pu.queries(B, Hq, Sq, D, 1), pu.i64(lengths)

    def given_up(counts):
        t = pu.unused(table, lengths, P)
        for b, (length, count) in enumerate(zip(lengths, counts)):
            t[b, :max(length - count - window, 0) // P] = spare
        return t
    if Sq <= 16:
        got, want = (kv.decode(q, *pool, lens, table=t, window=window) for t in (given_up([Sq] * B), table))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    counts = [max(Sq - i % 4, 0) for i in range(B)]
    t = given_up(counts)
    out = lambda: dict(window=window, out=torch.zeros_like(q), lse=torch.zeros((B, Hq, Sq), device="cuda"))  # noqa: E731
    got, want = (kv.prefill(q, *pool, lens, pu.i64(counts), table=x, **out()) for x in (t, table))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    w, want = (kv.cache_weights(q, got[1], *pool[:2], lens, pu.i64(counts), table=x, window=window) for x in (t, table))
    assert torch.equal(w, want)
    assert ft.device_status() == 0
