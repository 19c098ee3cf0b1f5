"""The workspace a caller gives: any dense buffer of the call's device for the training forms, whatever the order of its
dimensions, and nothing with gaps."""
import pytest
import torch

from backward_adapter_gb300 import cache as kv
from backward_adapter_gb300 import fa_train as ft


def test_dense_is_without_gaps_in_any_order():
    t = torch.empty(6, 4, 5)
    for x in (t, t.transpose(0, 2), t.permute(1, 2, 0), t[2:4], t[:, :, :0], torch.empty(3, 1, 4).transpose(0, 1)):
        assert ft._dense(x)
    for x in (t[:, :3], t[::2], t[:, :, 1:].transpose(0, 1), t[:1].expand(6, 4, 5)):
        assert not ft._dense(x)


def chunk(fmt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, do, k, v = r(1, 4, 70, 64), r(1, 4, 70, 64), r(1, 2, 300, 64), r(1, 2, 300, 64)
    planes = kv.new_cache(1, 2, 300, 64, fmt)
    kv.cache_write(k, v, *planes, 0)
    return q, do, k, v, planes


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
def test_cache_forms_take_dense_workspaces(fmt):
    q, do, _, _, planes = chunk(fmt)
    fwd, bwd = (ft.fwd_q8, ft.bwd_q8) if fmt == "q8_0" else (ft.fwd_q4, ft.bwd_q4)
    o, lse = fwd(q, *planes, causal=True)
    grads = bwd(q, *planes, o, lse, do, causal=True, deterministic=True)
    for ws in (torch.empty((1 << 11, 1 << 13), dtype=torch.uint8, device="cuda").t(), torch.empty(1 << 22, device="cuda")):
        got = fwd(q, *planes, causal=True, workspace=ws)
        got += bwd(q, *planes, o, lse, do, causal=True, deterministic=True, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, (o, lse, *grads)))
    for ws in (torch.empty((1 << 12, 1 << 13), dtype=torch.uint8, device="cuda")[:, :4096],
               torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 24), torch.empty(1 << 24, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="workspace"):
            fwd(q, *planes, causal=True, workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            bwd(q, *planes, o, lse, do, causal=True, workspace=ws)
