"""Outputs and scratch of the training calls come from the memory of the stream that a call is given: the current stream's work may
still read what the allocator would hand out there, and what the call writes must not be handed out again too early."""
import contextlib

import pytest
import torch

from backward_adapter_gb300 import fa_train as ft


class FakeLibrary:
    """Every call succeeds and wants 1000 bytes of scratch; nothing is launched."""
    def __getattr__(self, name):
        return lambda *a: 1000 if name.endswith("workspace_size") else 0


def calls(q, k, do, o, lse, acc, idx):
    """acc: pairs of accumulators, one for each accumulating call, and a last one to gather from."""
    return {
        "fwd": lambda st: ft.fwd(q, k, k, causal=True, stream=st),
        "bwd": lambda st: ft.bwd(q, k, k, o, lse, do, causal=True, deterministic=True, stream=st),
        "bwd_accum": lambda st: [ft.bwd_accum(q, k, k, o, lse, do, *acc.pop(0), causal=True,
                                              deterministic=True, stream=st)],
        "bwd_accum_rows": lambda st: ft.bwd_accum_rows(q, k, k, o, lse, do, *acc.pop(0), 5, 20,
                                                       causal=True, deterministic=True, stream=st),
        "bwd_noalloc": lambda st: ft.bwd_noalloc(q, k, k, o, lse, do, causal=True, deterministic=True, stream=st),
        "set_rows": lambda st: [ft.set_rows_backward(acc[-1][0], idx, stream=st)],
    }


@pytest.mark.parametrize("name", ["fwd", "bwd", "bwd_accum", "bwd_accum_rows", "bwd_noalloc", "set_rows"])
def test_every_allocation_names_the_calls_stream(name, monkeypatch):
    """On the host, with a library that does nothing: no call allocates but through the one function that takes the stream."""
    asked, inside = [], []
    plain = {n: getattr(torch, n) for n in ("empty", "empty_like", "zeros")}

    def empty(shape, strides, dtype, device, stream=None):
        asked.append(stream)
        inside.append(1)
        try:
            return plain["empty"](shape, dtype=dtype, device=device)
        finally:
            inside.pop()

    def outside(n):
        def f(*a, **kw):
            assert inside, f"torch.{n} beside the call's stream"
            return plain[n](*a, **kw)
        return f
    z = lambda *s, dt=torch.bfloat16: plain["zeros"](s, dtype=dt)  # noqa: E731
    args = (z(1, 4, 40, 64), z(1, 2, 70, 64), z(1, 4, 40, 64), z(1, 4, 40, 64), z(1, 4, 40, dt=torch.float32),
            [[z(1, 2, 70, 64, dt=torch.float32) for _ in range(2)]] * 2, torch.arange(7))
    monkeypatch.setattr(ft, "load_library", lambda: FakeLibrary())
    monkeypatch.setattr(ft, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(ft, "_on_device", lambda t: contextlib.nullcontext())
    monkeypatch.setattr(ft, "_empty", empty)
    for n in plain:
        monkeypatch.setattr(torch, n, outside(n))
    calls(*args)[name](77)
    assert asked and set(asked) == {77}


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_memory_of_training_calls_on_a_stream_of_its_own(handle):
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q, do, k = r(1, 8, 128, 128).bfloat16(), r(1, 8, 128, 128).bfloat16(), r(1, 2, 2048, 128).bfloat16()
    o, lse = ft.fwd(q, k, k, causal=True)
    acc = [r(1, 2, 2048, 128) for _ in range(2)]
    every = calls(q, k, do, o, lse, [[x.clone() for x in acc] for _ in range(5)], torch.arange(100, 900, device="cuda"))
    want = {n: [x.clone() for x in f(None)] for n, f in every.items()}
    side = torch.cuda.Stream()
    for n, f in every.items():
        sizes = [x.numel() * x.element_size() for x in want[n]] + [1 << 20, 1 << 22, 1 << 24]
        held, sums = [torch.full((b,), 7, dtype=torch.uint8, device="cuda") for b in sizes], []
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)   # the current stream is behind: it reads these later
        for h in held:
            sums.append((h != 7).sum())
        del held, h                     # its memory is free for what comes on this stream
        got = f(side.cuda_stream if handle else side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(20_000_000)
        same = [(a != b).sum() for a, b in zip(got, want[n])]
        del got                         # likewise, and the side stream goes on
        with torch.cuda.stream(side):
            again = [torch.full((b,), 1, dtype=torch.uint8, device="cuda") for b in sizes]
        torch.cuda.synchronize()
        assert [int(x) for x in sums] == [0] * len(sums), n
        assert [int(x) for x in same] == [0] * len(same), n
        del again


def test_binding_works_without_torchs_private_calls(monkeypatch):
    """The current stream and device are found through the public functions where a version lacks the others."""
    import importlib.util
    import types
    for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice", "_dynamo"):
        monkeypatch.delattr(torch._C, n, raising=False)
    spec = importlib.util.spec_from_file_location("backward_adapter_gb300._fa_train_again", ft.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: types.SimpleNamespace(cuda_stream=100 + d))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    assert again._stream(torch.device("cuda", 5), None) == 105
    ran = []
    again._launch(torch.device("cuda", 3), lambda *a: ran.append(a) or ft.FA_OK, 1, 2)
    assert ran == [(1, 2)]
    assert again._empty((2, 3), (3, 1), torch.float32, torch.device("cpu")).shape == (2, 3)
