"""The operators around a cached window one after the other, as a program uses them: a serving step (norm and rotation, write,
attention of the new tokens) over a batch of sequences, and a training chunk (norm and rotation, write, forward, backward, the
gradient of norm and rotation) over a window; in streams and in captured graphs."""
import numpy as np
import pytest
import torch

import backward_adapter_gb300 as fa
from backward_adapter_gb300 import fa_train as ft
from oracle import attention as attn
from oracle import kv_cache as kv_ref
from oracle import rope as rope_ref
from oracle import set_rows as rows_ref
from tests import test_decode
from tests.test_rope import U, pair_magnitude


def test_gradient_through_rotation_and_attention_against_differences():
    """The chain of the two oracles' gradients, which the GPU is held to below, against differences of the loss."""
    rng = np.random.default_rng(0)
    B, Hq, Sq, Sk, D = 1, 2, 3, 7, 16
    x, w = rng.standard_normal((B, Hq, Sq, D)), rng.standard_normal(D)
    k, v, do = (rng.standard_normal(s) for s in ((B, 1, Sk, D), (B, 1, Sk, D), (B, Hq, Sq, D)))
    pos, f = [[4, 5, 6]], [1.0, 0.2, 0.05, 0.01]
    at = dict(causal=True, q_offset=4)

    def loss(x_):
        q = rope_ref.forward(x_, pos, f, w, 1e-3)
        return (attn.backward(q, k, v, do, 0.25, **at)["o"] * do).sum()

    dq = attn.backward(rope_ref.forward(x, pos, f, w, 1e-3), k, v, do, 0.25, **at)["dq"]
    dx, _ = rope_ref.backward(dq, x, pos, f, w, 1e-3)
    for ix in ((0, 0, 0, 0), (0, 1, 2, 5), (0, 0, 1, 15)):
        d = np.zeros_like(x)
        d[ix] = 1e-5
        assert abs((loss(x + d) - loss(x - d)) / 2e-5 - dx[ix]) < 1e-7


def step_state(B, Hq, Hkv, S, D, fmt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    f, factor = fa.rope_inv_freq(D, 10000.0, scaling="yarn", scale=4.0, original_length=1024, device="cuda")
    planes = fa.new_cache(B, Hkv, S, D, fmt)
    fa.cache_write(r(B, Hkv, S, D), r(B, Hkv, S, D), *planes, 0)
    return dict(qkv=r(B, 1, Hq + 2 * Hkv, D).to(torch.bfloat16), w=[(1 + 0.2 * r(D)).to(torch.bfloat16) for _ in range(2)],
                f=f, factor=factor, planes=planes, Hq=Hq, Hkv=Hkv)


def step(s, lengths, workspace=None, stream=None):
    """One new token of every sequence: position and place are lengths - 1; a length of 0 is an unused slot."""
    Hq, Hkv = s["Hq"], s["Hkv"]
    q, k, v = s["qkv"].split([Hq, Hkv, Hkv], dim=2)
    at = (lengths - 1)[:, None]
    q, k = fa.qk_norm_rope(q, k, s["f"], at, *s["w"], factor=s["factor"], layout="bshd", stream=stream)
    fa.cache_write(k, v, *s["planes"], lengths - 1, lengths.clamp(max=1), layout="bshd", stream=stream)
    o, lse = fa.decode(q, *s["planes"], lengths, layout="bshd", workspace=workspace, stream=stream)
    return q, k, v, o, lse


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,S", [("q4_0", 90), ("q4_0", 1500), ("q8_0", 700)])
def test_serving_steps(fmt, S):
    B, Hq, Hkv, D = 4, 8, 2, 128
    s = step_state(B, Hq, Hkv, S, D, fmt, S)
    lengths = torch.tensor([S - 2, 1, 0, S // 2], device="cuda")
    for n in range(3):
        before = [t.cpu().numpy().copy() for t in s["planes"]]
        q, k, v, o, lse = step(s, lengths)
        torch.cuda.synchronize()
        assert ft.device_status() == 0
        # the rotated token, against its definition
        pos = (lengths - 1)[:, None].cpu().numpy()
        for x, y, w in ((s["qkv"][:, :, :Hq], q, s["w"][0]), (s["qkv"][:, :, Hq:Hq + Hkv], k, s["w"][1])):
            want = rope_ref.forward(x.transpose(1, 2).double().cpu().numpy(), pos, s["f"].double().cpu().numpy(),
                                    w.double().cpu().numpy(), float(np.float32(1e-6)), factor=float(np.float32(s["factor"])))
            err = np.abs(y.transpose(1, 2).double().cpu().numpy() - want)
            assert np.all(err <= 2.0 ** -8 * np.abs(want) + 32 * U * pair_magnitude(want, D // 2, False))
        # its place in the cache, and every other one
        for i, x in ((0, k), (2, v)):
            nq, nd = kv_ref.quantize(x.transpose(1, 2).float().cpu().numpy(), fmt)
            for b, length in enumerate(lengths.tolist()):
                if length > 0:
                    before[i][b, :, length - 1], before[i + 1][b, :, length - 1] = nq[b, :, 0], nd[b, :, 0]
            np.testing.assert_array_equal(s["planes"][i].cpu().numpy(), before[i])
            np.testing.assert_array_equal(s["planes"][i + 1].cpu().numpy(), before[i + 1])
        test_decode.check(q.transpose(1, 2).contiguous(), s["planes"], lengths, (o.transpose(1, 2), lse))
        assert bool((o[2] == 0).all()) and bool((lse[2] == 0).all())
        lengths = torch.where(lengths > 0, lengths + 1, lengths)
        s["qkv"] = s["qkv"].roll(1, -1)


@pytest.mark.gpu
def test_captured_steps_replay_with_new_lengths():
    """Two graphs over two states, each with a workspace of its own, replayed in turn and against eager steps."""
    S = 1500
    states = [step_state(3, 8, 2, S, 64, "q4_0", 5 + i) for i in range(2)]
    twins = [dict(s, planes=[t.clone() for t in s["planes"]]) for s in states]
    lens = [torch.tensor([700, 1, 0], device="cuda"), torch.tensor([1499, 64, 33], device="cuda")]
    graphs, outs = [], []
    for s, n in zip(states, lens):
        warm = [t.clone() for t in s["planes"]]
        step(s, n)
        for t, w in zip(s["planes"], warm):
            t.copy_(w)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(s, n))
        graphs.append(g)
    for turn in range(3):
        for g in graphs:
            g.replay()
        for s, n, out in zip(twins, lens, outs):
            want = step(s, n)
            assert all(torch.equal(a, b) for a, b in zip(out, want))
        for s, t in zip(states, twins):
            assert all(torch.equal(a, b) for a, b in zip(s["planes"], t["planes"]))
        for n in lens:   # what the graphs read, changed in place
            n.copy_(torch.where((n > 0) & (n < S), n + 1, n))


@pytest.mark.gpu
def test_steps_on_streams_of_their_own():
    """The calls take a stream; work on two of them does not mix, and their scratch is not handed out too early."""
    S = 1400
    states = [step_state(2, 16, 4, S, 128, "q4_0", 11 + i) for i in range(2)]
    lens = torch.tensor([S - 5, 1100], device="cuda")
    want = [step(dict(s, planes=[t.clone() for t in s["planes"]]), lens) for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for n in range(4):
        for i, st in enumerate(streams):
            q, k, v = states[i]["qkv"].split([16, 4, 4], dim=2)
            got.append((i, fa.decode(want[i][0], *states[i]["planes"], lens, layout="bshd", stream=st)))
            got.append((i, fa.decode(want[i][0], *states[i]["planes"], lens, layout="bshd", stream=st.cuda_stream)))
    torch.cuda.synchronize()
    clean = [fa.decode(want[i][0], *states[i]["planes"], lens, layout="bshd") for i in range(2)]
    for i, (o, lse) in got:
        assert torch.equal(o, clean[i][0]) and torch.equal(lse, clean[i][1])
    for i, st in enumerate(streams):
        with torch.cuda.stream(st):
            out = step(states[i], lens)
        st.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


@pytest.mark.gpu
def test_training_chunk_over_the_window():
    """A chunk's queries and keys are rotated, its keys and values written at the end of a 4-bit window, and the loss's
    gradient taken back to the chunk's queries before norm and rotation, and to the window."""
    B, Hq, Hkv, Sq, Sk, D = 1, 4, 2, 96, 400, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, k, v, do = r(B, Hq, Sq, D), r(B, Hkv, Sq, D), r(B, Hkv, Sq, D), r(B, Hq, Sq, D)
    w = [(1 + 0.2 * r(D).float()).to(torch.bfloat16) for _ in range(2)]
    f = fa.rope_inv_freq(D, device="cuda")[0]
    planes = fa.new_cache(B, Hkv, Sk, D, "q4_0")
    fa.cache_write(r(B, Hkv, Sk, D), r(B, Hkv, Sk, D), *planes, 0)
    off = Sk - Sq
    q, kr = fa.qk_norm_rope(x, k, f, None, *w, offset=off)
    fa.cache_write(kr, v, *planes, off)
    o, lse = fa.fwd_q4(q, *planes, causal=True)
    acc = [torch.zeros((B, Hkv, Sk, D), device="cuda") for _ in range(2)]
    dq = fa.bwd_q4(q, *planes, o, lse, do, causal=True, dk_acc=acc[0], dv_acc=acc[1])
    dkr = fa.set_rows_backward(acc[0], torch.arange(off, Sk, device="cuda"))   # the chunk's own rows, read back
    dx, dk, dwq, dwk = fa.qk_norm_rope_bwd(dq, dkr, x, k, f, None, *w, offset=off)
    torch.cuda.synchronize()
    assert ft.device_status() == 0

    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    pos = np.arange(off, Sk)[None]
    vals = [rows_ref.to_bf16_bits(kv_ref.values(planes[i].cpu().numpy(), planes[i + 1].cpu().numpy()).astype(np.float32))
            for i in (0, 2)]
    rq = rope_ref.forward(n(x), pos, n(f), n(w[0]), 1e-6)
    a = attn.backward(rq, *vals, n(do), D ** -0.5, causal=True, q_offset=off)
    want = rope_ref.backward(a["dq"], n(x), pos, n(f), n(w[0]), 1e-6)
    want += rope_ref.backward(a["dk"][:, :, off:], n(k), pos, n(f), n(w[1]), 1e-6)
    # The op's bound on what it returns in bf16 (1e-2 of the largest, and 1e-3), twice: the gradient of the rotation is
    # linear in it, with a factor of 1 / rms(x) * w, and q itself was rounded to bf16 on the way.
    for got, ref in zip((dx, dwq, dk, dwk), want):
        e = np.abs(n(got) - ref).max()
        assert e <= 2e-2 * np.abs(ref).max() + 2e-3, e
    assert np.abs(n(o) - a["o"]).max() <= 1e-2 * np.abs(a["o"]).max() + 1e-3


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_memory_of_a_call_on_a_stream_of_its_own(handle):
    """Memory that the current stream's work still reads is not what a call on another stream is given to write, for
    its results or its scratch; nor is what it wrote given out again while the current stream reads that."""
    B, Hq, Hkv, S, D = 1, 8, 2, 2048, 128
    s = step_state(B, Hq, Hkv, S, D, "q4_0", 31)
    lens = torch.tensor([S], device="cuda")
    q = torch.randn((B, Hq, 64, D), device="cuda").to(torch.bfloat16)
    one = q[:, :, :1].contiguous()
    rot = s["f"]
    calls = {
        "decode": lambda st: fa.decode(one, *s["planes"], lens, stream=st),
        "rope": lambda st: fa.qk_norm_rope(q, q[:, :Hkv], rot, stream=st),
        "read": lambda st: fa.cache_read(*s["planes"], stream=st),
        "fwd": lambda st: fa.fwd_q4(q, *s["planes"], stream=st),
        "bwd": lambda st: fa.bwd_q4(q, *s["planes"], *fwd, q, deterministic=True, stream=st),
    }
    fwd = fa.fwd_q4(q, *s["planes"])
    want = {n: [x.clone() for x in f(None)] for n, f in calls.items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for n, f in calls.items():
        sizes = [x.numel() * x.element_size() for x in want[n]] + [1 << 22, 1 << 24]
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
