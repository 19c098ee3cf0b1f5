"""The operators over a cache in pages one after the other, as a serving program uses them: a ragged prompt (norm and rotation, write,
attention of the chunk, the weights its keys got), tokens one by one that add to the weights, eviction into other pages and in
place, and tokens behind it, whose position is no longer their place in the cache; on streams and in captured graphs."""
import numpy as np
import pytest
import torch

import backward_adapter_gb300 as fa
from backward_adapter_gb300 import cache as kv
from backward_adapter_gb300 import fa_train as ft
from tests import paged_util as pu
from tests import test_cache_evict, test_cache_weights, test_decode, test_prefill

ROOM, P = 320, 32


class Session:
    """Sequences over a pool that has the pages of two tables for each, in an order of the seed's."""

    def __init__(self, B, Hq, Hkv, D, fmt, seed):
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
        M = ROOM // P
        self.pool = fa.new_cache(2 * B * M + 1, Hkv, P, D, fmt)
        at = torch.from_numpy(np.random.default_rng(seed).permutation(2 * B * M + 1)[:2 * B * M].astype(np.int32)).cuda()
        self.table, self.other = at.view(2, B, M)
        self.f = fa.rope_inv_freq(D, device="cuda")[0]
        self.w = [(1 + 0.2 * self.r(D).float()).to(torch.bfloat16) for _ in range(2)]
        self.weights = torch.zeros((B, Hkv, ROOM), device="cuda")
        self.lengths = torch.zeros(B, dtype=torch.int64, device="cuda")   # keys in the cache
        self.seen = self.lengths.clone()                                  # tokens so far
        self.qkv = None

    def copy(self):
        twin = object.__new__(Session)
        twin.__dict__ = {k: v.clone() if isinstance(v, torch.Tensor) else [t.clone() for t in v] if isinstance(v, (list, tuple)) else v
                         for k, v in self.__dict__.items()}
        return twin

    def rotated(self, qkv, pos):
        q, k, v = qkv.split([self.Hq, self.Hkv, self.Hkv], dim=2)
        return *fa.qk_norm_rope(q, k, self.f, pos, *self.w, layout="bshd"), v

    def prompt(self, qkv, count):
        q, k, v = self.rotated(qkv, self.seen[:, None] + torch.arange(qkv.shape[1], device="cuda"))
        fa.cache_write(k, v, *self.pool, self.lengths, count, table=self.table, layout="bshd")
        self.lengths += count
        self.seen += count
        o, lse = fa.prefill(q, *self.pool, self.lengths, count, table=self.table, layout="bshd",
                            out=torch.zeros_like(q), lse=torch.zeros((q.shape[0], self.Hq, q.shape[1]), device="cuda"))
        fa.cache_weights(q, lse, self.pool[0], self.pool[1], self.lengths, count, weights=self.weights, out=self.weights, table=self.table,
                         layout="bshd")
        return q, o, lse

    def token(self):
        """One more of every sequence that has any."""
        one = self.lengths.clamp(max=1)
        q, k, v = self.rotated(self.qkv, self.seen[:, None])
        fa.cache_write(k, v, *self.pool, self.lengths, one, table=self.table, layout="bshd")
        self.lengths += one
        self.seen += one
        o, lse = fa.decode(q, *self.pool, self.lengths, table=self.table, layout="bshd")
        fa.cache_weights(q, lse, self.pool[0], self.pool[1], self.lengths, one, weights=self.weights, out=self.weights, table=self.table,
                         layout="bshd")
        return q, o, lse

    def evict(self, keep, **kw):
        kept, left = fa.cache_evict(*self.pool, self.weights, self.lengths, keep, sinks=4, recent=16, table=self.table, **kw)
        self.lengths.copy_(left)
        return kept

    def planes(self, table=None):
        return [pu.gathered(p, self.table if table is None else table).clone() for p in self.pool]


def session(fmt, seed, D=128):
    s = Session(4, 8, 2, D, fmt, seed)
    s.qkv = s.r(4, 1, s.Hq + 2 * s.Hkv, D)
    return s, s.r(4, 260, s.Hq + 2 * s.Hkv, D), pu.i64([260, 0, 61, 133])


def tokens(s, n):
    """n of them, each against the oracle over what the pool holds."""
    for _ in range(n):
        before, lengths = s.weights.clone(), s.lengths.clone()
        q, o, lse = s.token()
        planes, lens = s.planes(), s.lengths.tolist()
        test_decode.check(q.transpose(1, 2).contiguous(), planes, s.lengths, (o.transpose(1, 2), lse))
        test_cache_weights.check(q, lse, planes, lens, [min(x, 1) for x in lens], s.weights, before, layout="bshd")
        assert torch.equal(s.lengths, torch.where(lengths > 0, lengths + 1, lengths))
        s.qkv = s.qkv.roll(1, -1)


@pytest.mark.parametrize("name", ["read", "decode", "prefill", "weights", "evict"])
def test_results_and_scratch_come_from_the_calls_stream(name, monkeypatch):
    """On the host, with a library that does nothing: no call allocates but through the one function that takes the stream."""
    z = lambda *s, dt=torch.int8: torch.zeros(s, dtype=dt)  # noqa: E731
    pool = (z(9, 2, 16, 64), z(9, 2, 16, 2, dt=torch.float16)) * 2
    q, lse, n, table = z(2, 4, 5, 64, dt=torch.bfloat16), z(2, 4, 5, dt=torch.float32), z(2, dt=torch.int64), z(2, 4, dt=torch.int32)
    w, plain, asked = z(2, 2, 64, dt=torch.float32), torch.empty, []

    class Library:
        def __getattr__(self, name):
            return lambda *a: 1000 if name.endswith("workspace_size") else 0

    def empty(shape, strides, dtype, device, stream=None):
        asked.append(stream)
        return plain(shape, dtype=dtype, device=device)

    def refused(*a, **kw):
        raise AssertionError("memory beside the call's stream")
    monkeypatch.setattr(ft, "load_library", Library)
    monkeypatch.setattr(ft, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(ft, "_rows", lambda t, layout: (0, 0, 0, 0))
    monkeypatch.setattr(ft, "_launch", lambda *a: None)
    monkeypatch.setattr(ft, "_empty", empty)
    for f in ("empty", "zeros", "empty_like", "zeros_like"):
        monkeypatch.setattr(torch, f, refused)
    {"read": lambda: kv.cache_read(*pool, n, 3, table=table, stream=77),
     "decode": lambda: kv.decode(q, *pool, n, table=table, stream=77),
     "prefill": lambda: kv.prefill(q, *pool, n, n, table=table, stream=77),
     "weights": lambda: kv.cache_weights(q, lse, *pool[:2], n, n, table=table, stream=77),
     "evict": lambda: kv.cache_evict(*pool, w, n, 9, table=table, stream=77)}[name]()
    assert asked and set(asked) == {77}


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,D", [("q4_0", 128), ("q8_0", 64)])
def test_prompts_tokens_and_eviction(fmt, D):
    s, qkv, count = session(fmt, 3, D)
    counts = count.tolist()
    q, o, lse = s.prompt(qkv, count)
    test_prefill.check(q, s.planes(), counts, counts, (o, lse), layout="bshd")
    test_cache_weights.check(q, lse, s.planes(), counts, counts, s.weights, None, layout="bshd")
    tokens(s, 3)

    def cut(keep, table_out=None):
        lens, w, planes = s.lengths.tolist(), s.weights.cpu(), s.planes()
        kept, left, weights, moved = test_cache_evict.expected(planes, w, lens, keep, 4, 16)
        got = s.evict(keep, table_out=table_out)
        s.table = s.table if table_out is None else table_out
        assert torch.equal(got.cpu(), kept) and torch.equal(s.lengths.cpu(), left) and torch.equal(s.weights.cpu(), weights)
        for a, b in zip(s.planes(), moved):
            assert all(torch.equal(a[i, :, :n].cpu(), b[i, :, :n]) for i, n in enumerate(left.tolist()))

    cut(100, s.other)
    tokens(s, 3)
    cut(64)
    tokens(s, 2)
    # a second chunk behind what was left
    more = pu.i64([40, 0, 7, 1])
    before = s.weights.clone()
    q, o, lse = s.prompt(qkv[:, :40].contiguous(), more)
    lens = s.lengths.tolist()
    test_prefill.check(q, s.planes(), lens, more.tolist(), (o, lse), layout="bshd")
    test_cache_weights.check(q, lse, s.planes(), lens, more.tolist(), s.weights, before, layout="bshd")
    assert ft.device_status() == 0


@pytest.mark.gpu
def test_captured_steps_with_eviction():
    """Tokens and eviction in two graphs over two sessions, replayed in turn, against eager ones, bit for bit."""
    sessions, twins, graphs, outs = [], [], [], []
    for i, fmt in enumerate(("q4_0", "q8_0")):
        s, qkv, count = session(fmt, 10 + i)
        s.prompt(qkv, count)
        twin = s.copy()
        s.copy().token()   # what a first call loads
        warm = s.copy()
        warm.evict(70)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((*s.token(), s.evict(70)))
        for x in (sessions, s), (twins, twin), (graphs, g):
            x[0].append(x[1])
    for turn in range(4):
        for g in graphs:
            g.replay()
        for s, t, out in zip(sessions, twins, outs):
            want = (*t.token(), t.evict(70))
            assert all(torch.equal(a, b) for a, b in zip(out, want)), turn
            assert all(torch.equal(a, b) for a, b in zip(s.pool, t.pool)) and torch.equal(s.weights, t.weights)
            assert torch.equal(s.lengths, t.lengths) and int(s.lengths.max()) == 70
            s.qkv.copy_(s.qkv.roll(1, -1))
            t.qkv.copy_(s.qkv)
    assert ft.device_status() == 0


@pytest.mark.gpu
def test_sessions_side_by_side_on_streams():
    """Two sessions on streams of their own, neither waiting for the other, give what each gives alone."""
    pairs = [session("q4_0", 20 + i) for i in range(2)]
    alone = []
    for s, qkv, count in pairs:
        t = s.copy()
        alone.append((t, [t.prompt(qkv, count), t.token(), t.evict(90), t.token()]))
    torch.cuda.synchronize()
    got, streams = [], [torch.cuda.Stream() for _ in pairs]
    for (s, qkv, count), st in zip(pairs, streams):
        with torch.cuda.stream(st):
            got.append([s.prompt(qkv, count), s.token(), s.evict(90), s.token()])
    torch.cuda.synchronize()
    for (s, *_), a, (t, b) in zip(pairs, got, alone):
        for x, y in zip(a, b):
            x, y = (x, y) if isinstance(x, tuple) else ((x,), (y,))
            assert all(torch.equal(i, j) for i, j in zip(x, y))
        assert all(torch.equal(i, j) for i, j in zip(s.pool, t.pool)) and torch.equal(s.weights, t.weights)
    assert ft.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("n", [3, 40])
def test_planes_of_any_room(fmt, D, n):
    """Planes whose room is no multiple of anything, so that a head's keys begin anywhere: the bits of the same keys in pages."""
    B, Hq, Hkv, S = 3, 9, 3, 333
    padded, pool, table = pu.make(B, Hkv, S, D, fmt, 48, n)
    planes = [p[:, :, :S].contiguous() for p in padded]
    q, lens, count = pu.queries(B, Hq, n, D, 1), pu.i64([S, 17, 150]), pu.i64([n, n, n - 1])
    out = lambda: dict(out=torch.zeros_like(q), lse=torch.zeros((B, Hq, n), device="cuda"))  # noqa: E731
    got, want = fa.prefill(q, *planes, lens, count, **out()), fa.prefill(q, *pool, lens, count, table=table, **out())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    had = torch.rand((B, Hkv, S), generator=torch.Generator().manual_seed(2)).cuda()
    w, want = (fa.cache_weights(q, got[1], p[0], p[1], lens, count, weights=had, **kw)
               for p, kw in ((planes, {}), (pool, dict(table=table))))
    assert torch.equal(w, want)
    none = q[:, :, :0].contiguous()
    assert torch.equal(fa.cache_weights(none, got[1][:, :, :0].contiguous(), *planes[:2], lens, weights=had), had)
    a, b = fa.cache_evict(*planes, w, lens, 101, sinks=3, recent=20), fa.cache_evict(*pool, want, lens, 101, sinks=3, recent=20, table=table)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and torch.equal(w, want)
    for x, y in zip(planes, pool):
        assert torch.equal(x, pu.gathered(y, table)[:, :, :S])
    assert ft.device_status() == 0
