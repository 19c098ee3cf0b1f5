"""Attention of a ragged chunk over a quantized cache, in pages and in one piece (fa_prefill), against the fp64 oracle.

Tolerances, from the data of each case. K, V and Q are bf16 numbers that the oracle has too; their products are exact in
fp32, and a sum of D of them in eight (four) steps of 16 is off by at most 17 truncations of 2^-24 of what has been added up in
each: E = 2^-17 scale sum_d |q_d k_d|, the largest over the keys a row sees. LSE is off by E and the roundings of its
terms near it, 2^-20 (1 + |LSE| + max |s|). A weight is off by the factor e^(+-E) and rounded to bf16 once, half a step, 2^-8 of its
value; the sum that divides is of unrounded ones. The result is rounded to bf16, 2^-8 of its value:
    |dO| <= (2^-8 + 2 E + 2^-16) sum p |v| / sum p + 2^-8 |O|.
What underflows: an exponential below 2^-126 is 0. It is relative to a reference of which the row's scores are at most 30 above and
the largest at most 1 below (base 2), in a part of the row and where parts are joined, so a key loses less than 2^(-126 + 30) / 2^-1 of the
row's sum, and all of them 2^-95 (number of keys) max |v| of O.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from backward_adapter_gb300 import build as fbuild
from backward_adapter_gb300 import cache as kv
from backward_adapter_gb300 import fa_train as ft
from oracle import paged
from tests import paged_util as pu


def score_error(q, k, lengths, counts, scale, window):
    """E of the module's comment and max |s|, for every (b, head, token)."""
    B, Hq, Sq, _ = q.shape
    G = Hq // k.shape[1]
    e, top = np.zeros((B, Hq, Sq)), np.zeros((B, Hq, Sq))
    for b in range(B):
        for i in range(int(counts[b])):
            a, z = paged.seen_keys(int(lengths[b]), int(counts[b]), i, window)
            for h in range(Hq if z > a else 0):
                kk = k[b, h // G, a:z]
                e[b, h, i] = 2.0 ** -17 * abs(scale) * (np.abs(kk) @ np.abs(q[b, h, i])).max()
                top[b, h, i] = abs(scale) * np.abs(kk @ q[b, h, i]).max()
    return e, top


def check(q, planes, lengths, counts, got, scale=None, window=0, layout="bhsd"):
    o, lse = (t.double().cpu().numpy() for t in got)
    qn = q.double().cpu().numpy()
    if layout == "bshd":
        o, qn = o.swapaxes(1, 2), qn.swapaxes(1, 2)
    scale = 1 / math.sqrt(q.shape[-1]) if scale is None else scale
    k, v = pu.rounded_kv(planes)
    want, want_lse, size = paged.prefill(qn, k, v, lengths, counts, scale, window)
    E, top = score_error(qn, k, lengths, counts, scale, window)
    for b, n in enumerate(counts):
        e = E[b, :, :n]
        err = np.abs(lse[b, :, :n] - want_lse[b, :, :n])
        assert np.all(err <= e + 2.0 ** -20 * (1 + np.abs(want_lse[b, :, :n]) + top[b, :, :n])), (b, err.max(), e.max())
        err, bound = np.abs(o[b, :, :n] - want[b, :, :n]), (2.0 ** -8 + 2 * e[..., None] + 2.0 ** -16) * size[b, :, :n]
        lost = 2.0 ** -95 * k.shape[2] * np.abs(v[b]).max()
        assert np.all(err <= bound + 2.0 ** -8 * np.abs(want[b, :, :n]) + lost), (b, err.max())
        none = size[b, :, :n].sum(-1) == 0
        assert np.all(o[b, :, :n][none] == 0) and np.all(lse[b, :, :n][none] == 0)


def run(B, Hq, Hkv, S, D, Sq, fmt, P, lengths=None, counts=None, window=0, layout="bhsd", scale=None, seed=0):
    """Paged and contiguous: the same bits, and the oracle's values; padding rows are left as they were."""
    planes, pool, table = pu.make(B, Hkv, S, D, fmt, P, seed)
    room = planes[0].shape[2]
    q = pu.queries(B, Hq, Sq, D, seed + 1, layout)
    lens, cnts = [room] * B if lengths is None else lengths, [Sq] * B if counts is None else counts
    out, lse = torch.full_like(q, 5), torch.full((B, Hq, Sq), 5.0, device="cuda")
    kw = dict(scale=scale, window=window, layout=layout)
    got = kv.prefill(q, *pool, pu.i64(lengths), pu.i64(counts), table=pu.unused(table, lens, P), out=out, lse=lse, **kw)
    assert ft.device_status() == 0
    check(q, planes, lens, cnts, got, scale, window, layout)
    rows = torch.arange(Sq, device="cuda") >= torch.tensor(cnts, device="cuda")[:, None]
    o = out if layout == "bhsd" else out.transpose(1, 2)
    assert bool((o.transpose(1, 2)[rows] == 5).all()) and bool((lse.transpose(1, 2)[rows] == 5).all())
    flat = kv.prefill(q, *planes, pu.i64(lengths), pu.i64(counts), out=torch.full_like(q, 5),
                      lse=torch.full((B, Hq, Sq), 5.0, device="cuda"), **kw)
    assert torch.equal(flat[0], got[0]) and torch.equal(flat[1], got[1])
    assert ft.device_status() == 0
    return got


# B, Hq, Hkv, S, D, Sq, P, lengths (None: all), counts (None: all), window
SHAPES = {
    "one_key": (1, 1, 1, 1, 64, 1, 16, [1], None, 0),
    "one_token": (2, 8, 2, 200, 128, 1, 16, [200, 37], None, 0),
    "no_keys": (3, 4, 2, 40, 64, 3, 16, [0, 2, 40], None, 0),
    "more_tokens_than_keys": (2, 4, 1, 130, 128, 140, 48, [5, 130], None, 0),
    "no_tokens": (4, 4, 2, 70, 128, 9, 32, [70, 3, 0, 64], [0, 3, 0, 9], 0),
    "ragged": (5, 6, 2, 300, 64, 77, 16, [300, 5, 129, 128, 127], [77, 5, 33, 64, 1], 0),
    "edges": (6, 4, 1, 300, 128, 33, 112, [127, 128, 129, 255, 256, 257], [31, 32, 33, 1, 32, 33], 0),
    "two_row_tiles": (1, 5, 1, 500, 128, 51, 64, [499], None, 0),
    "group_of_40": (1, 40, 1, 150, 64, 20, 16, [150], None, 0),
    "group_of_300": (1, 300, 1, 90, 64, 3, 16, [77], None, 0),
    "groups_of_one": (2, 3, 3, 260, 128, 130, 128, [260, 131], [130, 7], 0),
    "whole_prompt": (1, 4, 2, 640, 128, 640, 64, [640], None, 0),
    "window": (2, 4, 2, 700, 64, 100, 48, [700, 350], [100, 13], 130),
    "window_of_one": (1, 4, 2, 300, 128, 300, 16, [300], None, 1),
    "long_window": (1, 4, 1, 400, 128, 70, 16, [400], None, 1 << 30),
    "shared": (1, 4, 2, 3000, 128, 8, 64, [2999], None, 0),
    "one_tile_of_rows_over_many_keys": (12, 16, 16, 1500, 64, 9, 48, [1500, 1, 0, 700, 512, 513, 640, 641, 1300, 1499, 129, 900], [9, 1, 3] * 4, 0),
    "the_same_wide": (7, 8, 2, 1300, 128, 32, 16, [1300, 31, 520, 1024, 1025, 700, 1299], [32, 32, 1, 31, 20, 8, 32], 0),
    "one_tile_of_rows_in_a_window": (4, 8, 8, 2500, 64, 20, 16, [2500, 1100, 640, 2000], [20, 3, 20, 1], 900),
    "shared_by_many": (1, 1, 1, 9000, 64, 2, 256, [8999], None, 0),
    "many_sequences": (70, 2, 1, 48, 64, 4, 16, list(range(1, 48)) + [48] * 23, [1 + i % 4 for i in range(70)], 0),
}


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("name", list(SHAPES))
def test_prefill_against_the_oracle(name, fmt):
    B, Hq, Hkv, S, D, Sq, P, lengths, counts, window = SHAPES[name]
    run(B, Hq, Hkv, S, D, Sq, fmt, P, lengths, counts, window, seed=len(name))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("kw", [dict(layout="bshd"), dict(scale=-0.3), dict(scale=0.0), dict(scale=1.7),
                                dict(layout="bshd", window=19, scale=-0.05)], ids=lambda kw: "_".join(f"{k}{v}" for k, v in kw.items()))
def test_prefill_layouts_and_scales(kw, fmt, D):
    run(2, 6, 2, 190, D, 70, fmt, 16, [190, 81], [70, 44], seed=D, **kw)


@pytest.mark.gpu
def test_prefill_without_lengths_and_counts():
    run(2, 4, 2, 96, 128, 33, "q4_0", 48)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_of_tensors_at_any_multiple_of_16_bytes(D):
    planes, pool, table = pu.make(2, 2, 90, D, "q4_0", 16, 4)
    q = pu.queries(2, 4, 37, D, 5)
    want = kv.prefill(q, *pool, table=table)
    for first in (8, 16, 24):   # bf16 elements
        hold = [torch.zeros(q.numel() + 64, dtype=q.dtype, device="cuda")[first:first + q.numel()].view(q.shape) for _ in range(2)]
        lse = torch.zeros(want[1].numel() + 16, device="cuda")[4:4 + want[1].numel()].view(want[1].shape)
        hold[0].copy_(q)
        kv.prefill(hold[0], *pool, table=table, out=hold[1], lse=lse)
        assert torch.equal(hold[1], want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
def test_prefill_is_the_training_forward_over_the_same_cache():
    """One chunk of one length: fwd_q4's values, both within their roundings of each other, the weights' and the output's."""
    planes, pool, table = pu.make(2, 2, 512, 128, "q4_0", 64, 5)
    q = pu.queries(2, 8, 96, 128, 6)
    o, lse = kv.prefill(q, *pool, table=table)
    fo, flse = ft.fwd_q4(q, *planes, causal=True, q_offset=512 - 96)
    assert float((lse - flse).abs().max()) <= 2.0 ** -16
    k, v = pu.rounded_kv(planes)
    _, _, size = paged.prefill(q.double().cpu().numpy(), k, v, [512] * 2, [96] * 2, 128 ** -0.5)
    assert np.all((o - fo).double().abs().cpu().numpy() <= 2.0 ** -6 * size)   # two roundings of 2^-8 on each side


@pytest.mark.gpu
def test_prefill_of_more_sequences_than_a_launch_lists():
    B = 1100
    planes, pool, table = pu.make(B, 1, 20, 64, "q8_0", 16, 3)
    q = pu.queries(B, 2, 2, 64, 4)
    lens = [1 + i % 20 for i in range(B)]
    cnts = [i % 3 for i in range(B)]
    got = kv.prefill(q, *pool, pu.i64(lens), pu.i64(cnts), table=table)
    check(q, planes, lens, cnts, got)
    flat = kv.prefill(q, *planes, pu.i64(lens), pu.i64(cnts))
    for b in range(B):
        assert torch.equal(flat[0][b, :, :cnts[b]], got[0][b, :, :cnts[b]])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
def test_prefill_keys_that_nobody_sees_may_hold_anything(fmt):
    """Keys behind the length, and those that a window hides, with scales that are no numbers: the others' bits stay."""
    planes, pool, table = pu.make(2, 2, 400, 128, fmt, 16, 8)
    q = pu.queries(2, 4, 40, 128, 9)
    lens = pu.i64([333, 200])
    a = kv.prefill(q, *planes, lens, window=60)
    for bad in (float("inf"), float("nan"), -float("inf")):
        dirty = [p.clone() for p in planes]
        for i in (1, 3):
            dirty[i][0, :, 333:] = bad
            dirty[i][0, :, :333 - 40 - 60] = bad
            dirty[i][1, :, 200:] = bad
            dirty[i][1, :, :200 - 40 - 60] = bad
            dirty[i - 1][0, :, 333:] = 77
        b = kv.prefill(q, *dirty, lens, window=60)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # a key that only the later tokens see: the earlier ones' rows stay
    dirty = [p.clone() for p in planes]
    for i in (1, 3):
        dirty[i][0, :, 333 - 10] = float("nan")
    b = kv.prefill(q, *dirty, lens, window=60)
    assert torch.equal(a[0][0, :, :30], b[0][0, :, :30]) and torch.equal(a[0][1], b[0][1])
    assert bool(b[0][0, :, 30:].isnan().all()) and bool(b[1][0, :, 30:].isnan().all())


@pytest.mark.gpu
def test_prefill_of_padding_that_is_no_number():
    planes, pool, table = pu.make(2, 2, 200, 64, "q8_0", 16, 1)
    q = pu.queries(2, 4, 50, 64, 2)
    counts = [20, 33]
    clean = kv.prefill(q, *pool, pu.i64([200, 150]), pu.i64(counts), table=table)
    for b, n in enumerate(counts):
        q[b, :, n:] = float("nan")
    dirty = kv.prefill(q, *pool, pu.i64([200, 150]), pu.i64(counts), table=table)
    for b, n in enumerate(counts):
        assert torch.equal(clean[0][b, :, :n], dirty[0][b, :, :n]) and torch.equal(clean[1][b, :, :n], dirty[1][b, :, :n])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("n,D", [(20, 64), (20, 128), (130, 64), (130, 128)], ids=lambda x: str(x))
def test_prefill_scores_that_rise_from_tile_to_tile(n, D, fmt):
    """By more than 2^30 each 32 keys, for some rows all the way and for others now and then, so that what there is follows again
    and again; rows of one tile and of several."""
    B, Hq, Hkv, S = 2, 4, 2, 1500
    rng = np.random.default_rng(D + n)
    k = np.broadcast_to(np.arange(S)[None, None, :, None] * 0.1, (B, Hkv, S, D)).astype(np.float32).copy()
    k[:, 1] *= np.where(rng.random((B, S, 1)) < 0.02, 1.0, 0.5)
    k[1] = k[1, :, ::-1]   # falling: the first scores stay the reference
    planes = pu.planes_of(k, rng.standard_normal(k.shape).astype(np.float32), fmt)
    q = (1 + 0.05 * pu.queries(B, Hq, n, D, 4).float()).to(torch.bfloat16)
    lens = [S, S - 77]
    got = kv.prefill(q, *planes, pu.i64(lens), scale=8 / D)
    assert ft.device_status() == 0
    check(q, planes, lens, [n, n], got, scale=8 / D)


@pytest.mark.gpu
def test_prefill_values_of_every_size():
    """Scales from fp16's smallest to its largest, of both signs, beside each other."""
    for fmt in ("q8_0", "q4_0"):
        planes, pool, table = pu.make(1, 1, 300, 128, fmt, 64, 11)
        g = torch.Generator().manual_seed(3)
        for i, top in ((1, 8), (3, 15.9)):
            e = torch.rand(planes[i].shape, generator=g) * (top + 24) - 24
            s = torch.where(torch.rand(planes[i].shape, generator=g) < 0.5, -1.0, 1.0)
            planes[i] = (s * torch.exp2(e)).to(torch.float16).cuda()
        q = pu.queries(1, 4, 20, 128, 12) * 0.01
        got = kv.prefill(q, *planes, scale=0.01)
        check(q, planes, [planes[0].shape[2]], [20], got, scale=0.01)


@pytest.mark.gpu
def test_prefill_reports_what_it_cannot_use():
    planes, pool, table = pu.make(2, 1, 64, 64, "q8_0", 16, 1)
    q = pu.queries(2, 2, 8, 64, 2)
    want = kv.prefill(q, *pool, pu.i64([64, 0]), pu.i64([8, 0]), table=table)
    got = kv.prefill(q, *pool, pu.i64([65, -3]), pu.i64([9, -1]), table=table)
    assert ft.device_status() == 0x40000000 | 952
    assert torch.equal(got[0][0], want[0][0]) and torch.equal(got[1][0], want[1][0])
    # a page that is none: its keys count as zeros
    bad = table.clone()
    bad[0, 1] = pool[0].shape[0]
    zero = [p.clone() for p in planes]
    for i in (1, 3):
        zero[i][0, :, 16:32] = 0
    got = kv.prefill(q, *pool, table=bad)
    assert ft.device_status() == 0x40000000 | 953
    want = kv.prefill(q, *zero)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert ft.device_status() == 0


@pytest.mark.gpu
def test_prefill_twice_on_two_streams_and_in_a_graph():
    planes, pool, table = pu.make(3, 2, 2000, 128, "q4_0", 64, 21)
    q = [pu.queries(3, 8, 40, 128, s) for s in (1, 2)]
    lens, cnts = pu.i64([2000, 900, 64]), pu.i64([40, 8, 40])
    out = [(torch.zeros_like(x), torch.zeros(x.shape[:3], device="cuda")) for x in q]
    go = lambda x, o, **kw: kv.prefill(x, *pool, lens, cnts, table=table, out=o[0], lse=o[1], **kw)  # noqa: E731
    for x, o in zip(q, out):
        go(x, o)
    want = [[t.clone() for t in o] for o in out]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in q]
    for _ in range(5):
        for o in out:
            o[0].zero_()
        torch.cuda.synchronize()
        for s, x, o in zip(streams, q, out):
            go(x, o, stream=s)
        torch.cuda.synchronize()
        for o, w in zip(out, want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(q[0], out[0])
    for x in (q[1], q[0]):
        other = x.clone()
        q[0].copy_(other)
        out[0][0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        again = (torch.zeros_like(x), torch.zeros(x.shape[:3], device="cuda"))
        go(other, again)
        assert torch.equal(out[0][0], again[0]) and torch.equal(out[0][1], again[1])
    assert ft.device_status() == 0


F = 1 << 40   # addresses that nothing is read from: every call below is refused before


def _structs(**kw):
    c = dict(B=9, Hkv=2, S=16, D=64, kv_format=ft.FA_KV_Q8_0, reserved=0, k_q=F, k_d=2 * F, v_q=3 * F, v_d=4 * F)
    t = dict(table=5 * F, stride=4, B=2, M=4)
    p = dict(Hq=4, Sq=8, window=0, layout=0, scale=0.1, reserved=0)
    for n, v in kw.items():
        kind, name = n.split("__")
        dict(c=c, t=t, p=p)[kind][name] = v
    return ft.FaPrefillParams(**p), ft.FaCache(**c), ft.FaPages(**t)


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return ft.load_library()


REFUSED = [("p__Hq", 0, 1), ("p__Hq", 5, 1), ("p__Hq", 65538, 1), ("p__Sq", -1, 1), ("p__Sq", (1 << 24) + 1, 1), ("p__window", -1, 1),
           ("p__layout", 2, 1), ("p__scale", float("inf"), 1), ("p__scale", float("nan"), 1), ("p__reserved", 1, 1),
           ("c__B", 0, 1), ("c__S", 24, 1), ("c__S", 0, 1), ("c__D", 96, 2), ("c__kv_format", 2, 1), ("c__reserved", 1, 1),
           ("t__B", 0, 1), ("t__B", 65536, 1), ("t__M", 0, 1), ("t__M", (1 << 20) + 1, 1), ("t__stride", 3, 1), ("t__table", None, 1),
           ("t__table", 5 * F + 2, 1), ("c__k_q", F + 8, 1), ("c__v_d", None, 1)]


@pytest.mark.parametrize("what,value,code", REFUSED)
def test_c_abi_refuses_prefill(lib, what, value, code):
    R = ctypes.byref
    p, c, t = _structs(**{what: value})
    assert lib.fa_prefill_workspace_size(R(p), R(c), R(t)) == 0 or what in ("c__k_q", "c__v_d")
    assert lib.fa_prefill(R(p), 6 * F, R(c), R(t), None, None, 7 * F, 8 * F, 9 * F, 1 << 33, None) == code
    assert lib.fa_last_error()
    if what != "c__v_d":   # V is not looked at
        assert lib.fa_cache_weights(R(p), 6 * F, 8 * F, R(c), R(t), None, None, None, 64, 7 * F, None) == code


def test_c_abi_refuses_buffers_of_prefill(lib):
    R = ctypes.byref
    p, c, t = _structs()
    need = lib.fa_prefill_workspace_size(R(p), R(c), R(t))
    assert need > 0
    go = lambda q=6 * F, n=None, m=None, o=7 * F, lse=8 * F, ws=9 * F, size=need: lib.fa_prefill(  # noqa: E731
        R(p), q, R(c), R(t), n, m, o, lse, ws, size, None)
    assert go(q=None) == 1 and go(o=None) == 1 and go(lse=None) == 1 and go(q=6 * F + 8) == 1 and go(n=10 * F + 4) == 1
    assert go(m=10 * F + 4) == 1 and go(o=6 * F) == 1 and go(lse=7 * F + 16) == 1 and go(o=F) == 1 and go(o=5 * F) == 1
    assert go(n=7 * F) == 1 and go(m=8 * F) == 1
    assert go(size=need - 1) == ft.FA_ERR_WORKSPACE and go(ws=None) == ft.FA_ERR_WORKSPACE and go(ws=9 * F + 16) == 1 and go(ws=6 * F) == 1
    assert lib.fa_prefill(None, 6 * F, R(c), R(t), None, None, 7 * F, 8 * F, 9 * F, need, None) == 1
    assert lib.fa_prefill(R(p), 6 * F, None, R(t), None, None, 7 * F, 8 * F, 9 * F, need, None) == 1
    p.Sq = 0
    assert lib.fa_prefill(R(p), 6 * F, R(c), R(t), None, None, 7 * F, 8 * F, None, 0, None) == ft.FA_OK   # nothing to do
    p.Sq, t.B, c.Hkv, p.Hq = 1 << 24, 64, 2, 4
    assert lib.fa_prefill(R(p), 6 * F, R(c), R(t), None, None, 7 * F, 8 * F, 9 * F, 1 << 40, None) == ft.FA_ERR_UNSUPPORTED


def _cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_before_the_library(lib, monkeypatch):
    pool = (_cpu(9, 2, 16, 64, dtype=torch.int8), _cpu(9, 2, 16, 2, dtype=torch.float16)) * 2
    q, table, n = _cpu(2, 4, 8, 64), _cpu(2, 4, dtype=torch.int32), _cpu(2, dtype=torch.int64)
    ok = lambda **kw: kv.prefill(**{**dict(q=q, k_q=pool[0], k_d=pool[1], v_q=pool[2], v_d=pool[3], table=table,  # noqa: E731
                                           stream=0), **kw})
    with pytest.raises(ValueError, match="contiguous CUDA tensor"):
        ok()
    ran = []
    monkeypatch.setattr(ft, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(ft, "_launch", lambda device, call, *a: ran.append(a))
    ok(lengths=n, count=n, out=_cpu(2, 4, 8, 64), lse=_cpu(2, 4, 8, dtype=torch.float32))
    ok(table=_cpu(2, 7, dtype=torch.int32)[:, 1:4])   # rows of a larger table
    assert len(ran) == 2
    for kw, exc in [(dict(q=_cpu(3, 4, 8, 64)), ValueError), (dict(q=_cpu(2, 4, 8, 128)), ValueError),
                    (dict(q=_cpu(2, 4, 8, 64, dtype=torch.float32)), TypeError), (dict(q=_cpu(2, 8, 64)), ValueError),
                    (dict(table=table.long()), TypeError), (dict(table=table[0]), ValueError),
                    (dict(table=_cpu(4, 2, dtype=torch.int32).T), ValueError),
                    (dict(table=_cpu(3, 4, dtype=torch.int32)), ValueError), (dict(layout="sbhd"), ValueError),
                    (dict(k_d=pool[1][..., :1]), ValueError), (dict(v_q=pool[2][:8]), ValueError),
                    (dict(lengths=n.int()), TypeError), (dict(lengths=n[:1]), ValueError), (dict(count=_cpu(4, dtype=torch.int64)[::2]), ValueError),
                    (dict(out=_cpu(2, 4, 8, 128)), ValueError), (dict(lse=_cpu(2, 8, 4, dtype=torch.float32)), ValueError),
                    (dict(workspace=_cpu(1 << 12, 2)[:, 0]), ValueError)]:
        with pytest.raises(exc):
            ok(**kw)
    assert len(ran) == 2
