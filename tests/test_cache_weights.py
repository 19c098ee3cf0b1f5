"""The attention weight that keys got (fa_cache_weights) against the fp64 oracle.

Tolerance. With E the error of a score (bf16 products exact in fp32, a sum of D of them in steps of 16, 17 truncations of 2^-24
each: 2^-17 scale sum_d |q_d k_d|), the exponent of a term is off by E, by the roundings of the score's and the LSE's
factors and of their difference, 2^-23 (2 |s| + 2 |LSE|), and its exponential by 2^-21 of its value; a sum of n positive terms in
fp32 by n 2^-24 of it at most, and adding it to what was there by half a step of the result:
    |dW| <= sum exp(s - lse) (E + 2^-22 (|s| + |LSE|) + 2^-21 + n 2^-24) + 2^-24 |W|.
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


def bound(q, k, lse, lengths, counts, scale, window):
    """The sum's bound of the module's comment but for n 2^-24, for every key."""
    B, Hq, Sq, _ = q.shape
    Hkv, S = k.shape[1:3]
    G = Hq // Hkv
    out = np.zeros((B, Hkv, S))
    for b in range(B):
        for i in range(int(counts[b])):
            a, z = paged.seen_keys(int(lengths[b]), int(counts[b]), i, window)
            for h in range(Hq if z > a else 0):
                kk = k[b, h // G, a:z]
                s = scale * (kk @ q[b, h, i])
                e = 2.0 ** -17 * abs(scale) * (np.abs(kk) @ np.abs(q[b, h, i]))
                out[b, h // G, a:z] += np.exp(s - lse[b, h, i]) * (e + 2.0 ** -22 * (np.abs(s) + abs(lse[b, h, i])) + 2.0 ** -21)
    return out


def check(q, lse, planes, lengths, counts, got, before, scale=None, window=0, layout="bhsd"):
    qn = q.double().cpu().numpy()
    qn = qn.swapaxes(1, 2) if layout == "bshd" else qn
    scale = 1 / math.sqrt(q.shape[-1]) if scale is None else scale
    k, _ = pu.rounded_kv(planes)
    ln = lse.double().cpu().numpy()
    W = got.shape[2]
    k = k[:, :, :W]
    want, terms = paged.key_weights(qn, k, ln, lengths, counts, scale, window)
    limit = bound(qn, k, ln, lengths, counts, scale, window) + want * terms * 2.0 ** -24
    full = np.zeros(got.shape)
    full[:, :, :k.shape[2]] = want
    most = np.zeros(got.shape)
    most[:, :, :k.shape[2]] = limit
    if before is not None:
        full += before.double().cpu().numpy()
    err = np.abs(got.double().cpu().numpy() - full)
    assert np.all(err <= most + 2.0 ** -24 * np.abs(full)), (err.max(), most.max())
    dead = np.zeros(got.shape, bool)
    dead[:, :, :k.shape[2]] = terms == 0
    dead[:, :, k.shape[2]:] = True
    assert np.all(err[dead] == 0)   # keys that nobody sees keep what they had


# B, Hq, Hkv, S, D, Sq, P, lengths, counts (None: all), window
SHAPES = {
    "one_key": (1, 1, 1, 1, 64, 1, 16, [1], None, 0),
    "a_token_each": (4, 8, 2, 300, 128, 1, 16, [300, 0, 128, 129], None, 0),
    "draft_of_4": (2, 8, 2, 260, 64, 4, 48, [257, 3], None, 0),
    "seventeen_rows": (1, 17, 1, 140, 128, 1, 16, [131], None, 0),
    "ragged": (4, 6, 2, 300, 64, 77, 16, [300, 5, 129, 128], [77, 5, 0, 64], 0),
    "more_tokens_than_keys": (2, 4, 1, 130, 128, 140, 48, [5, 130], None, 0),
    "whole_prompt": (1, 4, 2, 640, 128, 640, 64, [640], None, 0),
    "window": (2, 4, 2, 700, 64, 100, 112, [700, 350], [100, 13], 130),
    "window_of_one": (1, 3, 1, 300, 128, 300, 16, [300], None, 1),
    "group_of_300": (1, 300, 1, 90, 64, 3, 16, [77], None, 0),
    "many_rows": (1, 8, 1, 256, 64, 250, 16, [256], None, 0),
    "nine_rows": (3, 9, 1, 130, 64, 1, 16, [130, 1, 33], None, 0),
    "sixteen_rows_in_a_window": (2, 8, 2, 400, 128, 4, 48, [399, 77], [4, 1], 50),
    "many_heads": (60, 8, 4, 300, 64, 3, 16, [1 + (37 * i) % 300 for i in range(60)], [i % 4 for i in range(60)], 0),
    "several_units_a_block": (4, 20, 20, 900, 64, 40, 64, [900, 257, 0, 600], [40, 33, 0, 40], 300),
}


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("name", list(SHAPES))
def test_weights_against_the_oracle(name, fmt):
    B, Hq, Hkv, S, D, Sq, P, lengths, counts, window = SHAPES[name]
    planes, pool, table = pu.make(B, Hkv, S, D, fmt, P, len(name))
    q = pu.queries(B, Hq, Sq, D, 3)
    cnts = [Sq] * B if counts is None else counts
    lens, cn, t = pu.i64(lengths), pu.i64(counts), pu.unused(table, lengths, P)
    lse = torch.zeros((B, Hq, Sq), device="cuda")
    kv.prefill(q, *pool, lens, cn, table=t, window=window, lse=lse)
    g = torch.Generator().manual_seed(9)
    before = torch.rand((B, Hkv, S), generator=g).cuda()
    keep = before.clone()
    got = kv.cache_weights(q, lse, pool[0], pool[1], lens, cn, weights=before, table=t, window=window)
    assert torch.equal(before, keep)
    check(q, lse, planes, lengths, cnts, got, before, window=window)
    flat = kv.cache_weights(q, lse, planes[0], planes[1], lens, cn, weights=before, window=window)
    assert torch.equal(flat, got)
    kv.cache_weights(q, lse, pool[0], pool[1], lens, cn, weights=before, out=before, table=t, window=window)
    assert torch.equal(before, got)   # in place
    new = kv.cache_weights(q, lse, pool[0], pool[1], lens, cn, table=t, window=window)
    assert new.shape[2] == planes[0].shape[2]
    check(q, lse, planes, lengths, cnts, new, None, window=window)
    total = sum(min(int(c), int(n)) if window == 0 else 0 for n, c in zip(lengths, cnts)) * Hq
    if window == 0:   # every token that sees a key gives a weight of 1 in all
        assert abs(float(new.double().sum()) - total) <= 2.0 ** -12 * max(total, 1)
    assert ft.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(layout="bshd"), dict(scale=-0.3), dict(scale=0.0), dict(scale=0.9, layout="bshd", window=19)],
                         ids=lambda kw: "_".join(f"{k}{v}" for k, v in kw.items()))
@pytest.mark.parametrize("Sq", [2, 70])
def test_weights_layouts_and_scales(kw, Sq):
    planes, pool, table = pu.make(2, 2, 190, 128, "q4_0", 16, 5)
    q = pu.queries(2, 6, Sq, 128, 6, kw.get("layout", "bhsd"))
    lens, cnts = [190, 81], [Sq, Sq // 2]
    lse = torch.zeros((2, 6, Sq), device="cuda")
    kv.prefill(q, *pool, pu.i64(lens), pu.i64(cnts), table=table, lse=lse, **kw)
    got = kv.cache_weights(q, lse, pool[0], pool[1], pu.i64(lens), pu.i64(cnts), table=table, **kw)
    check(q, lse, planes, lens, cnts, got, None, kw.get("scale"), kw.get("window", 0), kw.get("layout", "bhsd"))


@pytest.mark.gpu
def test_weights_of_a_decoded_token_without_lengths():
    planes, pool, table = pu.make(3, 2, 160, 64, "q8_0", 32, 8)
    q = pu.queries(3, 4, 1, 64, 2)
    _, lse = kv.decode(q, *pool, table=table)
    got = kv.cache_weights(q, lse, pool[0], pool[1], table=table)
    check(q, lse, planes, [160] * 3, [1] * 3, got, None)


@pytest.mark.gpu
@pytest.mark.parametrize("W", [1, 100, 128, 500])
def test_weights_of_another_width_than_the_cache(W):
    """Shorter than the sequences: the keys behind it are left out, and reported; longer: the rest is what it was."""
    planes, pool, table = pu.make(2, 1, 200, 64, "q8_0", 16, 4)
    q = pu.queries(2, 2, 9, 64, 2)
    lens = [200, 90]
    lse = torch.zeros((2, 2, 9), device="cuda")
    kv.prefill(q, *pool, pu.i64(lens), table=table, lse=lse)
    before = torch.rand((2, 1, W), device="cuda")
    got = kv.cache_weights(q, lse, pool[0], pool[1], pu.i64(lens), weights=before, table=table)
    assert ft.device_status() == (0x40000000 | 952 if W < 200 else 0)
    all_keys = kv.cache_weights(q, lse, pool[0], pool[1], pu.i64(lens), table=table)
    n = min(W, 208)
    want = before.clone()
    want[:, :, :n] += all_keys[:, :, :n]
    assert torch.equal(got, want)


@pytest.mark.gpu
def test_weights_of_keys_and_rows_that_are_no_numbers():
    """A key that nobody sees, padding, and pages that are none change nothing elsewhere."""
    planes, pool, table = pu.make(2, 2, 200, 128, "q4_0", 16, 4)
    q = pu.queries(2, 4, 40, 128, 2)
    lens, cnts = pu.i64([180, 100]), pu.i64([40, 21])
    lse = torch.zeros((2, 4, 40), device="cuda")
    kv.prefill(q, *planes, lens, cnts, lse=lse, window=30)
    want = kv.cache_weights(q, lse, planes[0], planes[1], lens, cnts, window=30)
    dirty = [p.clone() for p in planes]
    dirty[1][0, :, 180:], dirty[1][0, :, :180 - 40 - 30], dirty[1][1, :, 100:] = float("nan"), float("inf"), float("nan")
    q[1, :, 21:], lse[1, :, 21:] = float("nan"), float("nan")
    got = kv.cache_weights(q, lse, dirty[0], dirty[1], lens, cnts, window=30)
    assert torch.equal(got, want)
    assert ft.device_status() == 0
    bad = table.clone()
    bad[1, 2] = -9
    got = kv.cache_weights(q, lse, pool[0], pool[1], lens, cnts, table=bad, window=30)
    assert ft.device_status() == 0x40000000 | 953
    assert torch.equal(got[0], want[0])


@pytest.mark.gpu
def test_weights_in_a_graph_and_on_streams():
    planes, pool, table = pu.make(3, 2, 900, 128, "q8_0", 64, 21)
    q = pu.queries(3, 8, 40, 128, 1)
    lens = pu.i64([900, 500, 64])
    _, lse = kv.prefill(q, *pool, lens, table=table)
    w = torch.zeros((3, 2, 900), device="cuda")
    want = [w.clone()]
    for _ in range(3):
        want.append(kv.cache_weights(q, lse, pool[0], pool[1], lens, weights=want[-1], table=table))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.cache_weights(q, lse, pool[0], pool[1], lens, weights=w, out=w, table=table)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(w, want[i + 1])
    side = torch.cuda.Stream()
    got = [kv.cache_weights(q, lse, pool[0], pool[1], lens, table=table, stream=s) for s in (None, side, side.cuda_stream)]
    torch.cuda.synchronize()
    assert all(torch.equal(x[:, :, :900], want[1]) for x in got)


F = 1 << 40


def test_c_abi_refuses_buffers_of_weights():
    fbuild.build()
    lib, R = ft.load_library(), ctypes.byref
    p = ft.FaPrefillParams(4, 8, 0, 0, 0.1, 0)
    c = ft.FaCache(9, 2, 16, 64, ft.FA_KV_Q8_0, 0, F, 2 * F, None, None)   # V is not looked at
    t = ft.FaPages(5 * F, 4, 2, 4)
    go = lambda q=6 * F, lse=7 * F, n=None, m=None, w=None, W=64, out=8 * F: lib.fa_cache_weights(  # noqa: E731
        R(p), q, lse, R(c), R(t), n, m, w, W, out, None)
    assert go(q=None) == 1 and go(lse=None) == 1 and go(out=None) == 1 and go(out=8 * F + 4) == 1 and go(W=0) == 1 and go(W=(1 << 30) + 1) == 1
    assert go(n=10 * F + 4) == 1 and go(m=10 * F + 4) == 1 and go(w=9 * F + 8) == 1 and go(w=8 * F + 16) == 1 and go(out=F) == 1
    assert go(out=6 * F) == 1 and go(out=7 * F) == 1 and go(out=5 * F) == 1 and go(n=8 * F) == 1 and go(m=8 * F) == 1
    t.B, t.stride = 65535, 4
    assert go(W=1 << 30) == ft.FA_ERR_UNSUPPORTED
    assert lib.fa_cache_weights(None, 6 * F, 7 * F, R(c), R(t), None, None, None, 64, 8 * F, None) == 1


def test_binding_refuses_weights(monkeypatch):
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt)  # noqa: E731
    k_q, k_d = z(9, 2, 16, 64, dt=torch.int8), z(9, 2, 16, 2, dt=torch.float16)
    q, lse, table = z(2, 4, 8, 64, dt=torch.bfloat16), z(2, 4, 8), z(2, 4, dt=torch.int32)
    ran = []
    monkeypatch.setattr(ft, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(ft, "_launch", lambda device, call, *a: ran.append(a))
    go = lambda **kw: kv.cache_weights(**{**dict(q=q, lse=lse, k_q=k_q, k_d=k_d, table=table, stream=0), **kw})  # noqa: E731
    assert go().shape == (2, 2, 64)
    assert go(out=z(2, 2, 70)).shape == (2, 2, 70) and go(weights=z(2, 2, 50)).shape == (2, 2, 50)
    for kw, exc in [(dict(lse=z(2, 8, 4)), ValueError), (dict(lse=lse.double()), ValueError), (dict(weights=z(2, 2, 5).double()), TypeError),
                    (dict(weights=z(2, 4, 50)), ValueError), (dict(weights=z(2, 2)), ValueError), (dict(weights=z(2, 2, 50), out=z(2, 2, 51)), ValueError),
                    (dict(q=q.float()), TypeError), (dict(lengths=z(3, dt=torch.int64)), ValueError), (dict(k_d=k_d.float()), TypeError)]:
        with pytest.raises(exc):
            go(**kw)
    assert len(ran) == 3
