"""The attention weight that keys got from decoded tokens (fa_cache_weights_decoded), whose keys are not rounded to bf16, against the
fp64 oracle, and their sum against 1.

Tolerance. Each value d n is a bf16 number and another (4 bits: exactly; 8 bits: to within 2^-17 of it), whose products with q are exact in
fp32 and summed up apart, in D / 16 <= 8 steps of 16 with at most 17 truncations of 2^-24 of what has been added up: 136 for the first,
2^-8 of that for the second, one for their sum, and 2^7 of 2^-24 for the value's own: a score is off by E = 272 2^-24 scale
sum_d |q_d k_d| at most. The rest is tests/test_cache_weights.py's:
    |dW| <= sum exp(s - lse) (E + 2^-22 (|s| + |LSE|) + 2^-21 + n 2^-24) + 2^-24 |W|,
and for each 16 rows behind the first, whose sum is added to what the ones before left, 2^-24 |W| more.
The LSE of decode is off by what tests/test_decode.py says, E' + 2^-20 (1 + |LSE|), and all of a token's weights by the factor e to that.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from backward_adapter_gb300 import build as fbuild
from backward_adapter_gb300 import cache as kv
from backward_adapter_gb300 import fa_train as ft
from oracle import kv_cache as ref
from oracle import paged
from tests import paged_util as pu
from tests.test_decode import score_error

STEP = 272 * 2.0 ** -24


def bound(q, k, lse, lengths, scale, window):
    """(what a key's weight may be off by but for n 2^-24 and the sums' own, per key; the largest E + ... per token)."""
    B, Hq, Sq, _ = q.shape
    Hkv, S = k.shape[1:3]
    G = Hq // Hkv
    per_key, per_token = np.zeros((B, Hkv, S)), np.zeros((B, Hq, Sq))
    for b in range(B):
        for i in range(Sq):
            a, z = paged.seen_keys(int(lengths[b]), Sq, i, window)
            for h in range(Hq if z > a else 0):
                kk = k[b, h // G, a:z]
                s = scale * (kk @ q[b, h, i])
                e = STEP * abs(scale) * (np.abs(kk) @ np.abs(q[b, h, i])) + 2.0 ** -22 * (np.abs(s) + abs(lse[b, h, i])) + 2.0 ** -21
                per_key[b, h // G, a:z] += np.exp(s - lse[b, h, i]) * e
                per_token[b, h, i] = e.max()
    return per_key, per_token


def check(q, lse, planes, lengths, got, before, scale=None, window=0, layout="bhsd"):
    qn = q.double().cpu().numpy()
    qn = qn.swapaxes(1, 2) if layout == "bshd" else qn
    scale = 1 / math.sqrt(q.shape[-1]) if scale is None else scale
    n = pu.numpy_planes(planes)
    k, ln = ref.values(n[0], n[1]), lse.double().cpu().numpy()
    B, Hq, Sq, _ = qn.shape
    W, S = got.shape[2], min(got.shape[2], k.shape[2])
    k = k[:, :, :S]
    want, terms = paged.key_weights(qn, k, ln, lengths, [Sq] * B, scale, window)
    per_key, per_token = bound(qn, k, ln, lengths, scale, window)
    full, most = np.zeros(got.shape), np.zeros(got.shape)
    full[:, :, :S], most[:, :, :S] = want, per_key + want * terms * 2.0 ** -24
    if before is not None:
        full += before.double().cpu().numpy()
    launches = -(-(Hq // k.shape[1]) * Sq // 16)
    err = np.abs(got.double().cpu().numpy() - full)
    assert np.all(err <= most + launches * 2.0 ** -24 * np.abs(full)), (err.max(), most.max())
    return want, terms, per_token


def check_sum(q, lse, planes, lengths, got, want, per_token, scale=None, window=0):
    """got: from no weights. Every token that sees a key gives 1 in all."""
    scale = 1 / math.sqrt(q.shape[-1]) if scale is None else scale
    qn, ln = q.double().cpu().numpy(), lse.double().cpu().numpy()
    B, Hq, Sq, _ = qn.shape
    Hkv = planes[0].shape[1]
    sees = np.zeros((B, Hq, Sq), bool)
    for b in range(B):
        for i in range(Sq):
            a, z = paged.seen_keys(int(lengths[b]), Sq, i, window)
            sees[b, :, i] = z > a
    off = np.where(sees, np.expm1(per_token + score_error(qn, planes, lengths, scale, window) + 2.0 ** -20 * (1 + np.abs(ln))), 0)
    total, limit = (x.reshape(B, Hkv, -1).sum(-1) for x in (sees, off))
    n = (Hq // Hkv) * Sq   # terms of a key, at most
    err = np.abs(got.double().cpu().numpy().sum(-1) - total)
    assert np.all(err <= limit + total * n * 2.0 ** -23), (err.max(), limit.max())
    return np.abs(total), limit + total * n * 2.0 ** -23


# B, Hq, Hkv, S, D, Sq, P, lengths, window
SHAPES = {
    "one_key": (1, 1, 1, 1, 64, 1, 16, [1], 0),
    "a_token_each": (4, 8, 2, 300, 128, 1, 16, [300, 0, 128, 129], 0),
    "eight_rows": (2, 8, 1, 260, 64, 1, 48, [257, 3], 0),
    "nine_rows": (3, 9, 1, 130, 64, 1, 16, [130, 1, 33], 0),
    "draft_of_4": (2, 8, 2, 260, 64, 4, 48, [257, 3], 0),
    "twenty_rows": (3, 8, 2, 300, 128, 5, 16, [300, 2, 177], 0),
    "sixteen_tokens": (2, 6, 2, 400, 64, 16, 16, [399, 9], 0),
    "group_of_40": (1, 40, 1, 150, 128, 2, 16, [150], 0),
    "window": (2, 8, 2, 700, 64, 3, 112, [700, 77], 50),
    "window_of_one": (1, 3, 1, 300, 128, 2, 16, [300], 1),
    "many_heads": (60, 8, 4, 300, 64, 1, 16, [(37 * i) % 300 for i in range(60)], 0),
    "long": (1, 4, 1, 5000, 128, 1, 64, [4999], 0),
}


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("name", list(SHAPES))
def test_decoded_weights_against_the_oracle(name, fmt):
    B, Hq, Hkv, S, D, Sq, P, lengths, window = SHAPES[name]
    planes, pool, table = pu.make(B, Hkv, S, D, fmt, P, len(name))
    q, lens, t = pu.queries(B, Hq, Sq, D, 3), pu.i64(lengths), pu.unused(table, lengths, P)
    _, lse = kv.decode(q, *pool, lens, table=t, window=window)
    before = torch.rand((B, Hkv, S), generator=torch.Generator().manual_seed(9)).cuda()
    keep = before.clone()
    go = lambda w, **kw: kv.cache_weights(q, lse, *(kw.pop("planes", pool)[:2]), lens, weights=w, window=window, decoded=True, **kw)  # noqa: E731
    got = go(before, table=t)
    assert torch.equal(before, keep)
    check(q, lse, planes, lengths, got, before, window=window)
    assert torch.equal(go(before, planes=planes), got)
    go(before, out=before, table=t)
    assert torch.equal(before, got)   # in place
    new = go(None, table=t)
    want, terms, per_token = check(q, lse, planes, lengths, new, None, window=window)
    assert not new[:, :, :S].cpu().numpy()[terms[:, :, :S] == 0].any() and not new[:, :, S:].any()
    check_sum(q, lse, planes, lengths, new, want, per_token, window=window)
    assert ft.device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("Sq", [1, 5])
@pytest.mark.parametrize("kw", [dict(layout="bshd"), dict(scale=-0.3), dict(scale=0.0), dict(scale=0.9, layout="bshd", window=19)],
                         ids=lambda kw: "_".join(f"{k}{v}" for k, v in kw.items()))
def test_decoded_weights_layouts_and_scales(kw, Sq):
    planes, pool, table = pu.make(2, 2, 190, 128, "q4_0", 16, 5)
    q, lens = pu.queries(2, 8, Sq, 128, 6, kw.get("layout", "bhsd")), [190, 81]
    _, lse = kv.decode(q, *pool, pu.i64(lens), table=table, **kw)
    got = kv.cache_weights(q, lse, *pool[:2], pu.i64(lens), table=table, decoded=True, **kw)
    check(q, lse, planes, lens, got, None, kw.get("scale"), kw.get("window", 0), kw.get("layout", "bhsd"))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
def test_strong_keys_add_up_to_1_with_unrounded_keys_only(fmt):
    """Features that make scores of hundreds: what rounding K does to a weight is then far more than what fp32 does."""
    planes, pool, table = pu.make(2, 2, 512, 128, fmt, 64, 3, strong=60.0)
    q = pu.queries(2, 8, 2, 128, 4)
    _, lse = kv.decode(q, *pool, table=table)
    got, rounded = (kv.cache_weights(q, lse, *pool[:2], table=table, decoded=d) for d in (True, False))
    want, _, per_token = check(q, lse, planes, [512] * 2, got, None)
    total, limit = check_sum(q, lse, planes, [512] * 2, got, want, per_token)
    assert np.any(np.abs(rounded.double().cpu().numpy().sum(-1) - total) > 2 * limit)
    assert ft.device_status() == 0


@pytest.mark.gpu
def test_decoded_weights_step_by_step_and_in_a_graph():
    """Tokens of a draft at once and without lengths; a captured step replayed; on another stream; rows that are 16 and more."""
    planes, pool, table = pu.make(3, 2, 160, 64, "q8_0", 32, 8)
    q = pu.queries(3, 8, 6, 64, 2)
    _, lse = kv.decode(q, *pool, table=table)
    first = kv.cache_weights(q, lse, *pool[:2], table=table, decoded=True)
    check(q, lse, planes, [160] * 3, first, None)
    w, want = first.clone(), [first]
    for _ in range(3):
        want.append(kv.cache_weights(q, lse, *pool[:2], weights=want[-1], table=table, decoded=True))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.cache_weights(q, lse, *pool[:2], weights=w, out=w, table=table, decoded=True)
    for x in want[1:]:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(w, x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kv.cache_weights(q, lse, *pool[:2], table=table, decoded=True, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, first)
    bad = kv.cache_weights(q, lse, *pool[:2], pu.i64([161, 160, 160]), table=table, decoded=True)
    assert ft.device_status() == 0x40000000 | 952 and torch.equal(bad, first)
    none = kv.cache_weights(q[:, :, :0].contiguous(), lse[:, :, :0].contiguous(), *pool[:2], weights=first, table=table, decoded=True)
    assert torch.equal(none, first)


F = 1 << 40


def test_c_abi_refuses_decoded_weights():
    fbuild.build()
    lib, R = ft.load_library(), ctypes.byref

    def go(Hq=4, Sq=8, window=0, layout=0, scale=0.1, reserved=0, q=6 * F, lse=7 * F, n=None, w=None, W=64, out=8 * F, D=64, none=False):
        p, t = ft.FaDecodeParams(Hq, Sq, window, layout, scale, reserved), ft.FaPages(5 * F, 4, 2, 4)
        c = ft.FaCache(9, 2, 16, D, ft.FA_KV_Q8_0, 0, F, 2 * F, None, None)
        return lib.fa_cache_weights_decoded(None if none else R(p), q, lse, R(c), R(t), n, w, W, out, None)
    assert go(none=True) == 1 and go(Sq=17) == 1 and b"Sq=17" in lib.fa_last_error() and go(Sq=-1) == 1 and go(Hq=5) == 1 and go(window=-1) == 1
    assert go(layout=2) == 1 and go(scale=float("nan")) == 1 and go(reserved=1) == 1 and go(D=96) == 2 and go(W=0) == 1 and go(W=(1 << 30) + 1) == 1
    assert go(q=None) == 1 and go(lse=None) == 1 and go(out=None) == 1 and go(n=7 * F + 4) == 1 and go(w=8 * F + 16) == 1 and go(out=F) == 1
    assert go(out=6 * F) == 1 and go(out=7 * F) == 1 and go(out=5 * F) == 1 and go(n=8 * F) == 1


def test_binding_of_decoded_weights(monkeypatch):
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt)  # noqa: E731
    k_q, k_d = z(9, 2, 16, 64, dt=torch.int8), z(9, 2, 16, 2, dt=torch.float16)
    q, lse, table, n = z(2, 4, 8, 64, dt=torch.bfloat16), z(2, 4, 8), z(2, 4, dt=torch.int32), z(2, dt=torch.int64)
    ran, lib = [], ft.load_library()
    monkeypatch.setattr(ft, "_need_cuda", lambda *a: None)
    monkeypatch.setattr(ft, "_launch", lambda device, call, *a: ran.append((call, len(a))))
    go = lambda **kw: kv.cache_weights(q, lse, k_q, k_d, n, table=table, stream=0, **kw)  # noqa: E731
    go(decoded=True)
    go()
    assert ran == [(lib.fa_cache_weights_decoded, 10), (lib.fa_cache_weights, 11)]
    with pytest.raises(ValueError, match="no count"):
        go(decoded=True, count=n)
