"""Attention of the newest tokens over a quantized cache (fa_decode) against the fp64 oracle.

Tolerances, from the data of each case. A score is a sum of D products of whole numbers and q in fp32, block by block:
with Q_b the sum of |q| over a block, its partial sums stay below W Q_b (W = 8 in 4 bits, 127 in 8), and one accumulation of
17 terms is off by at most 17 truncations, 2^-19 of that for the two of a block and the sum over blocks.
So a score is off by at most E = 2^-19 scale sum_b |d_b| W Q_b over the keys a query sees; LSE by E and
the roundings of a logarithm near it, 2^-20 (1 + |LSE|). A weight p is off by the factor e^(+-E); in units in which the
largest one is at least 2^level, level = min(7, 21 - (the or of the exponent fields of the V scales it is summed with)), p and then
p * d are rounded to fp16: each is off by at most half a step, 2^-11 of its value (11 bits: a step is 2^-10 of the power of two
below it), 2^-10 for both, or 2^-25 where it is subnormal. The whole numbers
are at most W, sum p is at least 1, and the result is rounded to bf16, 2^-8 of its value, so with n keys and scales up to d
    |dO| <= (2^-10 + 2 E + 2^-16) sum p |v| / sum p + n W (1 + d) 2^(-25 - level) + 2^-8 |O|.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from backward_adapter_gb300 import cache as kv
from backward_adapter_gb300 import fa_train as ft
from oracle import kv_cache as ref


def planes_of(k, v, fmt):
    out = []
    for x in (k, v):
        out += [torch.from_numpy(t).cuda() for t in ref.quantize(x, fmt)]
    return out


def score_error(q, planes, lengths, scale, window):
    """E of the module's comment for every (b, head, token)."""
    B, Hq, Sq, D = q.shape
    d = np.abs(planes[1].cpu().numpy().astype(np.float64))
    w = 8.0 if planes[0].dtype == torch.uint8 else 127.0
    G = Hq // d.shape[1]
    e = np.zeros((B, Hq, Sq))
    qb = np.abs(q.reshape(B, Hq, Sq, D // 32, 32)).sum(-1)
    for b in range(B):
        for i in range(Sq):
            pos = int(lengths[b]) - Sq + i
            first = max(0, pos - window) if window > 0 else 0
            if pos < first:
                continue
            for h in range(Hq):
                e[b, h, i] = 2.0 ** -19 * abs(scale) * (d[b, h // G, first:pos + 1] @ (w * qb[b, h, i])).max()
    return e


def weight_step(planes, lengths, Hq, Sq, window):
    """n W (1 + d) 2^(-25 - level) of the module's comment for every (b, head, token)."""
    d = planes[3].cpu().numpy()
    bits = np.bitwise_or.reduce((d.view(np.uint16).astype(np.int64) >> 10) & 31, axis=-1)   # [B, Hkv, S]
    d = np.abs(d.astype(np.float64)).max(-1)
    w = 8.0 if planes[0].dtype == torch.uint8 else 127.0
    B, Hkv, _ = bits.shape
    out = np.zeros((B, Hq, Sq))
    for b in range(B):
        for i in range(Sq):
            pos = int(lengths[b]) - Sq + i
            first = max(0, pos - window) if window > 0 else 0
            if pos < first:
                continue
            level = np.minimum(7.0, 21.0 - np.bitwise_or.reduce(bits[b, :, first:pos + 1], axis=-1))
            step = (pos + 1 - first) * w * (1 + d[b, :, first:pos + 1].max(-1)) * 2.0 ** (-25.0 - level)
            out[b, :, i] = np.repeat(step, Hq // Hkv)
    return out


def check(q, planes, lengths, got, scale=None, window=0):
    o, lse = (t.double().cpu().numpy() for t in got)
    qn = q.double().cpu().numpy()
    scale = 1 / math.sqrt(q.shape[-1]) if scale is None else scale
    k, v = (ref.values(planes[i].cpu().numpy(), planes[i + 1].cpu().numpy()) for i in (0, 2))
    n = np.full(q.shape[0], k.shape[2]) if lengths is None else lengths.cpu().numpy()
    want, want_lse = ref.decode(qn, k, v, n, scale, window)
    size, _ = ref.decode(qn, k, np.abs(v), n, scale, window)
    E = score_error(qn, planes, n, scale, window)
    bad = np.abs(lse - want_lse) > E + 2.0 ** -20 * (1 + np.abs(want_lse))
    assert not bad.any(), (np.abs(lse - want_lse).max(), E.max())
    e, step = E[..., None], weight_step(planes, n, q.shape[1], q.shape[2], window)[..., None]
    err = np.abs(o - want)
    assert np.all(err <= (2.0 ** -10 + 2 * e + 2.0 ** -16) * size + step + 2.0 ** -8 * np.abs(want)), err.max()
    empty = want_lse == 0
    if empty.any():
        assert np.all(o[empty & (np.abs(want).sum(-1) == 0)] == 0)


def make(B, Hq, Hkv, S, D, Sq, fmt, seed):
    rng = np.random.default_rng(seed)
    k, v = (rng.standard_normal((B, Hkv, S, D)).astype(np.float32) for _ in range(2))
    k[..., ::29] *= 4
    q = torch.from_numpy(rng.standard_normal((B, Hq, Sq, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    return q, planes_of(k, v, fmt)


# B, Hq, Hkv, S, D, Sq, lengths (None: all), window
SHAPES = {
    "one_key": (1, 1, 1, 1, 64, 1, None, 0),
    "one_key_of_many": (2, 4, 2, 70, 128, 1, [1, 0], 0),
    "tile_edges": (6, 4, 1, 130, 128, 1, [31, 32, 33, 64, 127, 130], 0),
    "odd_heads": (2, 9, 3, 77, 64, 1, [77, 5], 0),
    "group_of_16": (1, 16, 1, 300, 128, 1, [299], 0),
    "group_of_40": (1, 40, 1, 45, 64, 1, None, 0),
    "two_tokens": (3, 4, 2, 90, 64, 2, [1, 0, 90], 0),
    "draft_of_5": (2, 8, 2, 200, 128, 5, [3, 200], 0),
    "draft_of_16": (1, 6, 2, 150, 64, 16, [77], 0),
    "split": (2, 8, 2, 1500, 128, 1, [1500, 700], 0),
    "split_ragged": (5, 4, 4, 1111, 64, 1, [0, 1, 257, 512, 1111], 0),
    "split_draft": (2, 4, 1, 1900, 128, 3, [1900, 2], 0),
    "split_group_of_40": (2, 40, 1, 1300, 64, 1, [1300, 33], 0),
    "split_heads": (3, 16, 8, 1200, 128, 1, [1200, 64, 1055], 0),
    "split_short_lengths": (7, 4, 2, 4000, 64, 1, [33, 1, 0, 64, 2, 31, 65], 0),
    "split_all_empty": (2, 4, 2, 4000, 64, 1, [0, 0], 0),
    "window": (3, 4, 2, 1000, 128, 1, [1000, 40, 555], 100),
    "window_of_1": (2, 4, 2, 400, 64, 1, [400, 1], 1),
    "window_draft": (2, 4, 2, 800, 64, 4, [799, 3], 33),
    "window_wider": (1, 4, 2, 600, 128, 1, [600], 5000),
    "window_split": (1, 2, 1, 3000, 64, 2, [2900], 1300),
}


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("name", SHAPES)
def test_matches_oracle(name, fmt):
    B, Hq, Hkv, S, D, Sq, lens, window = SHAPES[name]
    q, planes = make(B, Hq, Hkv, S, D, Sq, fmt, len(name))
    lengths = None if lens is None else torch.tensor(lens, device="cuda")
    got = kv.decode(q, *planes, lengths, window=window)
    torch.cuda.synchronize()
    assert ft.device_status() == 0
    check(q, planes, lengths, got, window=window)
    qt = q.transpose(1, 2).contiguous()
    o, lse = kv.decode(qt, *planes, lengths, window=window, layout="bshd")
    assert torch.equal(o.transpose(1, 2), got[0]) and torch.equal(lse, got[1])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("S", [200, 1400])
def test_what_hidden_keys_hold_does_not_matter(fmt, S):
    """Scales that are infinite or not numbers outside what a query sees: past the length, before the window, and, for
    the first token of a draft, in the later tokens' own keys."""
    B, Hq, Hkv, D, Sq, window = 2, 4, 2, 64, 3, 60
    q, planes = make(B, Hq, Hkv, S, D, Sq, fmt, 5)
    lens = [S - 40, 45]
    clean = kv.decode(q, *planes, torch.tensor(lens, device="cuda"), window=window)
    for b, n in enumerate(lens):
        for i in (1, 3):
            planes[i][b, :, n:] = float("inf")
            planes[i][b, :, n + 3] = float("nan")
            planes[i][b, :, :max(0, n - Sq - window)] = float("nan")
    dirty = kv.decode(q, *planes, torch.tensor(lens, device="cuda"), window=window)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])
    for bad in (float("nan"), float("inf")):   # the last key is seen by the last token alone
        for i in (1, 3):
            planes[i][0, :, lens[0] - 1] = bad
        part = kv.decode(q, *planes, torch.tensor(lens, device="cuda"), window=window)
        assert torch.equal(part[0][:, :, :2], clean[0][:, :, :2]) and torch.equal(part[1][:, :, :2], clean[1][:, :, :2])
        assert bool(part[0][0, :, 2].isnan().all())
        assert torch.equal(part[0][1], clean[0][1])


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_any_finite_scale(scale):
    q, planes = make(2, 4, 2, 700, 64, 1, "q4_0", 9)
    got = kv.decode(q, *planes, scale=scale)
    check(q, planes, None, got, scale=scale)


@pytest.mark.gpu
def test_lengths_outside_the_cache_are_held_to_it_and_reported():
    q, planes = make(3, 4, 2, 100, 64, 1, "q8_0", 10)
    ft.device_status()
    got = kv.decode(q, *planes, torch.tensor([101, -1, 1 << 40], device="cuda"))
    torch.cuda.synchronize()
    assert ft.device_status() == (0x40000000 | 952)
    want = kv.decode(q, *planes, torch.tensor([100, 0, 100], device="cuda"))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert ft.device_status() == 0


@pytest.mark.gpu
def test_no_tokens_and_given_outputs():
    q, planes = make(2, 4, 2, 1400, 64, 1, "q4_0", 11)
    o, lse = kv.decode(q[:, :, :0].contiguous(), *planes)
    assert o.shape == (2, 4, 0, 64) and lse.shape == (2, 4, 0)
    want = kv.decode(q, *planes)
    out, lse = torch.empty_like(q), torch.empty((2, 4, 1), device="cuda")
    ws = torch.full((1 << 22,), 0xff, dtype=torch.uint8, device="cuda")   # garbage: NaN in every float
    got = kv.decode(q, *planes, out=out, lse=lse, workspace=ws)
    assert got[0] is out and torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
def test_offsets_beyond_32_bits(fmt):
    B, Hkv, S, D = 2, 8, (1 << 21) + 5, 128
    width, kind = (D // 2, torch.uint8) if fmt == "q4_0" else (D, torch.int8)
    planes = []
    for _ in range(2):
        planes.append(torch.empty((B, Hkv, S, width), dtype=kind, device="cuda"))
        planes.append(torch.empty((B, Hkv, S, D // 32), dtype=torch.float16, device="cuda"))
    q, small = make(1, 16, Hkv, 333, D, 1, fmt, 12)
    at = S - 333 - 2
    for p, s in zip(planes, small):
        p[1, :, at:at + 333] = s[0]
    got = kv.decode(torch.cat([q, q]), *planes, torch.tensor([0, at + 333], device="cuda"), window=332)
    want = kv.decode(q, *small)
    torch.cuda.synchronize()
    assert bool((got[0][0] == 0).all()) and bool((got[1][0] == 0).all())
    # the same keys in other tiles: the same weights, added in another order
    assert torch.allclose(got[1][1], want[1][0], rtol=2.0 ** -18, atol=2.0 ** -18)
    assert torch.allclose(got[0][1].float(), want[0][0].float(), rtol=2.0 ** -7, atol=2.0 ** -7)


def test_bad_arguments_are_refused_before_launch():
    from backward_adapter_gb300 import build as fbuild
    fbuild.build()
    lib = ft.load_library()
    R = ctypes.byref
    F = 1 << 34
    c = ft.FaCache(2, 3, 4000, 64, ft.FA_KV_Q8_0, 0, F, 2 * F, 3 * F, 4 * F)

    def p(**kw):
        x = ft.FaDecodeParams(6, 1, 0, 0, 0.125, 0)
        for n, v in kw.items():
            setattr(x, n, v)
        return x
    need = lib.fa_decode_workspace_size(R(p()), R(c))
    assert need > 0
    go = lambda pp=p(), q=5 * F, n=None, o=6 * F, lse=7 * F, ws=8 * F, size=need: lib.fa_decode(  # noqa: E731
        R(pp), q, R(c), n, o, lse, ws, size, None)
    for kw in (dict(Hq=0), dict(Hq=7), dict(Hq=70000), dict(Sq=-1), dict(Sq=17), dict(window=-1), dict(layout=3),
               dict(scale=float("nan")), dict(reserved=1)):
        assert go(p(**kw)) == ft.FA_ERR_INVALID_ARG, kw
        assert lib.fa_decode_workspace_size(R(p(**kw)), R(c)) == 0
    assert lib.fa_decode(None, 5 * F, R(c), None, 6 * F, 7 * F, 8 * F, need, None) == ft.FA_ERR_INVALID_ARG
    for kw in (dict(q=None), dict(q=5 * F + 8), dict(o=None), dict(o=F + 64), dict(lse=6 * F), dict(lse=7 * F + 4),
               dict(n=9 * F + 4), dict(n=6 * F + 16), dict(ws=8 * F + 16), dict(ws=5 * F)):
        assert go(**kw) == ft.FA_ERR_INVALID_ARG, kw
    assert go(size=need - 1) == ft.FA_ERR_WORKSPACE and go(ws=None) == ft.FA_ERR_WORKSPACE
    assert go(p(Sq=0), ws=None, size=0) == ft.FA_OK


def test_binding_refuses_what_does_not_fit():
    planes = kv.new_cache(2, 3, 40, 64, "q8_0", device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        kv.decode(torch.zeros(2, 6, 1, 64, dtype=torch.bfloat16), *planes)


def test_oracle_is_attention_of_a_causal_chunk():
    """The oracle of the newest tokens is the training oracle's causal chunk at the end of the keys."""
    from oracle import attention as attn
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((1, 4, 3, 64)), rng.standard_normal((1, 2, 20, 64)), rng.standard_normal((1, 2, 20, 64))
    for window in (0, 6):
        o, lse = ref.decode(q, k, v, [20], 0.125, window)
        r = attn.backward(q, k, v, np.zeros_like(q), 0.125, causal=True, q_offset=17, window=window)
        np.testing.assert_allclose(o, r["o"], atol=1e-13)
        np.testing.assert_allclose(lse, r["lse"], atol=1e-13)


@pytest.mark.gpu
def test_windows_longer_than_any_cache_hide_nothing():
    q, planes = make(2, 4, 2, 1400, 64, 2, "q4_0", 21)
    want = kv.decode(q, *planes)
    for window in (1400, (1 << 31) - 1, 1 << 31, (1 << 32) + 3, 1 << 70):
        got = kv.decode(q, *planes, window=window)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for window in (-1, -(1 << 32) + 5):
        with pytest.raises(ft.FaError, match="window"):
            kv.decode(q, *planes, window=window)


@pytest.mark.gpu
def test_workspaces_that_do_not_fit_the_call_are_refused():
    q, planes = make(2, 4, 2, 1400, 64, 1, "q4_0", 22)
    for ws in (torch.empty(1 << 22, dtype=torch.uint8),
               torch.empty((2, 1 << 22), dtype=torch.uint8, device="cuda").t()):
        with pytest.raises(ValueError, match="workspace"):
            kv.decode(q, *planes, workspace=ws)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,D", [("q4_0", 128), ("q8_0", 64)])
def test_many_short_sequences_in_a_roomy_cache(fmt, D):
    """Heads of a few tiles, of one and of none, so that runs and slices begin and end with a head's beginning."""
    B, S = 50, 700 if D == 128 else 1056
    q, planes = make(B, 8, 4, S, D, 1, fmt, 23)
    g = torch.Generator().manual_seed(24)
    lens = torch.randint(0, 130, (B,), generator=g)
    lens[::7] = 0
    lens[5], lens[44], lens[-1] = S, 1, 32
    got = kv.decode(q, *planes, lens.cuda())
    check(q, planes, lens, got)
    again = kv.decode(q, *planes, lens.cuda())
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("D,fmt", [(64, "q4_0"), (128, "q4_0"), (128, "q8_0")])
@pytest.mark.parametrize("B", [128, 129, 700, 1024, 1025])
def test_sequences_on_both_sides_of_the_lists_sizes(B, D, fmt):
    """Short sequences in a roomy cache against the same in a small one, which takes another path: the same weights,
    added in another order."""
    S, g = 1056 if D == 64 else 544, torch.Generator(device="cuda").manual_seed(B)
    planes = kv.new_cache(B, 2, S, D, fmt)
    for i in (0, 2):
        planes[i].random_(*((0, 256) if fmt == "q4_0" else (-127, 128)), generator=g)
        planes[i + 1].copy_(torch.rand(planes[i + 1].shape, device="cuda", generator=g) * 0.1)
    q = torch.randn((B, 6, 1, D), device="cuda", generator=g).to(torch.bfloat16)
    lens = torch.randint(0, 65, (B,), device="cuda", generator=g)
    got = kv.decode(q, *planes, lens)
    want = kv.decode(q, *(t[:, :, :64].contiguous() for t in planes), lens)
    torch.cuda.synchronize()
    assert torch.allclose(got[1], want[1], rtol=2.0 ** -18, atol=2.0 ** -18)
    # both are off by two fp16 half steps of each weight, 2^-10 of the largest value, and a bf16 half step of the result
    top = float(planes[3].max()) * (8 if fmt == "q4_0" else 127)
    assert torch.allclose(got[0].float(), want[0].float(), rtol=2.0 ** -7, atol=2.0 ** -9 * top)
    assert bool((got[0][lens == 0] == 0).all()) and bool((got[1][lens == 0] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("D,Sq", [(64, 1), (128, 1), (64, 5), (128, 5)])
def test_blocks_with_an_sm_to_themselves(D, Sq, fmt):
    """Few heads of a moderate length: a wide block for each, with tiles for all of its warps, for some and for none."""
    q, planes = make(4, 8, 4, 900, D, Sq, fmt, 25)
    lens = torch.tensor([900, 33, 0, 517])
    for window in (0, 250):
        got = kv.decode(q, *planes, lens.cuda(), window=window)
        check(q, planes, lens, got, window=window)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("D,G", [(64, 1), (128, 4), (128, 12)])
def test_many_heads_of_any_length(D, G, fmt):
    """Twice as many heads as SMs and more, cut anywhere, against each sequence by itself, whose few heads take other
    paths: the same weights, added in another order."""
    B, Hkv, S = 80, 4, 800 if D == 128 else 1500
    gen = torch.Generator(device="cuda").manual_seed(26)
    planes = kv.new_cache(B, Hkv, S, D, fmt)
    for i in (0, 2):
        planes[i].random_(*((0, 256) if fmt == "q4_0" else (-127, 128)), generator=gen)
        planes[i + 1].copy_(torch.rand(planes[i + 1].shape, device="cuda", generator=gen) * (0.1 if fmt == "q4_0" else 0.01))
    q = torch.randn((B, Hkv * G, 1, D), device="cuda", generator=gen).to(torch.bfloat16)
    lens = torch.randint(0, S + 1, (B,), device="cuda", generator=gen)
    lens[3], lens[4], lens[5] = 0, S, 1
    got = kv.decode(q, *planes, lens)
    for b in list(range(8)) + [40, 78, 79]:
        want = kv.decode(q[b:b + 1], *(t[b:b + 1] for t in planes), lens[b:b + 1])
        assert torch.allclose(got[1][b], want[1][0], rtol=2.0 ** -18, atol=2.0 ** -18)
        # as above
        top = float(planes[3][b].max()) * (8 if fmt == "q4_0" else 127)
        err = (got[0][b].float() - want[0][0].float()).abs()
        assert bool((err <= 2.0 ** -9 * top + 2.0 ** -7 * want[0][0].float().abs()).all()), float(err.max())
