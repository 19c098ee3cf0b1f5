"""fa_decode where weights and V's scales differ by many powers of two: a first key that takes most of the weight and has
small values (an attention sink) or none, single large values elsewhere, scales on both sides of 1, 2 and 4, and scales near
fp16's smallest. Against the definition in 64 bits, with a bound in the output's own terms.

Derivation. In every case here a key's weight times its block's scale is within 2^-24 of the largest such product of
its query row: weights differ by 14 nats (2^-20.2) at most, and where the heaviest key's scales are not zero they are so small, or
the others' so large, that 2^-14 remains. Such a product is rounded once to fp16, off by at most half a step, 2^-11 of its value.
Scores, exponentials and sums are fp32: with W the largest whole number of the format (8, 127) and Q_b the sum of |q| over a
block, a score is off by E = 2^-19 scale max_j sum_b |d_jb| W Q_b (two accumulations of 17 terms a block, see
test_decode), a weight and the sum of weights each by E and by the rounding of an exponent below 64 to fp32 (2^-18 of the weight);
the accumulations over n <= 4608 keys and the matrix instructions' truncations stay below 2^-12 of sum p |v|. With the
result's rounding to bf16, 2^-8 of it,
    |dO| <= (2^-11 + 2^-12 + 2 E + 2^-16) sum p |v| / sum p + 2^-8 |O| <= (2^-10 + 2 E) sum p |v| / sum p + 2^-8 |O|,
and |dLSE| <= E + 2^-18 + 2^-20 (1 + |LSE|).
"""
import math

import pytest
import torch

from backward_adapter_gb300 import cache as kv
from backward_adapter_gb300 import fa_train as ft

# B, Hq, Hkv, S: one block a head, few warps with runs of many tiles; one block a head, wide; slices; slices of wide blocks;
# 12 query rows a key/value head
PATHS = {"runs_of_36_tiles": (1025, 2, 1, 4608), "wide_blocks": (2, 8, 2, 1000), "slices": (1, 8, 2, 4608),
         "wide_slices": (38, 16, 8, 1300), "group_of_12": (2, 24, 2, 4608)}
VALUES = ["15.5", "16.5", "1000", "steps", "tiny"]


def definition(q, planes, lens, scale):
    """(O, sum p |v| / sum p, LSE, E) in float64 of one token a sequence."""
    def values(x, d):
        if x.dtype == torch.uint8:
            b = x.unflatten(-1, (-1, 16))
            n = torch.cat([b & 15, b >> 4], -1).double() - 8
        else:
            n = x.unflatten(-1, (-1, 32)).double()
        return (n * d.double()[..., None]).flatten(-2)
    B, Hq, _, D = q.shape
    Hkv, S = planes[0].shape[1:3]
    G = Hq // Hkv
    out = []
    for b in range(B):
        n = int(lens[b])
        k, v = (values(planes[i][b, :, :n], planes[i + 1][b, :, :n]) for i in (0, 2))
        x = q[b, :, 0].double().unflatten(0, (Hkv, G))
        s = scale * x @ k.transpose(-1, -2)
        p = s.softmax(-1)
        W = 8.0 if planes[0].dtype == torch.uint8 else 127.0
        Q = x.abs().unflatten(-1, (-1, 32)).sum(-1)
        E = 2.0 ** -19 * scale * W * (Q @ planes[1][b, :, :n].double().abs().transpose(-1, -2)).amax(-1)
        out.append([y.flatten(0, 1) for y in (p @ v, p @ v.abs(), s.logsumexp(-1), E)])
    return [torch.stack(x) for x in zip(*out)]


def inputs(path, values, fmt, D, gap, seed):
    B, Hq, Hkv, S = PATHS[path]
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = 0.25 * torch.randn((B, Hq, 1, D), generator=g, device="cuda")
    q[..., :32] += 1
    k = 0.5 * torch.randn((B, Hkv, S, D), generator=g, device="cuda")
    k[:, :, 0, :32] = gap * math.sqrt(D) / 32   # the first key's score, above the others' by about gap
    v = 0.5 + 0.25 * torch.randn((B, Hkv, S, D), generator=g, device="cuda")
    if values == "steps":   # scales 1.5 and 2.5 in turn
        v *= torch.tensor([1.5, 2.5], device="cuda").repeat((S + 1) // 2)[:S, None] * (8 if fmt == "q4_0" else 127)
        v[:, :, 0] = 0
    elif values == "tiny":
        v *= 2.0 ** -13
        v[:, :, 0] = 0
    else:
        v[:, :, 5, 40] = float(values)
        v[:, :, 0] *= 0.008
    planes = kv.new_cache(B, Hkv, S, D, fmt)
    kv.cache_write(k, v, *planes, 0)
    lens = torch.full((B,), S, device="cuda")
    lens[B // 2:] -= 33
    return q.to(torch.bfloat16), planes, lens


@pytest.mark.gpu
@pytest.mark.parametrize("values", VALUES)
@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("path", PATHS)
def test_weights_and_scales_far_apart(path, D, fmt, values):
    scale = 1 / math.sqrt(D)
    for gap in (0.0, 10.0, 12.0, 14.0):
        q, planes, lens = inputs(path, values, fmt, D, gap, 7)
        o, lse = kv.decode(q, *planes, lens)
        torch.cuda.synchronize()
        assert ft.device_status() == 0
        want, size, want_lse, E = definition(q, planes, lens, scale)
        err = (o[:, :, 0].double() - want).abs()
        bound = (2.0 ** -10 + 2 * E[..., None]) * size + 2.0 ** -8 * want.abs()
        assert bool((err <= bound).all()), (gap, float((err / bound).max()), float((err / size).max()))
        assert bool(((lse[:, :, 0].double() - want_lse).abs() <= E + 2.0 ** -18 + 2.0 ** -20 * (1 + want_lse.abs())).all())


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("D", [64, 128])
def test_blocks_of_different_scales_and_keys_without_values(D, fmt):
    """The first block's values 2^6 times the others', every third key without values, all keys without values, and a cache
    of zeros."""
    q, planes, lens = inputs("slices", "15.5", fmt, D, 8.0, 9)
    planes[3][..., 0] *= 64
    planes[3][:, :, ::3] = 0
    for n in range(3):
        o, lse = kv.decode(q, *planes, lens)
        torch.cuda.synchronize()
        want, size, want_lse, E = definition(q, planes, lens, 1 / math.sqrt(D))
        err = (o[:, :, 0].double() - want).abs()
        assert bool((err <= (2.0 ** -10 + 2 * E[..., None]) * size + 2.0 ** -8 * want.abs()).all())
        assert bool(((lse[:, :, 0].double() - want_lse).abs() <= E + 2.0 ** -18 + 2.0 ** -20 * (1 + want_lse.abs())).all())
        planes[3].zero_()
        if n == 1:
            planes = kv.new_cache(*planes[0].shape[:3], D, fmt)


# B, Hq, Hkv, S, Sq, lengths, window, range of log2 of V's scales
SCALES = {
    "whole_range": (3, 8, 2, 1500, 1, [1500, 700, 33], 0, (-24, 16)),
    "whole_range_draft_in_a_window": (2, 8, 2, 900, 3, [900, 2], 100, (-24, 16)),
    "subnormal": (2, 4, 4, 2100, 1, [2100, 64], 0, (-24, -14)),
    "large": (1, 16, 1, 600, 2, [600], 0, (0, 16)),
    "many_heads": (50, 16, 8, 800, 1, None, 0, (-24, 16)),
}


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name", SCALES)
def test_scales_anywhere_in_fp16(name, D, fmt):
    """V's scales of any sign and size, a third of the keys without values, scores some tens of nats apart. Here products far
    below the largest one occur too: T = max p max_b |d_b| of a query row (a key without values counts with 2^-32) is at least the
    largest product of each of the row's runs, and what is below 2^-24 of that is off by at most 2^-35 of it, so n keys
    add n W 2^-35 T / sum p to the module's bound."""
    B, Hq, Hkv, S, Sq, lens, window, (lo, hi) = SCALES[name]
    g = torch.Generator(device="cuda").manual_seed(D)
    r = lambda t: torch.rand(t.shape, generator=g, device="cuda")  # noqa: E731
    planes = kv.new_cache(B, Hkv, S, D, fmt)
    W = 8.0 if fmt == "q4_0" else 127.0
    for i in (0, 2):
        planes[i].random_(*((0, 256) if fmt == "q4_0" else (-127, 128)), generator=g)
    planes[1].copy_((2 * r(planes[1]) - 1) * 2 / W)
    planes[3].copy_(torch.exp2(lo + (hi - lo) * r(planes[3])).clamp(max=65504) * torch.where(r(planes[3]) < 0.5, -1.0, 1.0))
    planes[3].masked_fill_(r(planes[3][..., :1]) < 1 / 3, 0)
    q = torch.randn((B, Hq, Sq, D), generator=g, device="cuda").to(torch.bfloat16)
    n = torch.full((B,), S, device="cuda") if lens is None else torch.tensor(lens, device="cuda")
    o, lse = kv.decode(q, *planes, n, window=window)
    torch.cuda.synchronize()
    scale, G = 1 / math.sqrt(D), Hq // Hkv

    def values(x, d):
        if x.dtype == torch.uint8:
            b = x.unflatten(-1, (-1, 16))
            x = torch.cat([b & 15, b >> 4], -1).double() - 8
        else:
            x = x.unflatten(-1, (-1, 32)).double()
        return (x * d.double()[..., None]).flatten(-2)
    k, v = (values(planes[i], planes[i + 1]).repeat_interleave(G, 1) for i in (0, 2))
    at, j = n[:, None] - Sq + torch.arange(Sq, device="cuda"), torch.arange(S, device="cuda")
    seen = j <= at[..., None]
    if window > 0:
        seen &= at[..., None] - j <= window
    seen = seen[:, None]
    s = (scale * q.double() @ k.transpose(-1, -2)).masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=-1e300)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    one = torch.where(total > 0, total, torch.ones_like(total))
    want, size = p @ v / one, p @ v.abs() / one
    d = planes[3].double().abs().amax(-1).repeat_interleave(G, 1)[:, :, None]
    T = (p * torch.where(d == 0, 2.0 ** -32, d)).amax(-1, keepdim=True) / one
    Q = q.double().abs().unflatten(-1, (-1, 32)).sum(-1)
    E = 2.0 ** -19 * scale * W * (Q @ planes[1].double().abs().repeat_interleave(G, 1).transpose(-1, -2))
    E = E.masked_fill(~seen, 0).amax(-1, keepdim=True)
    bound = (2.0 ** -10 + 2 * E) * size + seen.sum(-1, keepdim=True) * W * 2.0 ** -35 * T + 2.0 ** -8 * want.abs()
    err = (o.double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    want_lse = torch.where(total > 0, top + torch.log(one), torch.zeros_like(one))[..., 0]
    assert bool(((lse.double() - want_lse).abs() <= E[..., 0] + 2.0 ** -18 + 2.0 ** -20 * (1 + want_lse.abs())).all())
