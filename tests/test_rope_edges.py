"""Norm and rotation (and the read of a cache) at the edges of their shapes: a side without heads, outputs in parts of one tensor."""
import ctypes

import pytest
import torch

from backward_adapter_gb300 import build as fbuild
from backward_adapter_gb300 import cache as kv
from backward_adapter_gb300 import fa_train as ft
from backward_adapter_gb300 import rope


@pytest.mark.gpu
@pytest.mark.parametrize("S", [0, 5, 3000])
@pytest.mark.parametrize("side", ["q", "k"])
def test_a_side_without_heads_has_a_weight_gradient_of_zero(side, S):
    """The sum over no rows is written like any other, into memory that holds something else."""
    D = 64
    g = torch.Generator(device="cuda").manual_seed(S)
    x, dx = (torch.randn((2, 4, S, D), generator=g, device="cuda") for _ in range(2))
    none = torch.empty((2, 0, S, D), device="cuda")
    f, w = rope.rope_inv_freq(D, device="cuda")[0], torch.rand(D, device="cuda")
    args = (dx, none, x, none) if side == "k" else (none, dx, none, x)
    at, other = (3, 2) if side == "k" else (2, 3)
    got = rope.qk_norm_rope_bwd(*args, f, q_weight=w, k_weight=w, dq_weight=torch.full((D,), 7.0, device="cuda"),
                                dk_weight=torch.full((D,), 7.0, device="cuda"))
    assert torch.equal(got[at], torch.zeros(D, device="cuda"))
    want = rope.qk_norm_rope_bwd(dx, dx, x, x, f, q_weight=w, k_weight=w)
    assert torch.equal(got[0 if side == "k" else 1], want[0])
    # with other heads beside them the same n terms are added in another order: each sum is off by at most (n + 64) 2^-24 of
    # the sum of magnitudes (see test_rope), a term's being that of its rotated pair times |x| r
    n, m = 8 * S, torch.hypot(dx[..., :32].double(), dx[..., 32:].double()).repeat(1, 1, 1, 2)
    size = (m * x.double().abs() * (x.double().square().mean(-1, keepdim=True) + 1e-6).rsqrt()).sum((0, 1, 2))
    assert bool(((got[other].double() - want[other].double()).abs() <= 2 * (n + 64) * 2.0 ** -24 * size).all())


def parts_of(order, B, S, Hq, Hkv, D, dtype, fill):
    """Views [B, S, H, D] of two parts of one tensor, filled with `fill`, and the tensor: the tokens of a sequence one after
    another or of all sequences one after another (as in a tensor [S, B, H, D]), the heads of both in turn, or all three
    kinds of a head side by side."""
    H = Hq + 2 * Hkv
    if order == "tokens":
        whole = torch.full((B, S, H, D), fill, dtype=dtype, device="cuda")
        return whole[:, :, :Hq], whole[:, :, Hq:Hq + Hkv], whole
    if order == "sequences":
        whole = torch.full((S, B, H, D), fill, dtype=dtype, device="cuda")
        x = whole.transpose(0, 1)
        return x[:, :, Hkv:Hkv + Hq], x[:, :, :Hkv], whole
    shape = (S, B) if order == "heads_sequences" else (B, S)
    whole = torch.full((*shape, max(Hq, Hkv), 3, D), fill, dtype=dtype, device="cuda")
    x = whole.transpose(0, 1) if order == "heads_sequences" else whole
    return x[:, :, :Hq, 0], x[:, :, :Hkv, 2], whole


@pytest.mark.gpu
@pytest.mark.parametrize("order", ["tokens", "sequences", "heads", "heads_sequences"])
@pytest.mark.parametrize("B,S,Hq,Hkv", [(1, 1, 4, 4), (3, 1, 4, 2), (1, 9, 2, 2), (2, 70, 4, 1), (2, 5, 1, 4)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_outputs_in_parts_of_a_fused_tensor_in_any_order(order, B, S, Hq, Hkv, dtype):
    D = 64
    g = torch.Generator(device="cuda").manual_seed(S)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    q, k, dq, dk = r(B, S, Hq, D), r(B, S, Hkv, D), r(B, S, Hq, D), r(B, S, Hkv, D)
    f, w = rope.rope_inv_freq(D, device="cuda")[0], torch.rand(D, device="cuda")
    kw = dict(q_weight=w, k_weight=w, layout="bshd")
    for call, names in ((lambda **o: rope.qk_norm_rope(q, k, f, **kw, **o), ("q_out", "k_out")),
                        (lambda **o: rope.qk_norm_rope_bwd(dq, dk, q, k, f, **kw, **o), ("dq", "dk"))):
        want = call()
        a, b, whole = parts_of(order, B, S, Hq, Hkv, D, dtype, 3.0)
        got = call(**dict(zip(names, (a, b))))
        assert got[0] is a and all(torch.equal(x, y) for x, y in zip(got, want))
        a.fill_(3.0)
        b.fill_(3.0)
        assert bool((whole == 3.0).all())   # what is between the parts is as it was


@pytest.mark.gpu
@pytest.mark.parametrize("order", ["tokens", "sequences", "heads"])
def test_cache_read_into_parts_of_one_tensor(order):
    B, H, S, D = 2, 3, 50, 64
    planes = kv.new_cache(B, H, S, D, "q4_0")
    kv.cache_write(torch.randn((B, H, S, D), device="cuda"), torch.randn((B, H, S, D), device="cuda"), *planes, 0)
    want = kv.cache_read(*planes, 4, 40, layout="bshd")
    a, b, whole = parts_of(order, B, 40, H, H, D, torch.bfloat16, 3.0)
    got = kv.cache_read(*planes, 4, 40, layout="bshd", k=a, v=b)
    assert got[0] is a and torch.equal(a, want[0]) and torch.equal(b, want[1])
    a.fill_(3.0)
    b.fill_(3.0)
    assert bool((whole == 3.0).all())
    for x, y in ((a, a), (a, whole.flatten()[D // 2:][:a.numel()].view(a.shape) if order == "tokens" else a[:, :, :])):
        with pytest.raises(ft.FaError, match="overlap"):
            kv.cache_read(*planes, 4, 40, layout="bshd", k=x, v=y)


def test_parts_that_share_elements_are_refused():
    """Heads in turn that reach into one another, or whose tokens do, in either order of tokens and sequences."""
    fbuild.build()
    lib, R, f = ft.load_library(), ctypes.byref, 1 << 40
    p = ft.FaRopeParams(2, 5, 4, 4, 64, ft.FA_BF16, ft.FA_BF16, 64, 0, 1, 1e-6, 1.0, 0, 5, 0)
    x = [ft.FaView((1 << 32) * (i + 1), 20 * 64, 64, 5 * 64) for i in range(2)]

    def go(at, sb, ss, sh, other=None):
        a, b = ft.FaView(1 << 36, sb, ss, sh), ft.FaView((1 << 36) + 2 * at, sb, ss, sh if other is None else other)
        st = lib.fa_qk_norm_rope(R(p), R(x[0]), R(x[1]), f, f + 4096, f + 8192, f + 12288, R(a), R(b), None)
        return st, lib.fa_last_error()
    for bad in ((32, 5 * 768, 768, 192), (144, 5 * 768, 768, 192), (64, 5 * 760, 760, 192), (64, 5 * 768 + 64, 768, 192),
                (64, 5 * 1024, 1024, 192, 256), (192, 512, 1024, 64), (320, 512, 1024, 64), (0, 512, 1024, 64),
                (256, 640, 1344, 64)):
        st, msg = go(*bad)
        assert st == ft.FA_ERR_INVALID_ARG and b"overlap" in msg, bad
