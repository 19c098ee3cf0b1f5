"""Norm and rotation of query and key heads (fa_qk_norm_rope) and its backward against the fp64 oracle.

Tolerances, u = 2^-24 (half a step of float32), for a feature whose rotated pair has magnitude M (the rotation keeps
it): the mean of squares is off by 13 u (8 products and 4 + 1 additions on a lane's path), 1/sqrt by half of that and
4 u of its own, the weight's products by 2 u; the angle is the exact one rounded once (at most half a turn: pi u), sine
and cosine are within 4 u, the factor and the two products of the rotation 3 u: below 32 u M in all. The backward has a
second sum of the same depth and two more products: below 64 u of its terms' magnitudes. A result in bfloat16 adds half a
step, 2^-8 of its value. A weight's gradient is a sum over n rows: n + 64 roundings of the sum of magnitudes at most.
"""
import ctypes

import numpy as np
import pytest
import torch

from backward_adapter_gb300 import build as fbuild
from backward_adapter_gb300 import fa_train as ft
from backward_adapter_gb300 import rope
from oracle import rope as ref

U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}


def pair_magnitude(y, half, interleaved):
    """Per feature: the magnitude of its rotated pair; of itself where it is not rotated."""
    m = np.abs(y).astype(np.float64)
    idx = np.arange(half)
    a, b = (2 * idx, 2 * idx + 1) if interleaved else (idx, idx + half)
    n = np.hypot(y[..., a], y[..., b])
    m[..., a], m[..., b] = n, n
    return m


def to_np(t):
    return t.detach().double().cpu().numpy()


def case(B, S, Hq, Hkv, D, rot, dtype=torch.bfloat16, layout="bhsd", interleaved=False, norm="same", pos="rows", far=0,
         factor=1.0, strided=False, seed=0):
    return dict(B=B, S=S, Hq=Hq, Hkv=Hkv, D=D, rot=rot, dtype=dtype, layout=layout, interleaved=interleaved, norm=norm,
                pos=pos, far=far, factor=factor, strided=strided, seed=seed)


CASES = {
    "one_token": case(1, 1, 1, 1, 128, 128),
    "odd_tokens_d64": case(3, 7, 6, 2, 64, 64, seed=1),
    "part_of_the_head": case(2, 19, 4, 4, 128, 40, layout="bshd", seed=2),
    "interleaved_f32": case(2, 33, 5, 1, 64, 24, dtype=torch.float32, interleaved=True, factor=1.37, seed=3),
    "interleaved_bf16": case(1, 130, 8, 2, 128, 128, interleaved=True, layout="bshd", strided=True, seed=4),
    "fused_projection_view": case(2, 17, 8, 2, 128, 128, layout="bshd", strided=True, norm="f32", seed=5),
    "rotation_alone": case(2, 21, 4, 2, 128, 64, norm=None, seed=6),
    "norm_alone": case(2, 21, 4, 2, 64, 0, seed=7),
    "far_positions": case(2, 5, 4, 2, 128, 128, dtype=torch.float32, far=(1 << 31) - 9, seed=8),
    "negative_positions": case(1, 9, 2, 2, 64, 64, dtype=torch.float32, far=-100000, seed=9),
    "shared_positions": case(4, 6, 2, 1, 64, 64, pos="shared", seed=10),
    "offset": case(2, 6, 2, 1, 64, 64, pos="offset", far=67072, seed=11),
    "many_heads": case(1, 3, 70, 35, 64, 32, seed=12),
    "many_tokens": case(2, 1500, 20, 4, 128, 128, layout="bshd", seed=13),
    "f32_weights_f32": case(1, 40, 3, 3, 128, 96, dtype=torch.float32, strided=True, seed=14),
}


def inputs(c, device="cuda"):
    g = torch.Generator().manual_seed(c["seed"])
    B, S, Hq, Hkv, D = c["B"], c["S"], c["Hq"], c["Hkv"], c["D"]

    def rows(H, std=1.0):
        shape = (B, H, S, D) if c["layout"] == "bhsd" else (B, S, H, D)
        return (torch.randn(shape, generator=g) * std).to(c["dtype"])

    t = {"q": rows(Hq), "k": rows(Hkv), "dq": rows(Hq, 0.1), "dk": rows(Hkv, 0.1)}
    if B * S > 2:   # a row of zeros, one of large and one of small values
        t["q"][0].flatten(0, 1)[0] = 0
        t["q"][0].flatten(0, 1)[-1] *= 1e4
        t["k"][-1].flatten(0, 1)[-1] *= 1e-4
    wd = {"same": c["dtype"], "f32": torch.float32, None: None}[c["norm"]]
    t["qw"] = (1 + 0.3 * torch.randn(D, generator=g)).to(wd) if wd else None
    t["kw"] = (1 + 0.3 * torch.randn(D, generator=g)).to(wd) if wd else None
    t["inv_freq"] = rope.rope_inv_freq(c["rot"], 10000.0)[0] if c["rot"] else None
    if c["pos"] == "rows":
        t["pos"] = c["far"] + torch.arange(S) + 3 * torch.arange(B)[:, None]
    elif c["pos"] == "shared":
        t["pos"] = c["far"] + torch.arange(S).flip(0)
    else:
        t["pos"] = None
    t = {n: None if x is None else x.to(device) for n, x in t.items()}
    if c["strided"]:   # queries, keys and something else of a token side by side
        H = Hq + 2 * Hkv
        dim = 1 if c["layout"] == "bhsd" else 2
        for names in (("q", "k"), ("dq", "dk")):
            shape = (B, H, S, D) if dim == 1 else (B, S, H, D)
            whole = torch.full(shape, 7.0, dtype=c["dtype"], device=device)
            q, k = whole.narrow(dim, 0, Hq), whole.narrow(dim, Hq, Hkv)
            q.copy_(t[names[0]])
            k.copy_(t[names[1]])
            t[names[0]], t[names[1]] = q, k
    return t


def call_kw(c, t):
    return dict(positions=t["pos"], q_weight=t["qw"], k_weight=t["kw"], eps=1e-5, interleaved=c["interleaved"],
                factor=c["factor"], offset=c["far"] if c["pos"] == "offset" else 0, layout=c["layout"])


def ref_kw(c, t, which):
    pos = t["pos"]
    if pos is None:
        pos = c["far"] + torch.arange(c["S"])
    pos = pos.cpu().expand(c["B"], c["S"]).numpy()
    w = t[which + "w"]
    return dict(positions=pos, inv_freq=np.zeros(0) if t["inv_freq"] is None else to_np(t["inv_freq"]),
                weight=None if w is None else to_np(w), eps=float(np.float32(1e-5)), interleaved=c["interleaved"],
                factor=float(np.float32(c["factor"])))


def bhsd(x, c):
    return x if c["layout"] == "bhsd" else x.transpose(0, 2, 1, 3)


# ---- CPU ---------------------------------------------------------------------------------------------


def test_oracle_rotation_is_the_textbook_one():
    x = np.random.default_rng(0).standard_normal((1, 1, 3, 8))
    y = ref.forward(x, [[0, 5, 11]], [1.0, 0.1], interleaved=True, factor=2.0)
    np.testing.assert_allclose(y[0, 0, 0, :4], 2 * x[0, 0, 0, :4])
    z = (x[0, 0, :, 0] + 1j * x[0, 0, :, 1]) * np.exp(1j * np.array([0, 5, 11])) * 2
    np.testing.assert_allclose(y[0, 0, :, 0] + 1j * y[0, 0, :, 1], z)
    np.testing.assert_array_equal(y[..., 4:], x[..., 4:])
    h = ref.forward(x, [[0, 5, 11]], [1.0, 0.1])
    z = (x[0, 0, :, 1] + 1j * x[0, 0, :, 3]) * np.exp(0.1j * np.array([0, 5, 11]))
    np.testing.assert_allclose(h[0, 0, :, 1] + 1j * h[0, 0, :, 3], z)


def test_oracle_backward_against_differences():
    rng = np.random.default_rng(1)
    x, dy, w = rng.standard_normal((2, 2, 3, 16)), rng.standard_normal((2, 2, 3, 16)), rng.standard_normal(16)
    kw = dict(positions=[[3, 9, 4], [0, 1, 7]], inv_freq=[1.0, 0.3, 0.01, 0.5], eps=1e-3, factor=1.2)
    for weight in (w, None):
        dx, dw = ref.backward(dy, x, weight=weight, **kw)
        loss = lambda x_, w_: (ref.forward(x_, weight=w_, **kw) * dy).sum()  # noqa: E731
        e = 1e-6
        for at in ((0, 1, 2, 3), (1, 0, 0, 15), (1, 1, 1, 0)):
            d = np.zeros_like(x)
            d[at] = e
            assert abs((loss(x + d, weight) - loss(x - d, weight)) / (2 * e) - dx[at]) < 1e-7
        if weight is not None:
            for j in (0, 5, 15):
                d = np.zeros(16)
                d[j] = e
                assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * e) - dw[j]) < 1e-7


def test_scaled_frequencies():
    f, factor = rope.rope_inv_freq(64, 10000.0)
    np.testing.assert_allclose(f.numpy(), 10000.0 ** (-np.arange(32) / 32.0), rtol=2.0 ** -24)
    assert factor == 1.0
    lin, factor = rope.rope_inv_freq(64, 10000.0, scaling="linear", scale=4.0)
    np.testing.assert_allclose(lin.numpy(), f.numpy() / 4, rtol=2.0 ** -23)
    ntk, factor = rope.rope_inv_freq(64, 10000.0, scaling="ntk", scale=4.0)
    assert ntk[0] == 1.0 and abs(float(ntk[-1] / f[-1]) - 0.25) < 2.0 ** -20 and factor == 1.0
    yarn, factor = rope.rope_inv_freq(64, 10000.0, scaling="yarn", scale=4.0, original_length=4096)
    assert yarn[0] == f[0] and abs(float(yarn[-1] / f[-1]) - 0.25) < 2.0 ** -20
    assert np.all(np.diff(yarn.numpy()) < 0) and abs(factor - (0.1 * np.log(4.0) + 1)) < 1e-12
    for bad in (dict(rotary_dim=12), dict(rotary_dim=0), dict(rotary_dim=64, scaling="twice"),
                dict(rotary_dim=64, scale=0.5)):
        with pytest.raises(ValueError):
            rope.rope_inv_freq(**bad)


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return ft.load_library()


R = ctypes.byref


def params(**kw):
    p = ft.FaRopeParams(2, 5, 4, 2, 64, ft.FA_BF16, ft.FA_BF16, 64, 0, 1, 1e-6, 1.0, 0, 5, 0)
    for n, v in kw.items():
        setattr(p, n, v)
    return p


BAD = [("B0", dict(B=0), 1), ("S_negative", dict(S=-1), 1), ("no_heads", dict(Hq=0, Hkv=0), 1), ("D96", dict(D=96), 2),
       ("dtype", dict(dtype=5), 1), ("w_dtype", dict(dtype=0, w_dtype=1), 1), ("rot_12", dict(rot=12), 1),
       ("rot_72", dict(rot=72), 1), ("interleaved", dict(interleaved=2), 1), ("norm", dict(norm=3), 1),
       ("eps_0", dict(eps=0.0), 1), ("eps_nan", dict(eps=float("nan")), 1), ("factor", dict(factor=float("inf")), 1),
       ("pos_stride", dict(pos_stride_b=-1), 1), ("reserved", dict(reserved=1), 1), ("offset", dict(offset=(1 << 62) + 1), 1),
       ("too_large", dict(B=65535, S=1 << 24, Hq=65535), 1)]


def views(base, p, n):
    d = p.D
    return [ft.FaView(base * (i + 1), (p.Hq if i % 2 == 0 else p.Hkv) * p.S * d, d, p.S * d) for i in range(n)]


@pytest.mark.parametrize("name,kw,code", BAD, ids=[b[0] for b in BAD])
def test_bad_parameters_are_refused_before_launch(lib, name, kw, code):
    p, good = params(**kw), params()
    v = views(1 << 32, good, 6)
    f = 1 << 40
    assert lib.fa_qk_norm_rope(R(p), R(v[0]), R(v[1]), f, f + 4096, f + 8192, f + 12288, R(v[2]), R(v[3]), None) == code
    assert lib.fa_last_error()
    assert lib.fa_qk_norm_rope_bwd_workspace_size(R(p)) == 0
    assert lib.fa_qk_norm_rope_bwd(R(p), *map(R, v[:4]), f, f + 4096, f + 8192, f + 12288, R(v[4]), R(v[5]), f + (1 << 20),
                                   f + (2 << 20), f + (3 << 20), 1 << 30, None) == code


def test_bad_views_pointers_and_workspaces_are_refused(lib):
    p = params()
    f = 1 << 40
    small = (f, f + 4096, f + 8192, f + 12288)

    def fwd(change=None, at=0, small=small):
        v = views(1 << 32, p, 4)
        if change is not None:
            for n, x in change.items():
                setattr(v[at], n, x)
        st = lib.fa_qk_norm_rope(R(p), R(v[0]), R(v[1]), *small, R(v[2]), R(v[3]), None)
        return st, lib.fa_last_error().decode()

    for change, at, word in ((dict(ptr=(1 << 32) + 8), 0, "aligned"), (dict(ptr=0), 1, "NULL"),
                             (dict(stride_s=-64), 0, "stride"), (dict(stride_h=65), 1, "16 bytes"),
                             (dict(stride_s=32), 2, "overlap"), (dict(stride_h=0), 3, "overlap"),
                             (dict(ptr=(1 << 32) + 64), 2, "overlaps"), (dict(stride_b=1 << 41), 0, "stride")):
        st, msg = fwd(change, at)
        assert st == ft.FA_ERR_INVALID_ARG and word in msg, (change, msg)
    for i, bad in ((0, None), (2, None), (0, f + 8), (2, f + 2), (3, f + 4), (3, 3 << 32)):
        s = list(small)
        s[i] = bad
        st, msg = fwd(small=s)
        assert st == ft.FA_ERR_INVALID_ARG, (i, bad, msg)
    v = views(1 << 32, p, 6)
    need = lib.fa_qk_norm_rope_bwd_workspace_size(R(p))
    assert need > 0
    out = (R(v[4]), R(v[5]), f + (1 << 20), f + (2 << 20))
    assert lib.fa_qk_norm_rope_bwd(R(p), *map(R, v[:4]), *small, *out, f + (3 << 20), need - 1, None) == ft.FA_ERR_WORKSPACE
    assert lib.fa_qk_norm_rope_bwd(R(p), *map(R, v[:4]), *small, *out, None, need, None) == ft.FA_ERR_WORKSPACE
    assert lib.fa_qk_norm_rope_bwd(R(p), *map(R, v[:4]), *small, *out, 1 << 32, need, None) == ft.FA_ERR_INVALID_ARG
    assert lib.fa_qk_norm_rope(R(params(S=0)), *map(R, v[:2]), *small, R(v[2]), R(v[3]), None) == ft.FA_OK   # nothing to do


def test_struct_layout_matches_header(tmp_path):
    import os
    import shutil
    import subprocess
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    names = {"fa_rope_params": ft.FaRopeParams, "fa_view": ft.FaView, "fa_cache": ft.FaCache,
             "fa_decode_params": ft.FaDecodeParams, "fa_kv_q4": ft.FaKvQ4}
    lines, want = [], []
    for n, t in names.items():
        lines.append(f'printf("%zu ", sizeof({n}));')
        want.append(ctypes.sizeof(t))
        for f, _ in t._fields_:
            lines.append(f'printf("%zu ", offsetof({n}, {f}));')
            want.append(getattr(t, f).offset)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "fa_train.h"\nint main(void){' + "".join(lines) +
                   "return 0;}\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([gcc, "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "layout")], check=True)
    got = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == want


def test_binding_refuses_what_does_not_fit():
    c = case(2, 5, 4, 2, 64, 64)
    t = inputs(c, "cpu")
    kw = call_kw(c, t)
    fbuild.build()
    go = lambda **x: rope.qk_norm_rope(**{**dict(q=t["q"], k=t["k"], inv_freq=t["inv_freq"]), **kw, **x})  # noqa: E731
    with pytest.raises(ValueError, match="CUDA tensor"):
        go()
    for x, exc, word in ((dict(k=t["k"][:, :, :4]), ValueError, "k has shape"),
                         (dict(k=t["k"].float()), TypeError, "k has dtype"),
                         (dict(q=t["q"][0]), ValueError, "4-D"), (dict(layout="sbhd"), ValueError, "layout"),
                         (dict(q_weight=None), ValueError, "both"), (dict(q_weight=t["qw"][:32]), ValueError, "q_weight"),
                         (dict(q_weight=t["qw"].half(), k_weight=t["kw"].half()), TypeError, "weights"),
                         (dict(inv_freq=t["inv_freq"].double()), TypeError, "inv_freq"),
                         (dict(positions=t["pos"].int()), TypeError, "positions"),
                         (dict(positions=t["pos"][:, :4]), ValueError, "positions"),
                         (dict(q=t["q"].half(), k=t["k"].half()), TypeError, "unsupported dtype"),
                         (dict(q_out=t["q"][:1]), ValueError, "q_out")):
        with pytest.raises(exc, match=word):
            go(**x)
    with pytest.raises(ValueError, match="dq_out has shape"):
        rope.qk_norm_rope_bwd(t["dq"][:1], t["dk"], t["q"], t["k"], t["inv_freq"], **kw)


# ---- GPU ---------------------------------------------------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_forward_matches_oracle(name):
    c = CASES[name]
    t = inputs(c)
    got = rope.qk_norm_rope(t["q"], t["k"], t["inv_freq"], **call_kw(c, t))
    torch.cuda.synchronize()
    for which, y in zip("qk", got):
        assert y.shape == t[which].shape and y.dtype == c["dtype"] and y.is_contiguous()
        want = ref.forward(bhsd(to_np(t[which]), c), **ref_kw(c, t, which))
        err = np.abs(bhsd(to_np(y), c) - want)
        m = pair_magnitude(want, c["rot"] // 2, c["interleaved"])
        assert np.all(err <= HALF_STEP[c["dtype"]] * np.abs(want) + 32 * U * m + 1e-37), err.max()


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_backward_matches_oracle(name):
    c = CASES[name]
    t = inputs(c)
    got = rope.qk_norm_rope_bwd(t["dq"], t["dk"], t["q"], t["k"], t["inv_freq"], **call_kw(c, t))
    torch.cuda.synchronize()
    for i, which in enumerate("qk"):
        x, dy = bhsd(to_np(t[which]), c), bhsd(to_np(t["d" + which]), c)
        kw = ref_kw(c, t, which)
        want, dw = ref.backward(dy, x, **kw)
        g = ref.backward(dy, x, **{**kw, "weight": None})[0]
        m = pair_magnitude(g, c["rot"] // 2, c["interleaved"])
        if kw["weight"] is not None:
            r = ((x ** 2).mean(-1, keepdims=True) + kw["eps"]) ** -0.5
            t_m = m * np.abs(kw["weight"])
            m_dw = (m * np.abs(x) * r).sum((0, 1, 2))
            m = r * (t_m + np.abs(x) * r ** 2 * (t_m * np.abs(x)).mean(-1, keepdims=True))
            rows = x.shape[0] * x.shape[1] * x.shape[2]
            assert got[2 + i].dtype == torch.float32
            assert np.all(np.abs(to_np(got[2 + i]) - dw) <= (rows + 64) * U * m_dw)
        else:
            assert got[2 + i] is None
        err = np.abs(bhsd(to_np(got[i]), c) - want)
        assert np.all(err <= HALF_STEP[c["dtype"]] * np.abs(want) + 64 * U * m + 1e-37), err.max()


@pytest.mark.gpu
def test_weight_gradients_are_the_same_from_run_to_run_and_strided_outputs_are_left_alone():
    c = CASES["many_tokens"]
    t = inputs(c)
    kw = call_kw(c, t)
    first = rope.qk_norm_rope_bwd(t["dq"], t["dk"], t["q"], t["k"], t["inv_freq"], **kw)
    whole = torch.full((c["B"], c["S"], c["Hq"] + c["Hkv"] + 3, c["D"]), 9.0, dtype=c["dtype"], device="cuda")
    dq, dk = whole[:, :, 1:1 + c["Hq"]], whole[:, :, 2 + c["Hq"]:2 + c["Hq"] + c["Hkv"]]
    # side by side in one buffer they may be written, but not with a head that both have
    with pytest.raises(ft.FaError, match="overlap"):
        both = whole[:, :, c["Hq"]:c["Hq"] + c["Hkv"]]
        rope.qk_norm_rope_bwd(t["dq"], t["dk"], t["q"], t["k"], t["inv_freq"], dq=dq, dk=both, **kw)
    rope.qk_norm_rope_bwd(t["dq"], t["dk"], t["q"], t["k"], t["inv_freq"], dq=dq, dk=dk, **kw)
    torch.cuda.synchronize()
    assert torch.equal(first[0], dq) and torch.equal(first[1], dk)
    whole.fill_(9.0)
    again = rope.qk_norm_rope_bwd(t["dq"], t["dk"], t["q"], t["k"], t["inv_freq"], dq=dq, **kw)
    torch.cuda.synchronize()
    assert torch.equal(first[0], dq) and all(torch.equal(a, b) for a, b in zip(first[1:], again[1:]))
    rest = torch.ones(whole.shape[2], dtype=torch.bool, device="cuda")
    rest[1:1 + c["Hq"]] = False
    assert bool((whole[:, :, rest] == 9.0).all())


@pytest.mark.gpu
def test_frequencies_that_are_no_numbers_show():
    q = torch.randn((1, 2, 3, 64), device="cuda")
    f = rope.rope_inv_freq(64, device="cuda")[0]
    f[3], f[17] = float("nan"), float("inf")
    y = rope.qk_norm_rope(q, q[:, :1], f)[0]
    bad = torch.zeros(64, dtype=torch.bool, device="cuda")
    bad[[3, 17, 35, 49]] = True
    assert bool(y[..., bad].isnan().all()) and bool(y[..., ~bad].isfinite().all())


@pytest.mark.gpu
def test_no_tokens_and_broadcast_inputs():
    e = torch.empty((2, 4, 0, 64), dtype=torch.bfloat16, device="cuda")
    f = rope.rope_inv_freq(64, device="cuda")[0]
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    q, k = rope.qk_norm_rope(e, e[:, :2], f, q_weight=w, k_weight=w)
    assert q.shape == e.shape and k.shape == (2, 2, 0, 64)
    got = rope.qk_norm_rope_bwd(e, e[:, :2], e, e[:, :2], f, q_weight=w, k_weight=w)
    assert torch.equal(got[2], torch.zeros(64, device="cuda")) and torch.equal(got[3], got[2])
    # one key head seen as four (stride 0): read like any other
    q = torch.randn((1, 4, 6, 64), device="cuda")
    k1 = torch.randn((1, 1, 6, 64), device="cuda")
    a = rope.qk_norm_rope(q, k1.expand(1, 4, 6, 64), f)[1]
    b = rope.qk_norm_rope(q, k1.expand(1, 4, 6, 64).contiguous(), f)[1]
    assert torch.equal(a, b)


def side_views(p, base, shift, token):
    """Views of p.Hq and p.Hkv heads in tokens of `token` elements, the second `shift` elements after the first."""
    return [ft.FaView(base + 2 * at, p.S * token, token, p.D) for at in (0, shift)]


def test_outputs_side_by_side_must_not_share_elements(lib):
    """The parts of a fused projection's gradient may not reach into one another, whichever comes first."""
    p = params()   # 4 and 2 heads of 64, 5 tokens, 2 sequences
    f = 1 << 40
    small, x = (f, f + 4096, f + 8192, f + 12288), views(1 << 32, p, 4)
    sums = (f + (1 << 20), f + (2 << 20), f + (3 << 20), 1 << 30)
    # one head of q in k; k's last head in the next token's q; k from the next token on, likewise; other strides
    for shift, token in ((192, 512), (320, 384), (512 + 192, 512), (384 * 5 + 128, 384)):
        a, b = side_views(p, 1 << 36, shift, token)
        assert lib.fa_qk_norm_rope(R(p), R(x[0]), R(x[1]), *small, R(a), R(b), None) == ft.FA_ERR_INVALID_ARG
        assert b"overlap" in lib.fa_last_error()
        assert lib.fa_qk_norm_rope_bwd(R(p), *map(R, x), *small, R(a), R(b), *sums, None) == ft.FA_ERR_INVALID_ARG
        assert b"overlap" in lib.fa_last_error()
    a, b = side_views(p, 1 << 36, 256, 512)
    b.stride_s = 576
    assert lib.fa_qk_norm_rope(R(p), R(x[0]), R(x[1]), *small, R(a), R(b), None) == ft.FA_ERR_INVALID_ARG
    a, b = side_views(p, 1 << 36, 256, 512)
    a.stride_b = b.stride_b = 5 * 512 + 64   # the second sequence's tokens are elsewhere in the first's
    assert lib.fa_qk_norm_rope(R(p), R(x[0]), R(x[1]), *small, R(a), R(b), None) == ft.FA_ERR_INVALID_ARG
    assert b"overlap" in lib.fa_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
@pytest.mark.parametrize("B,S", [(1, 1), (3, 1), (1, 9), (2, 300)])
def test_outputs_side_by_side_in_one_tensor(B, S, layout):
    """Q and K, and their gradients, written into the parts of a fused projection's tensor; the rest of it stays."""
    c = case(B, S, 4, 2, 128, 64, layout="bshd", strided=True, seed=20)
    t = inputs(c)
    kw = call_kw(c, t)
    turn = (lambda x: x) if layout == "bshd" else (lambda x: x.transpose(1, 2))
    kw["layout"] = layout
    q, k, dq, dk = (turn(t[n]) for n in ("q", "k", "dq", "dk"))
    want = rope.qk_norm_rope(q, k, t["inv_freq"], **kw)
    want_bwd = rope.qk_norm_rope_bwd(dq, dk, q, k, t["inv_freq"], **kw)
    for first in ("q", "k"):
        parts = (slice(0, 4), slice(4, 6)) if first == "q" else (slice(2, 6), slice(0, 2))
        whole, grad = (torch.full((B, S, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        a, b = (turn(whole[:, :, x]) for x in parts)
        rope.qk_norm_rope(q, k, t["inv_freq"], q_out=a, k_out=b, **kw)
        assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and bool((whole[:, :, 6:] == 3).all())
        a, b = (turn(grad[:, :, x]) for x in parts)
        got = rope.qk_norm_rope_bwd(dq, dk, q, k, t["inv_freq"], dq=a, dk=b, **kw)
        assert got[0] is a and all(torch.equal(x, y) for x, y in zip(got, want_bwd)) and bool((grad[:, :, 6:] == 3).all())


def test_offsets_that_a_64_bit_number_does_not_hold_are_refused(lib):
    t = inputs(case(2, 5, 4, 2, 64, 64), "cpu")
    for n in (1 << 63, 1 << 64, -(1 << 64), (1 << 62) + 1):
        v = rope._params(t["q"], t["k"], t["inv_freq"], None, t["qw"], t["kw"], 1e-6, False, 1.0, n, "bhsd")
        p, good = ft.FaRopeParams(*v[:-1]), params()
        x = views(1 << 32, good, 4)
        f = 1 << 40
        assert lib.fa_qk_norm_rope(R(p), R(x[0]), R(x[1]), f, f + 4096, f + 8192, None, R(x[2]), R(x[3]), None) == 1
        assert b"offset" in lib.fa_last_error()
