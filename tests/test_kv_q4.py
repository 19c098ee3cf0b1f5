"""The op over a q4_0 K/V cache (fa_train_*_q4): bit for bit the op on the cache's values rounded to bf16, which the other
parity tests hold to the oracle; and against the oracle itself on the values the cache stands for."""
import ctypes

import numpy as np
import pytest
import torch

from backward_adapter_gb300 import build as fbuild
from backward_adapter_gb300 import cache as kv
from backward_adapter_gb300 import fa_train as ft
from oracle import attention as attn
from oracle import kv_cache as ref
from oracle import set_rows as rows_ref


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return ft.load_library()


def test_q4_calls_are_checked(lib):
    p = ft.FaParams(1, 2, 1, 64, 64, 64, ft.FA_F32, 0.125, 0, ft.FA_MASK_NONE, 1, 0, 0, 0, ft.FA_KV_Q4_0)
    f = 1 << 30
    q4 = ft.FaKvQ4(2 * f, 3 * f, 4 * f, 5 * f)
    fwd = lambda: lib.fa_train_fwd_q4(p, f, q4, None, 6 * f, 7 * f, 256 * f, 1 << 24, None)  # noqa: E731
    assert fwd() == ft.FA_ERR_UNSUPPORTED and b"bf16" in lib.fa_last_error()
    p.dtype = ft.FA_BF16
    assert lib.fa_train_fwd_q4(p, f, None, None, 6 * f, 7 * f, None, 0, None) == ft.FA_ERR_INVALID_ARG
    q4.v_d = 0
    assert fwd() == ft.FA_ERR_INVALID_ARG and b"v_d is NULL" in lib.fa_last_error()
    q4.v_d = 5 * f
    p.kv_format = ft.FA_KV_Q8_0
    assert fwd() == ft.FA_ERR_INVALID_ARG and b"_q8" in lib.fa_last_error()
    # a q4_0 format through any other entry point
    p.kv_format = ft.FA_KV_Q4_0
    q8 = ft.FaKvQ8(2 * f, 3 * f, 4 * f, 5 * f)
    assert lib.fa_train_fwd(p, f, 2 * f, 3 * f, None, 6 * f, 7 * f, None, 0, None) == ft.FA_ERR_INVALID_ARG
    assert lib.fa_train_fwd_q8(p, f, ctypes.byref(q8), None, 6 * f, 7 * f, None, 0, None) == ft.FA_ERR_INVALID_ARG
    assert lib.fa_train_bwd(p, f, 2 * f, 3 * f, None, 6 * f, 7 * f, 8 * f, 9 * f, 10 * f, 11 * f, None, 0, None) == \
        ft.FA_ERR_INVALID_ARG
    p.kv_format = ft.FA_KV_DTYPE
    plain = (lib.fa_train_fwd_workspace_size(p), lib.fa_train_bwd_workspace_size(p))
    p.kv_format = ft.FA_KV_Q4_0
    copy = 2 * 64 * 64 * 2
    assert copy <= lib.fa_train_fwd_workspace_size(p) - plain[0] < copy + 512
    assert copy <= lib.fa_train_bwd_workspace_size(p) - plain[1] < copy + 512


def test_binding_checks_the_planes():
    planes = kv.new_cache(2, 2, 70, 64, "q4_0", device="cpu")
    q = torch.zeros(2, 4, 40, 64, dtype=torch.bfloat16)
    lse = torch.zeros(2, 4, 40)
    for layout in ("bhsd", "bshd"):
        x = q if layout == "bhsd" else q.transpose(1, 2).contiguous()
        for call in (lambda: ft.fwd_q4(x, *planes, layout=layout), lambda: ft.bwd_q4(x, *planes, x, lse, x, layout=layout)):
            with pytest.raises(ValueError, match="contiguous CUDA tensor"):
                call()
    with pytest.raises(TypeError, match="uint8"):
        ft.fwd_q4(q, *kv.new_cache(2, 2, 70, 64, "q8_0", device="cpu"))
    with pytest.raises(ValueError, match="v_q has shape"):
        ft.fwd_q4(q, planes[0], planes[1], planes[2][:, :, :60], planes[3])


CASES = {   # B, Hq, Hkv, Sq, Sk, D, causal, window, mask, layout
    "one_row": (1, 1, 1, 1, 1, 64, True, 0, None, "bhsd"),
    "causal_chunk": (1, 4, 2, 100, 333, 128, True, 0, None, "bhsd"),
    "causal_bshd": (2, 4, 1, 70, 190, 64, True, 0, None, "bshd"),
    "windowed_mask": (2, 4, 2, 130, 260, 64, False, 50, "bool", "bhsd"),
    "additive_bshd": (1, 2, 2, 60, 129, 128, False, 0, "add", "bshd"),
    "long_keys": (1, 4, 1, 64, 2100, 128, True, 0, None, "bhsd"),
}


def inputs(name, seed=0):
    B, Hq, Hkv, Sq, Sk, D, causal, window, mask, layout = CASES[name]
    rng = np.random.default_rng(seed + len(name))
    n = {x: rows_ref.to_bf16_bits(rng.standard_normal((B, Hq, Sq, D)).astype(np.float32)) for x in ("q", "do")}
    planes = []
    for _ in range(2):
        planes += list(ref.quantize(rng.standard_normal((B, Hkv, Sk, D)).astype(np.float32), "q4_0"))
    m = None
    if mask == "bool":
        m = (rng.random((B, Sq, Sk)) < 0.6).astype(np.uint8)
        m[:, 3] = 0
    if mask == "add":
        m = np.where(rng.random((1, Sq, Sk)) < 0.7, rng.standard_normal((1, Sq, Sk)), -np.inf).astype(np.float32)
        m[:, 5] = np.finfo(np.float32).min   # a row hidden by the type's lowest value
    off = Sk - Sq if causal else (40 if window else 0)
    return n, planes, m, dict(causal=causal, window=window, q_offset=off), layout


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_is_the_op_on_the_rounded_values(name):
    n, planes, m, kw, layout = inputs(name)
    t = [torch.from_numpy(x).cuda() for x in planes]
    L = (lambda x: x) if layout == "bhsd" else (lambda x: x.transpose(1, 2).contiguous())  # noqa: E731
    q, do = (L(torch.from_numpy(n[x]).to(torch.bfloat16).cuda()) for x in ("q", "do"))
    mask = None if m is None else torch.from_numpy(m).cuda()
    k, v = kv.cache_read(*t, layout=layout)
    kw = dict(kw, layout=layout)
    o, lse = ft.fwd(q, k, v, mask, **kw)
    o4, lse4 = ft.fwd_q4(q, *t, mask, **kw)
    grads = ft.bwd(q, k, v, o, lse, do, mask, deterministic=True, **kw)
    grads4 = ft.bwd_q4(q, *t, o, lse, do, mask, deterministic=True, **kw)
    acc = [torch.randn(x.shape, device="cuda") for x in (k, v)]
    acc4 = [x.clone() for x in acc]
    ft.bwd_accum(q, k, v, o, lse, do, *acc, mask, deterministic=True, **kw)
    dq4 = ft.bwd_q4(q, *t, o, lse, do, mask, deterministic=True, dk_acc=acc4[0], dv_acc=acc4[1], **kw)
    torch.cuda.synchronize()
    assert ft.device_status() == 0
    for a, b in zip((o, lse, *grads, grads[0], *acc), (o4, lse4, *grads4, dq4, *acc4)):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_matches_oracle_on_the_rounded_values(name):
    n, planes, m, kw, layout = inputs(name)
    vals = [rows_ref.to_bf16_bits(ref.values(planes[i], planes[i + 1]).astype(np.float32)) for i in (0, 2)]
    D = vals[0].shape[-1]
    want = attn.backward(n["q"], *vals, n["do"], D ** -0.5, mask=m,
                         mask_kind="none" if m is None else ("bool" if m.dtype == np.uint8 else "add"), **kw)
    t = [torch.from_numpy(x).cuda() for x in planes]
    L = (lambda x: x) if layout == "bhsd" else (lambda x: x.transpose(1, 2).contiguous())  # noqa: E731
    q, do = (L(torch.from_numpy(n[x]).to(torch.bfloat16).cuda()) for x in ("q", "do"))
    mask = None if m is None else torch.from_numpy(m).cuda()
    o, lse = ft.fwd_q4(q, *t, mask, layout=layout, **kw)
    got = dict(zip(("o", "dq", "dk", "dv"), (o, *ft.bwd_q4(q, *t, o, lse, do, mask, layout=layout, **kw))))
    torch.cuda.synchronize()
    for x, g in got.items():   # the bounds of the op's other bf16 parity tests
        e = np.abs(L(g).double().cpu().numpy() - want[x]).max()
        assert e <= 1e-2 * np.abs(want[x]).max() + 1e-3, (x, e)
    assert np.abs(lse.double().cpu().numpy() - want["lse"]).max() <= 1e-3
