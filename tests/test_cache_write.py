"""Writing a quantized K/V cache and reading it back: bit for bit the oracle's blocks, and nothing else touched."""
import ctypes

import numpy as np
import pytest
import torch

from backward_adapter_gb300 import build as fbuild
from backward_adapter_gb300 import cache as kv
from backward_adapter_gb300 import fa_train as ft
from backward_adapter_gb300 import workloads as wl
from oracle import attention as attn_ref
from oracle import kv_cache as ref
from oracle import set_rows as rows_ref


# ---- CPU ---------------------------------------------------------------------------------------------


def test_oracle_blocks_agree_with_the_formats():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 3, 64)).astype(np.float32)
    q, d = ref.quantize(x, "q8_0")
    wq, wd = wl.quantize_q8_0(x)   # the caller's side of the training tests
    np.testing.assert_array_equal(q, wq)
    np.testing.assert_array_equal(d, wd)
    np.testing.assert_array_equal(ref.values(q, d), attn_ref.dequantize_q8_0(q, d))
    q, d = ref.quantize(x, "q4_0")
    v = ref.values(q, d)
    step = np.repeat(np.abs(d.astype(np.float64)), 32, -1)
    # the end of the range opposite to m reaches 7 steps only: one step off there, half elsewhere
    assert np.all(np.abs(v - x) <= step * (1 + 2.0 ** -8)) and np.mean(np.abs(v - x) <= step * (0.5 + 2.0 ** -8)) > 0.9
    b = np.zeros(32, np.float32)
    b[3], b[20] = -4.0, 4.0   # the first of two equal magnitudes gives the sign: -4 = -8 d, d = 0.5
    q, d = ref.quantize(b, "q4_0")
    assert d[0] == 0.5 and q[3] & 15 == 0 and q[4] >> 4 == 15 and q[0] == 0x88


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return ft.load_library()


F = 1 << 34


def R(x):
    return None if x is None else ctypes.byref(x)


def cache(**kw):
    c = ft.FaCache(2, 3, 40, 64, ft.FA_KV_Q4_0, 0, F, 2 * F, 3 * F, 4 * F)
    for n, v in kw.items():
        setattr(c, n, v)
    return c


def view(i, n=5, **kw):
    v = ft.FaView(i * F, 3 * n * 64, 64, n * 64)
    for name, x in kw.items():
        setattr(v, name, x)
    return v


BAD_CACHE = [("B", dict(B=0), 1), ("Hkv", dict(Hkv=70000), 1), ("S", dict(S=0), 1), ("D", dict(D=96), 2),
             ("D_negative", dict(D=-64), 1), ("format", dict(kv_format=ft.FA_KV_F16), 1), ("reserved", dict(reserved=2), 1),
             ("plane", dict(k_d=0), 1), ("aligned", dict(v_q=3 * F + 8), 1),
             ("too_large", dict(B=65535, Hkv=65535, S=1 << 24), 1)]


@pytest.mark.parametrize("name,kw,code", BAD_CACHE, ids=[b[0] for b in BAD_CACHE])
def test_bad_caches_are_refused_before_launch(lib, name, kw, code):
    c = cache(**kw)
    assert lib.fa_cache_write(R(c), R(view(5)), R(view(6)), ft.FA_BF16, 5, None, 0, None, None) == code
    assert lib.fa_last_error()
    assert lib.fa_cache_read(R(c), 0, 5, ft.FA_BF16, R(view(5)), R(view(6)), None) == code
    p = ft.FaDecodeParams(6, 1, 0, 0, 0.125, 0)
    assert lib.fa_decode(R(p), 5 * F, R(c), None, 6 * F, 7 * F, 8 * F, 1 << 33, None) == code


def test_bad_rows_are_refused_before_launch(lib):
    w = lambda n=5, k=view(5), v=view(6), dt=ft.FA_BF16, at=None, first=0, count=None: lib.fa_cache_write(  # noqa: E731
        R(cache()), R(k), R(v), dt, n, at, first, count, None)
    for bad in (dict(n=-1), dict(dt=9), dict(first=-1), dict(first=36), dict(n=41), dict(at=8 * F + 4),
                dict(count=8 * F + 2), dict(k=view(5, ptr=5 * F + 8)), dict(k=None), dict(v=view(6, stride_s=4)),
                dict(v=view(6, ptr=F + 128)), dict(at=F + 8)):
        assert w(**bad) == ft.FA_ERR_INVALID_ARG, bad
    assert w(n=0) == ft.FA_OK
    r = lambda n=5, k=view(5), v=view(6), dt=ft.FA_BF16, first=0: lib.fa_cache_read(  # noqa: E731
        R(cache()), first, n, dt, R(k), R(v), None)
    for bad in (dict(n=-1), dict(dt=9), dict(first=-1), dict(first=36), dict(k=None), dict(k=view(5, stride_s=32)),
                dict(v=view(5)), dict(v=view(6, ptr=2 * F + 16)), dict(v=view(6, stride_h=0))):
        assert r(**bad) == ft.FA_ERR_INVALID_ARG, bad
    assert r(n=0) == ft.FA_OK


def test_binding_refuses_what_does_not_fit():
    planes = kv.new_cache(2, 3, 40, 64, "q4_0", device="cpu")
    assert planes[0].shape == (2, 3, 40, 32) and planes[1].shape == (2, 3, 40, 2)
    k = torch.zeros(2, 3, 5, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        kv.cache_write(k, k.clone(), *planes, 0)
    for args, exc, word in (((planes[0].float(), *planes[1:]), TypeError, "k_q has dtype"),
                            ((planes[0], planes[1].float(), *planes[2:]), TypeError, "float16"),
                            ((planes[0], planes[1][:, :, :3], *planes[2:]), ValueError, "shapes"),
                            ((*planes[:2], planes[2].to(torch.int8), planes[3]), TypeError, "v_q has dtype"),
                            ((*planes[:2], planes[2][:, :2], planes[3]), ValueError, "v_q has shape"),
                            ((planes[0][0], *planes[1:]), ValueError, "4-D")):
        for call in (lambda: kv.cache_write(k, k, *args, 0), lambda: kv.cache_read(*args),
                     lambda: kv.decode(torch.zeros(2, 6, 1, 64, dtype=torch.bfloat16), *args)):
            with pytest.raises(exc, match=word):
                call()
    with pytest.raises(ValueError, match="fmt"):
        kv.new_cache(1, 1, 1, 64, "q5_0", device="cpu")


# ---- GPU ---------------------------------------------------------------------------------------------


def source(shape, seed):
    """Rows with ordinary blocks and with blocks at the edges: zeros, ties, one value, tiny, huge, not numbers."""
    x = np.random.default_rng(seed).standard_normal(shape).astype(np.float32)
    rows = x.reshape(-1, shape[-1])
    n = len(rows)
    rows[0 % n, :32] = 0
    rows[1 % n, :32] = np.where(np.arange(32) % 2, 3.0, -3.0)
    rows[2 % n, 32:64] = 0
    rows[2 % n, 40] = -7.25
    rows[3 % n, :32] *= 1e-9
    rows[4 % n, :32] *= 1e9
    rows[5 % n, 3] = np.inf
    rows[5 % n, 35] = np.nan
    rows[6 % n, :32] *= 2e-6   # scales that are subnormal in fp16
    rows[7 % n, 7] = -np.inf
    rows[8 % n, :32] = np.arange(32) - 15.5
    return x


def tensor(x, dtype, layout, strided):
    t = torch.from_numpy(x).to(dtype).cuda()
    t = t if layout == "bhsd" else t.transpose(1, 2)
    if not strided:
        return t.contiguous()
    wide = torch.full((*t.shape[:2], t.shape[2] + 3, t.shape[3] + 8), 5.0, dtype=dtype, device="cuda")
    out = wide[:, :, 1:1 + t.shape[2], :t.shape[3]]
    return out.copy_(t)


CASES = [("q8_0", torch.bfloat16, "bhsd", False, 64), ("q8_0", torch.float32, "bshd", True, 128),
         ("q4_0", torch.bfloat16, "bshd", True, 128), ("q4_0", torch.float32, "bhsd", False, 64),
         ("q4_0", torch.bfloat16, "bhsd", False, 128), ("q8_0", torch.bfloat16, "bshd", False, 128)]


def fill(B, H, S, D, fmt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for t in kv.new_cache(B, H, S, D, fmt):
        if t.dtype == torch.float16:
            out.append(torch.randn(t.shape, generator=g, device="cuda").half())
        else:
            lo, hi = (0, 256) if t.dtype == torch.uint8 else (-127, 128)
            out.append(torch.randint(lo, hi, t.shape, generator=g, device="cuda").to(t.dtype))
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,dtype,layout,strided,D", CASES)
@pytest.mark.parametrize("how", ["same", "each", "counted"])
def test_written_rows_are_the_oracles_blocks(fmt, dtype, layout, strided, D, how):
    B, H, S, n = 3, 2, 37, 11
    planes = fill(B, H, S, D, fmt, 1)
    before = [t.cpu().numpy().copy() for t in planes]
    src = [source((B, H, n, D), s) for s in (2, 3)]
    t = [tensor(x, dtype, layout, strided) for x in src]
    begin = [26, 26, 26] if how == "same" else [0, 9, 26]
    count = [11, 0, 5] if how == "counted" else [n] * B
    at = 26 if how == "same" else torch.tensor(begin, device="cuda")
    kv.cache_write(t[0], t[1], *planes, at, torch.tensor(count, device="cuda") if how == "counted" else None, layout=layout)
    torch.cuda.synchronize()
    assert ft.device_status() == 0
    after = [x.cpu().numpy() for x in planes]
    for i, x in enumerate(src):
        q, d = ref.quantize(torch.from_numpy(x).to(dtype).float().numpy(), fmt)
        for b in range(B):
            rows = slice(begin[b], begin[b] + count[b])
            want = [before[2 * i][b].copy(), before[2 * i + 1][b].copy()]
            want[0][:, rows], want[1][:, rows] = q[b, :, :count[b]], d[b, :, :count[b]]
            np.testing.assert_array_equal(after[2 * i][b], want[0])
            np.testing.assert_array_equal(after[2 * i + 1][b], want[1])


@pytest.mark.gpu
def test_rows_outside_the_cache_are_not_written_and_reported():
    B, H, S, D, n = 4, 2, 16, 64, 3
    planes = fill(B, H, S, D, "q4_0", 4)
    before = [t.clone() for t in planes]
    x = source((B, H, n, D), 5)
    t = tensor(x, torch.bfloat16, "bhsd", False)
    ft.device_status()
    kv.cache_write(t, t.clone(), *planes, torch.tensor([-2, 15, 1 << 40, -(1 << 62)], device="cuda"))
    torch.cuda.synchronize()
    assert ft.device_status() == (0x40000000 | 951)
    q, d = ref.quantize(t.float().cpu().numpy(), "q4_0")
    want = [b.cpu().numpy().copy() for b in before]
    for i in (0, 2):
        want[i][0, :, 0], want[i + 1][0, :, 0] = q[0, :, 2], d[0, :, 2]
        want[i][1, :, 15], want[i + 1][1, :, 15] = q[1, :, 0], d[1, :, 0]
    for a, b in zip(planes, want):
        np.testing.assert_array_equal(a.cpu().numpy(), b)
    # a count beyond the rows is the rows
    kv.cache_write(t, t.clone(), *planes, 4, torch.tensor([99, -5, 3, 1], device="cuda"))
    torch.cuda.synchronize()
    assert ft.device_status() == 0
    np.testing.assert_array_equal(planes[0][0, :, 4:7].cpu().numpy(), q[0])
    np.testing.assert_array_equal(planes[0][1].cpu().numpy(), want[0][1])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,dtype,layout,strided,D", CASES)
def test_read_back_is_exact(fmt, dtype, layout, strided, D):
    B, H, S, n = 2, 3, 41, 17
    planes = fill(B, H, S, D, fmt, 6)
    planes[1][0, 0, 3, 0] = 6.0e-8
    planes[1][0, 1, 20, 1] = 65504.0
    out = {}
    if strided:
        shape = (B, H, n, D) if layout == "bhsd" else (B, n, H, D)
        out = {x: tensor(np.zeros((B, H, n, D), np.float32), dtype, layout, True) for x in "kv"}
        assert out["k"].shape == shape
    for begin, rows in ((9, n), (S - n, n)):
        got = kv.cache_read(*planes, begin, rows, dtype=dtype, layout=layout, **out)
        torch.cuda.synchronize()
        for i, x in enumerate(got):
            want = ref.values(planes[2 * i].cpu().numpy(), planes[2 * i + 1].cpu().numpy())[:, :, begin:begin + rows]
            if dtype == torch.bfloat16:
                want = rows_ref.to_bf16_bits(want.astype(np.float32))
            x = x if layout == "bhsd" else x.transpose(1, 2)
            np.testing.assert_array_equal(x.double().cpu().numpy(), want.astype(np.float64))
    if strided:   # what lies between the rows is as it was
        base = out["k"]._base
        mask = torch.ones(base.shape, dtype=torch.bool, device="cuda")
        mask[:, :, 1:-2, :D] = False
        assert bool((base[mask] == 5.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
def test_offsets_beyond_32_bits(fmt):
    B, H, S, D = 2, 8, (1 << 21) + 5, 128   # 4.3e9 numbers a plane
    width, kind = (D // 2, torch.uint8) if fmt == "q4_0" else (D, torch.int8)
    planes = []
    for _ in range(2):
        planes.append(torch.empty((B, H, S, width), dtype=kind, device="cuda"))
        planes.append(torch.empty((B, H, S, D // 32), dtype=torch.float16, device="cuda"))
    x = source((B, H, 6, D), 7)
    t = tensor(x, torch.bfloat16, "bhsd", False)
    kv.cache_write(t, -t, *planes, S - 6)
    k, v = kv.cache_read(*planes, S - 6)
    torch.cuda.synchronize()
    for i, sign in ((0, 1.0), (2, -1.0)):
        q, d = ref.quantize(sign * t.float().cpu().numpy(), fmt)
        np.testing.assert_array_equal(planes[i][:, :, S - 6:].cpu().numpy(), q)
        np.testing.assert_array_equal(planes[i + 1][:, :, S - 6:].cpu().numpy(), d)
    q, d = ref.quantize(t.float().cpu().numpy(), fmt)
    np.testing.assert_array_equal(k.float().cpu().numpy(), rows_ref.to_bf16_bits(ref.values(q, d).astype(np.float32)))


@pytest.mark.gpu
def test_begins_that_a_64_bit_number_does_not_hold_are_refused():
    planes = kv.new_cache(1, 2, 16, 64, "q4_0")
    before = [t.clone() for t in planes]
    x = torch.ones((1, 2, 3, 64), dtype=torch.bfloat16, device="cuda")
    for begin in (14, -1, 1 << 63, 1 << 64, (1 << 64) + 2, -(1 << 64)):
        with pytest.raises(ft.FaError, match="outside"):
            kv.cache_write(x, x, *planes, begin)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(planes, before))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["q4_0", "q8_0"])
def test_quotients_between_two_numbers_and_odd_scales(fmt):
    """Values half way between two stored numbers, scales that fp16 holds with few bits or not at all, equal magnitudes of both
    signs in either half of a block, and rows of nothing: the oracle's blocks, bit for bit."""
    g = np.random.default_rng(7)
    B, H, n, D = 1, 2, 300, 128
    half = g.integers(-254, 255, (B, H, n, D)).astype(np.float32) / 2
    x = half * np.exp2(g.integers(-30, 12, (B, H, n, 1))).astype(np.float32)
    x[:, :, ::5] = g.integers(-16, 17, x[:, :, ::5].shape) / np.float32(2)
    x[:, :, 1::50] = 0
    x[:, :, 2::50] *= np.float32(1e-8)
    x[:, :, 3::50] *= np.float32(1e30)
    x[:, 0, 4::50, 3] = np.inf
    x[:, 1, 4::50, 40] = np.nan
    y = -x[:, :, ::-1].copy()
    for dtype in (torch.float32, torch.bfloat16):
        planes = kv.new_cache(B, H, n, D, fmt)
        t = [torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda() for a in (x, y)]
        kv.cache_write(t[0], t[1], *planes, 0)
        torch.cuda.synchronize()
        for i, a in enumerate(t):
            q, d = ref.quantize(a.float().cpu().numpy(), fmt)
            np.testing.assert_array_equal(planes[2 * i].cpu().numpy(), q)
            np.testing.assert_array_equal(planes[2 * i + 1].cpu().numpy(), d)
