"""A quantized K/V cache: written, read back and attended to in place (fa_cache_write, fa_cache_read, fa_decode).

The cache is four planes: k_q, v_q (int8 [B, Hkv, S, D] for q8_0, uint8 [B, Hkv, S, D / 2] for q4_0) and k_d, v_d
(float16 [B, Hkv, S, D / 32]); new_cache makes them, and fwd_q8 / bwd_q8 / fwd_q4 / bwd_q4 train over them.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import fa_train as ft

FORMATS = {"q8_0": ft.FA_KV_Q8_0, "q4_0": ft.FA_KV_Q4_0}


def new_cache(B: int, Hkv: int, S: int, D: int, fmt: str = "q8_0", device="cuda"):
    """Planes (k_q, k_d, v_q, v_d) of a cache whose values are all 0, with room for S keys per sequence."""
    if fmt not in FORMATS:
        raise ValueError(f"fmt {fmt!r}: 'q8_0' or 'q4_0'")
    if D % 32 != 0:
        raise ValueError(f"D {D}: a multiple of 32")
    planes = []
    for _ in range(2):
        if fmt == "q4_0":
            planes.append(torch.full((B, Hkv, S, D // 2), 0x88, dtype=torch.uint8, device=device))
        else:
            planes.append(torch.zeros((B, Hkv, S, D), dtype=torch.int8, device=device))
        planes.append(torch.zeros((B, Hkv, S, D // 32), dtype=torch.float16, device=device))
    return tuple(planes)


# fa_cache and what goes with it side by side, filled in one go: the C ABI gets the address of each.
_CACHE = ctypes.sizeof(ft.FaCache)
_VIEW = ctypes.sizeof(ft.FaView)


class _RowsCall(ctypes.Structure):
    _fields_ = list(ft.FaCache._fields_) + [(f"{n}{i}", t) for i in range(2) for n, t in ft.FaView._fields_]


class _DecodeCall(ctypes.Structure):
    _fields_ = list(ft.FaCache._fields_) + [("d" + n, t) for n, t in ft.FaDecodeParams._fields_]


assert _RowsCall.ptr0.offset == _CACHE and _RowsCall.ptr1.offset == _CACHE + _VIEW and _DecodeCall.dHq.offset == _CACHE


def _cache(k_q, k_d, v_q, v_d):
    """The values of fa_cache for the planes, after the checks that the C ABI cannot make; the format follows from
    the values' dtype."""
    shape, kind = k_q.shape, k_q.dtype
    if len(shape) != 4:
        raise ValueError(f"k_q must be 4-D (got {k_q.dim()}-D)")
    B, Hkv, S, D = shape
    if kind == torch.uint8:
        fmt, D = ft.FA_KV_Q4_0, 2 * D
    elif kind == torch.int8:
        fmt = ft.FA_KV_Q8_0
    else:
        raise TypeError(f"k_q has dtype {kind}: int8 (q8_0) or uint8 (q4_0)")
    if max(shape) > 0x7fffffff:   # the C ABI's numbers are 32-bit ones, and ctypes would wrap it
        raise ValueError(f"k_q has shape {tuple(shape)}: every dimension below 2^31")
    if v_q.dtype != kind:
        raise TypeError(f"v_q has dtype {v_q.dtype}, expected {kind}")
    if k_d.dtype != torch.float16 or v_d.dtype != torch.float16:
        raise TypeError("k_d and v_d must be float16 [B, Hkv, S, D / 32]")
    if v_q.shape != shape:
        raise ValueError(f"v_q has shape {tuple(v_q.shape)}, expected {tuple(shape)}")
    scales = (B, Hkv, S, D // 32)
    if k_d.shape != scales or v_d.shape != scales:
        raise ValueError(f"k_d, v_d have shapes {tuple(k_d.shape)}, {tuple(v_d.shape)}, expected {scales}")
    on = k_q.get_device()
    if not (k_d.get_device() == on == v_q.get_device() == v_d.get_device()):
        raise ValueError("the planes of a cache must be on one device")
    ft._need_cuda(k_q, k_d, v_q, v_d)
    return B, Hkv, S, D, fmt, 0, k_q.data_ptr(), k_d.data_ptr(), v_q.data_ptr(), v_d.data_ptr()


def _rows_shape(c, n: int, layout: str):
    if layout == "bhsd":
        return (c[0], c[1], n, c[3])
    if layout == "bshd":
        return (c[0], n, c[1], c[3])
    raise ValueError(f"layout {layout!r}: 'bhsd' or 'bshd'")


def _per_sequence(name: str, t: torch.Tensor, B: int, device) -> int:
    if t.dtype != torch.int64:
        raise TypeError(f"{name} has dtype {t.dtype}, expected torch.int64")
    if t.shape != (B,):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(B,)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def cache_write(k, v, k_q, k_d, v_q, v_d, begin, count=None, *, layout: str = "bhsd", stream=None) -> None:
    """Quantizes new rows of K and V into the cache: row r of sequence b becomes key begin[b] + r.

    k, v: [B, Hkv, n, D] (or [B, n, Hkv, D] with layout "bshd"), bfloat16 or float32, strided like qk_norm_rope's
    inputs. begin: an int for every sequence, or int64 [B] on the device (a row that would land outside the cache is
    not written and is reported by device_status()). count: int64 [B] on the device: only the first count[b] rows of
    sequence b are written. Nothing else in the cache changes.
    """
    c = _cache(k_q, k_d, v_q, v_d)
    device = k_q.device
    n = k.shape[2 if layout == "bhsd" else 1] if k.dim() == 4 else -1
    shape = _rows_shape(c, n, layout)
    if k.shape != shape or v.shape != shape:
        raise ValueError(f"k, v have shapes {tuple(k.shape)}, {tuple(v.shape)}, expected {shape}")
    if k.get_device() != device.index or v.get_device() != device.index:
        raise ValueError(f"k is on {k.device}, v on {v.device}, the cache on {device}")
    if v.dtype != k.dtype:
        raise TypeError(f"v has dtype {v.dtype}, expected {k.dtype}")
    if isinstance(begin, torch.Tensor):
        begins, first = _per_sequence("begin", begin, c[0], device), 0
    else:
        begins, first = None, ft._held(begin)
    counts = None if count is None else _per_sequence("count", count, c[0], device)
    call = _RowsCall(*c, *ft._rows(k, layout), *ft._rows(v, layout))
    at = ctypes.addressof(call)
    ft._launch(device, ft.load_library().fa_cache_write, at, at + _CACHE, at + _CACHE + _VIEW, ft._dtype_code(k),
               min(n, 0x7fffffff), begins, first, counts, ft._stream(device, stream))


def cache_read(k_q, k_d, v_q, v_d, begin: int = 0, n_rows=None, *, dtype=torch.bfloat16, layout: str = "bhsd", k=None,
               v=None, stream=None):
    """The values of keys begin .. begin + n_rows - 1 (default: to the end) of every sequence and head: (k, v)
    [B, Hkv, n_rows, D] (or [B, n_rows, Hkv, D]) in dtype (bfloat16 or float32), or written into the given k and v."""
    c = _cache(k_q, k_d, v_q, v_d)
    device, S = k_q.device, c[2]
    begin = int(begin)
    n = S - begin if n_rows is None else int(n_rows)
    if begin < 0 or n < 0 or begin + n > S:
        raise ValueError(f"rows [{begin}, {begin + n}) outside the {S} keys")
    shape = _rows_shape(c, n, layout)
    given = k is not None or v is not None
    strides = (shape[1] * shape[2] * shape[3], shape[2] * shape[3], shape[3], 1)
    k = ft._empty(shape, strides, dtype, device, stream) if k is None else k
    v = ft._empty(shape, strides, k.dtype, device, stream) if v is None else v
    if given:
        for name, t in (("k", k), ("v", v)):
            if t.shape != shape:
                raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
            if t.dtype != k.dtype:
                raise TypeError(f"{name} has dtype {t.dtype}, expected {k.dtype}")
            if t.device != device:
                raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    call = _RowsCall(*c, *ft._rows(k, layout), *ft._rows(v, layout))
    at = ctypes.addressof(call)
    ft._launch(device, ft.load_library().fa_cache_read, at, begin, n, ft._dtype_code(k), at + _CACHE,
               at + _CACHE + _VIEW, ft._stream(device, stream))
    return k, v


def decode(q, k_q, k_d, v_q, v_d, lengths=None, *, scale=None, window: int = 0, layout: str = "bhsd", out=None,
           lse=None, workspace=None, stream=None):
    """Attention of the newest Sq tokens (1 to 16) of every sequence over its quantized cache: (O, LSE [B, Hq, Sq]).

    q: bfloat16 [B, Hq, Sq, D] (or [B, Sq, Hq, D] with layout "bshd"). lengths: int64 [B] on the device, the keys of
    each sequence with the Sq tokens' own among them (without: all S keys); query i sits at lengths[b] - Sq + i and sees
    the keys up to its position, with window > 0 only the last `window` before it. A query that sees no key gets O = 0
    and LSE = 0.
    """
    c = _cache(k_q, k_d, v_q, v_d)
    device = k_q.device
    if q.dtype != torch.bfloat16:
        raise TypeError(f"q has dtype {q.dtype}, expected torch.bfloat16")
    if q.dim() != 4:
        raise ValueError(f"q must be 4-D (got {q.dim()}-D)")
    B, Hq, Sq, D = q.shape
    code = ft.FA_LAYOUT_BHSD
    if layout == "bshd":
        Hq, Sq, code = Sq, Hq, ft.FA_LAYOUT_BSHD
    elif layout != "bhsd":
        raise ValueError(f"layout {layout!r}: 'bhsd' or 'bshd'")
    if B != c[0] or D != c[3]:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected batch {c[0]} and {c[3]} features as in the cache")
    if q.device != device:
        raise ValueError(f"q is on {q.device}, the cache on {device}")
    ft._need_cuda(q)
    if out is None:
        out = ft._like(q, stream)
    else:
        if out.shape != q.shape or out.dtype != q.dtype or out.device != device:
            raise ValueError(f"out must be {q.dtype} {tuple(q.shape)} on {device}")
        ft._need_cuda(out)
    if lse is None:
        lse = ft._empty((B, Hq, Sq), (Hq * Sq, Sq, 1), torch.float32, device, stream)
    else:
        if lse.shape != (B, Hq, Sq) or lse.dtype != torch.float32 or lse.device != device:
            raise ValueError(f"lse must be float32 {(B, Hq, Sq)} on {device}")
        ft._need_cuda(lse)
    lens = None if lengths is None else _per_sequence("lengths", lengths, B, device)
    if not 0 <= window <= 0x7fffffff:   # as a 32-bit number; a longer window than any cache hides nothing
        window = -1 if window < 0 else 0x7fffffff
    call = _DecodeCall(*c, Hq, Sq, window, code, 1.0 / math.sqrt(D) if scale is None else scale, 0)
    at = ctypes.addressof(call)
    lib = ft.load_library()
    ws_bytes = lib.fa_decode_workspace_size(at + _CACHE, at)
    ws = ft._scratch(ws_bytes, device, workspace, stream)
    ft._launch(device, lib.fa_decode, at + _CACHE, q.data_ptr(), at, lens, out.data_ptr(), lse.data_ptr(), ft._ptr(ws),
               ws_bytes, ft._stream(device, stream))
    return out, lse
