"""A quantized K/V cache, in one piece for each sequence or in pages: written, read back, attended to in place and cut to the
keys that matter (fa_cache_write, fa_cache_read, fa_decode, fa_prefill, fa_cache_weights, fa_cache_evict).

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
    """Planes (k_q, k_d, v_q, v_d) of a cache whose values are all 0, with room for S keys per sequence.

    A pool of pages is the same with B pages of S keys (a multiple of 16); the calls that take a `table` find key j of
    sequence b at row j % S of page table[b, j // S] of it (int32 [sequences, pages of a sequence] on the device; entries
    behind a sequence's keys are not looked at, one that is no page is reported by device_status(); in place of a page that a
    window hides and that was given up any page of the pool will do)."""
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


def _paged(c, table, device):
    """(the sequences and the keys they have room for: (B, Hkv, S, D), the address of fa_pages, what holds it) of a cache's
    values c and its page table. Without a table they are the first four of c, which the callers take without a call: one
    costs a tenth of a launch."""
    if table.dtype != torch.int32:
        raise TypeError(f"table has dtype {table.dtype}, expected torch.int32")
    if table.dim() != 2:
        raise ValueError(f"table must be [B, pages of a sequence] (got {table.dim()}-D)")
    if table.device != device:
        raise ValueError(f"table is on {table.device}, the cache on {device}")
    B, M = table.shape
    stride, step = table.stride()
    if step != 1 and M > 1:
        raise ValueError("the entries of a sequence in table must be contiguous")
    if max(B, M) > 0x7fffffff:
        raise ValueError(f"table has shape {tuple(table.shape)}: every dimension below 2^31")
    pages = ft.FaPages(table.data_ptr(), stride, B, M)
    return (B, c[1], M * c[2], c[3]), ctypes.addressof(pages), pages


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


def cache_write(k, v, k_q, k_d, v_q, v_d, begin, count=None, *, table=None, layout: str = "bhsd", stream=None) -> None:
    """Quantizes new rows of K and V into the cache: row r of sequence b becomes key begin[b] + r.

    k, v: [B, Hkv, n, D] (or [B, n, Hkv, D] with layout "bshd"), bfloat16 or float32, strided like qk_norm_rope's
    inputs. begin: an int for every sequence, or int64 [B] on the device (a row that would land outside the cache is
    not written and is reported by device_status()). count: int64 [B] on the device: only the first count[b] rows of
    sequence b are written. Nothing else in the cache changes. table: the planes are a pool of pages (see new_cache).
    """
    c = _cache(k_q, k_d, v_q, v_d)
    device = k_q.device
    seen, pages, held = _paged(c, table, device) if table is not None else (c, None, None)
    n = k.shape[2 if layout == "bhsd" else 1] if k.dim() == 4 else -1
    shape = _rows_shape(seen, n, layout)
    if k.shape != shape or v.shape != shape:
        raise ValueError(f"k, v have shapes {tuple(k.shape)}, {tuple(v.shape)}, expected {shape}")
    if k.get_device() != device.index or v.get_device() != device.index:
        raise ValueError(f"k is on {k.device}, v on {v.device}, the cache on {device}")
    if v.dtype != k.dtype:
        raise TypeError(f"v has dtype {v.dtype}, expected {k.dtype}")
    if isinstance(begin, torch.Tensor):
        begins, first = _per_sequence("begin", begin, seen[0], device), 0
    else:
        begins, first = None, ft._held(begin)
    counts = None if count is None else _per_sequence("count", count, seen[0], device)
    call = _RowsCall(*c, *ft._rows(k, layout), *ft._rows(v, layout))
    at = ctypes.addressof(call)
    ft._launch(device, ft.load_library().fa_cache_write_pages, at, pages, at + _CACHE, at + _CACHE + _VIEW,
               ft._dtype_code(k), min(n, 0x7fffffff), begins, first, counts, ft._stream(device, stream))


def cache_read(k_q, k_d, v_q, v_d, begin=0, n_rows=None, *, table=None, dtype=torch.bfloat16, layout: str = "bhsd",
               k=None, v=None, stream=None):
    """The values of keys begin .. begin + n_rows - 1 (default: to the end) of every sequence and head: (k, v)
    [B, Hkv, n_rows, D] (or [B, n_rows, Hkv, D]) in dtype (bfloat16 or float32), or written into the given k and v.
    begin: a number for every sequence (in a tensor too), or int64 [B] on the device (with n_rows; a row outside
    the cache is read as zeros and is reported by device_status()). table: the planes are a pool of pages (see new_cache)."""
    c = _cache(k_q, k_d, v_q, v_d)
    device = k_q.device
    seen, pages, held = _paged(c, table, device) if table is not None else (c, None, None)
    S = seen[2]
    begins = None
    own = type(begin) is not int and isinstance(begin, torch.Tensor)   # of each sequence, or a number in a tensor
    if own and begin.numel() == 1 and (begin.dim() == 0 or n_rows is None or begin.dtype != torch.int64 or begin.device != device):
        own = False
    if own:
        if n_rows is None:
            raise ValueError("n_rows is needed where every sequence has its own begin")
        begins, first, n = _per_sequence("begin", begin, seen[0], device), 0, int(n_rows)
        if not 0 <= n <= 0x7fffffff:
            raise ValueError(f"n_rows {n_rows}: not negative, below 2^31")
    else:
        first = int(begin)
        n = S - first if n_rows is None else int(n_rows)
        if first < 0 or n < 0 or first + n > S:
            raise ValueError(f"rows [{first}, {first + n}) outside the {S} keys")
    shape = _rows_shape(seen, n, layout)
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
    ft._launch(device, ft.load_library().fa_cache_read_pages, at, pages, begins, first, n, ft._dtype_code(k), at + _CACHE,
               at + _CACHE + _VIEW, ft._stream(device, stream))
    return k, v


def _queries(q, seen, device, layout: str, out, lse, stream, attend: bool = True):
    """(Hq, Sq, the layout's code, out, lse) of q [B, Hq, Sq, D] or [B, Sq, Hq, D] over a cache of shape `seen`: of a call that
    attends the results, new ones where none are given. (One function, as a call of Python's costs a tenth of a launch.)"""
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
    if B != seen[0] or D != seen[3]:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected batch {seen[0]} and {seen[3]} features as in the cache")
    if q.device != device:
        raise ValueError(f"q is on {q.device}, the cache on {device}")
    ft._need_cuda(q)
    if not attend:
        return Hq, Sq, code, out, lse
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
    return Hq, Sq, code, out, lse


def _window(window: int) -> int:
    """One that is no 32-bit number as one; a longer window than any cache hides nothing."""
    return -1 if window < 0 else 0x7fffffff


def decode(q, k_q, k_d, v_q, v_d, lengths=None, *, table=None, scale=None, window: int = 0, layout: str = "bhsd", out=None,
           lse=None, workspace=None, stream=None):
    """Attention of the newest Sq tokens (1 to 16) of every sequence over its quantized cache: (O, LSE [B, Hq, Sq]).

    q: bfloat16 [B, Hq, Sq, D] (or [B, Sq, Hq, D] with layout "bshd"). lengths: int64 [B] on the device, the keys of
    each sequence with the Sq tokens' own among them (without: all S keys); query i sits at lengths[b] - Sq + i and sees
    the keys up to its position, with window > 0 only the last `window` before it. A query that sees no key gets O = 0
    and LSE = 0. table: the planes are a pool of pages (see new_cache).
    """
    c = _cache(k_q, k_d, v_q, v_d)
    device = k_q.device
    seen, pages, held = _paged(c, table, device) if table is not None else (c, None, None)
    Hq, Sq, code, out, lse = _queries(q, seen, device, layout, out, lse, stream)
    lens = None if lengths is None else _per_sequence("lengths", lengths, seen[0], device)
    call = _DecodeCall(*c, Hq, Sq, window if 0 <= window <= 0x7fffffff else _window(window), code, 1.0 / math.sqrt(c[3]) if scale is None else scale, 0)
    at = ctypes.addressof(call)
    lib = ft.load_library()
    ws_bytes = lib.fa_decode_pages_workspace_size(at + _CACHE, at, pages)
    ws = ft._scratch(ws_bytes, device, workspace, stream)
    ft._launch(device, lib.fa_decode_pages, at + _CACHE, q.data_ptr(), at, pages, lens, out.data_ptr(), lse.data_ptr(),
               ft._ptr(ws), ws_bytes, ft._stream(device, stream))
    return out, lse


def prefill(q, k_q, k_d, v_q, v_d, lengths=None, count=None, *, table=None, scale=None, window: int = 0,
            layout: str = "bhsd", out=None, lse=None, workspace=None, stream=None):
    """Attention of a chunk of new tokens of every sequence, a ragged batch, over its quantized cache: (O, LSE [B, Hq, Sq]).

    q: bfloat16 [B, Hq, Sq, D] (or [B, Sq, Hq, D] with layout "bshd"), of any Sq. count: int64 [B] on the device, the
    tokens among the Sq rows of each sequence (without: all). lengths: int64 [B] on the device, the keys of each sequence
    with its tokens' own among them (without: all that it has room for). Token i sits at lengths[b] - count[b] + i and sees
    the keys up to its position, with window > 0 only the last `window` before it; one that sees no key gets O = 0 and
    LSE = 0. The rows from count[b] on are left as they are in out and lse. table: the planes are a pool of pages (see
    new_cache). K and V are rounded to bf16, as fwd_q8 and fwd_q4 do; for up to 16 tokens of each sequence decode is the
    faster form, on unrounded ones.
    """
    c = _cache(k_q, k_d, v_q, v_d)
    device = k_q.device
    seen, pages, held = _paged(c, table, device) if table is not None else (c, None, None)
    Hq, Sq, code, out, lse = _queries(q, seen, device, layout, out, lse, stream)
    lens = None if lengths is None else _per_sequence("lengths", lengths, seen[0], device)
    counts = None if count is None else _per_sequence("count", count, seen[0], device)
    call = _DecodeCall(*c, Hq, min(Sq, 0x7fffffff), window if 0 <= window <= 0x7fffffff else _window(window), code,
                       1.0 / math.sqrt(c[3]) if scale is None else scale, 0)
    at = ctypes.addressof(call)
    lib = ft.load_library()
    ws_bytes = lib.fa_prefill_workspace_size(at + _CACHE, at, pages)
    ws = ft._scratch(ws_bytes, device, workspace, stream)
    ft._launch(device, lib.fa_prefill, at + _CACHE, q.data_ptr(), at, pages, lens, counts, out.data_ptr(), lse.data_ptr(),
               ft._ptr(ws), ws_bytes, ft._stream(device, stream))
    return out, lse


def _key_weights(name: str, t, B: int, Hkv: int, device) -> int:
    """Elements a head has in weights float32 [B, Hkv, W]."""
    if t.dtype != torch.float32:
        raise TypeError(f"{name} has dtype {t.dtype}, expected torch.float32")
    if t.dim() != 3 or t.shape[:2] != (B, Hkv):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(B, Hkv, 'W')}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    ft._need_cuda(t)
    return t.shape[2]


def cache_weights(q, lse, k_q, k_d, lengths=None, count=None, *, weights=None, out=None, table=None, scale=None,
                  window: int = 0, layout: str = "bhsd", decoded: bool = False, stream=None):
    """The attention weight that every key got from the new tokens, added to `weights`: float32 [B, Hkv, W].

    out[b, h, j] = weights[b, h, j] + sum of exp(scale q k_j - lse) over the tokens that see key j and the query heads of
    head h. q, lengths, count, table, scale, window and layout are those of prefill, lse [B, Hq, Sq] is what it returned, and K is
    rounded to bf16 as there. decoded: they are those of decode (up to 16 tokens, all of them: no count), which does not round K,
    and the weights go with its LSE. weights: W at least the longest length (without: zeros, W what a
    sequence has room for). out may be weights; without, it is a new tensor.
    """
    if decoded and count is not None:
        raise ValueError("decode attends with all of q's tokens: no count")
    c = _cache(k_q, k_d, k_q, k_d)
    device = k_q.device
    seen, pages, held = _paged(c, table, device) if table is not None else (c, None, None)
    B, Hkv, S, D = seen[:4]
    Hq, Sq, code, out, lse = _queries(q, seen, device, layout, out, lse, stream, attend=False)
    if lse.shape != (B, Hq, Sq) or lse.dtype != torch.float32 or lse.device != device:
        raise ValueError(f"lse must be float32 {(B, Hq, Sq)} on {device}")
    ft._need_cuda(lse)
    W = S if weights is None else _key_weights("weights", weights, B, Hkv, device)
    if out is None:
        out = ft._empty((B, Hkv, W), (Hkv * W, W, 1), torch.float32, device, stream)
    elif _key_weights("out", out, B, Hkv, device) != W:
        if weights is not None:
            raise ValueError(f"out has shape {tuple(out.shape)}, weights {tuple(weights.shape)}")
        W = out.shape[2]
    lens = None if lengths is None else _per_sequence("lengths", lengths, B, device)
    counts = None if count is None else _per_sequence("count", count, B, device)
    call = _DecodeCall(*c, Hq, min(Sq, 0x7fffffff), window if 0 <= window <= 0x7fffffff else _window(window), code, 1.0 / math.sqrt(D) if scale is None else scale, 0)
    at = ctypes.addressof(call)
    lib, which = ft.load_library(), (lens,) if decoded else (lens, counts)
    ft._launch(device, lib.fa_cache_weights_decoded if decoded else lib.fa_cache_weights, at + _CACHE, q.data_ptr(), lse.data_ptr(),
               at, pages, *which, ft._ptr(weights), W, out.data_ptr(), ft._stream(device, stream))
    return out


def cache_evict(k_q, k_d, v_q, v_d, weights, lengths, keep: int, *, sinks: int = 0, recent: int = 0, table=None,
                table_out=None, weights_out=None, kept=None, lengths_out=None, stream=None):
    """Cuts every sequence that has more than `keep` keys to `keep` for each head: (kept int32 [B, Hkv, keep], new lengths
    int64 [B]).

    The keys below `sinks` and the last `recent` stay, and of the others those with the largest weights (float32 [B, Hkv, W],
    see cache_weights; of equal ones the lowest index), in the order they had: kept[b, h, i] is the index that key i of head
    h had, -1 behind the last. lengths: int64 [B] on the device. The rows move to the first pages of table, or to those of
    table_out (int32 [B, ...] with room for `keep` keys), which leaves the pages of table as they are; without a table,
    to the front of the sequence. A page that rows move to is in one place of one table only: sequences that share pages
    need a table_out (table itself, or its first columns, means in place). The weights of the keys that stay go to weights_out (default: weights itself), 0 behind them.
    """
    c = _cache(k_q, k_d, v_q, v_d)
    device = k_q.device
    seen, pages, held = _paged(c, table, device) if table is not None else (c, None, None)
    if table_out is not None and table is None:
        raise ValueError("table_out needs a table")
    to, to_held = None, None
    if table_out is not None:
        there, to, to_held = _paged(c, table_out, device)
        if there[0] != seen[0]:
            raise ValueError(f"table_out is for {there[0]} sequences, table for {seen[0]}")
    B, Hkv = seen[:2]
    W = _key_weights("weights", weights, B, Hkv, device)
    if weights_out is None:
        weights_out = weights
    elif _key_weights("weights_out", weights_out, B, Hkv, device) != W:
        raise ValueError(f"weights_out has shape {tuple(weights_out.shape)}, weights {tuple(weights.shape)}")
    lens = _per_sequence("lengths", lengths, B, device)
    keep, sinks, recent = (max(-1, min(int(n), 0x7fffffff)) for n in (keep, sinks, recent))
    if not 1 <= keep <= 1 << 24:   # before `kept` is made as large
        raise ValueError(f"keep {keep}: 1 to 2^24")
    if kept is None:
        kept = ft._empty((B, Hkv, keep), (Hkv * keep, keep, 1), torch.int32, device, stream)
    else:
        if kept.shape != (B, Hkv, keep) or kept.dtype != torch.int32 or kept.device != device:
            raise ValueError(f"kept must be int32 {(B, Hkv, keep)} on {device}")
        ft._need_cuda(kept)
    if lengths_out is None:
        lengths_out = ft._empty((B,), (1,), torch.int64, device, stream)
    new_lens = _per_sequence("lengths_out", lengths_out, B, device)
    params = ft.FaEvictParams(keep, sinks, recent, 0)
    call = ft.FaCache(*c)
    ft._launch(device, ft.load_library().fa_cache_evict, ctypes.addressof(params), ctypes.addressof(call), pages, to,
               weights.data_ptr(), W, lens, weights_out.data_ptr(), kept.data_ptr(), new_lens, ft._stream(device, stream))
    return kept, lengths_out
