"""RMS norm of query and key heads with the rotary position, and its backward (fa_qk_norm_rope*).

The step between a projection and the attention of this package: q and k may be views into the
fused projection's output, the results are what fwd / bwd / decode and cache_write take.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import fa_train as ft


def rope_inv_freq(rotary_dim: int, base: float = 10000.0, *, scaling: str = "none", scale: float = 1.0,
                  original_length: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """(inv_freq fp32 [rotary_dim / 2], factor) for qk_norm_rope: the angles base^(-2 i / rotary_dim), changed
    for contexts `scale` times as long as the trained one.

    scaling: "none"; "linear" (positions interpolated: every angle divided by scale); "ntk" (the base raised to
    base * scale^(rotary_dim / (rotary_dim - 2)): the slowest pair is interpolated, the fastest is not); "yarn"
    (YaRN, Peng et al. 2023: pairs that turn less than beta_slow times over original_length are interpolated, those
    above beta_fast are not, a linear ramp in between; factor = 0.1 ln(scale) + 1).
    """
    if rotary_dim < 8 or rotary_dim % 8 != 0:
        raise ValueError(f"rotary_dim {rotary_dim}: a positive multiple of 8")
    if not (scale >= 1.0 and math.isfinite(scale)):
        raise ValueError(f"scale {scale}: finite, at least 1")
    i = torch.arange(rotary_dim // 2, dtype=torch.float64)
    factor = 1.0
    if scaling == "ntk":
        base = base * scale ** (rotary_dim / (rotary_dim - 2))
    f = base ** (-2.0 * i / rotary_dim)
    if scaling == "linear":
        f = f / scale
    elif scaling == "yarn":
        def pair(turns):   # the pair that turns so often over original_length
            return rotary_dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))
        # The method's ramp is over pairs' indices. The upper bound, rotary_dim - 1 although pairs end at rotary_dim / 2 - 1, and
        # the least width, 1e-3, are those that models with these frequencies were trained with: kept, so that angles agree.
        low = max(math.floor(pair(beta_fast)), 0)
        high = min(math.ceil(pair(beta_slow)), rotary_dim - 1)
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        f = f / scale * ramp + f * (1 - ramp)
        factor = 0.1 * math.log(scale) + 1.0
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"scaling {scaling!r}: 'none', 'linear', 'ntk' or 'yarn'")
    return f.to(torch.float32).to(device or "cpu"), factor


# fa_rope_params and the call's views side by side, filled in one go: the C ABI gets the address of each.
_PARAMS = ctypes.sizeof(ft.FaRopeParams)
_VIEW = ctypes.sizeof(ft.FaView)


def _call_type(views: int):
    fields = list(ft.FaRopeParams._fields_) + [("padding", ctypes.c_int32)]
    for i in range(views):
        fields += [(f"{n}{i}", t) for n, t in ft.FaView._fields_]
    t = type(f"FaRopeCall{views}", (ctypes.Structure,), {"_fields_": fields})
    assert t.ptr0.offset == _PARAMS and ctypes.sizeof(t) == _PARAMS + views * _VIEW
    return t


_Forward, _Backward = _call_type(4), _call_type(6)


def _params(q, k, inv_freq, positions, q_weight, k_weight, eps, interleaved, factor, offset, layout):
    """The values of fa_rope_params, after the checks that the C ABI cannot make."""
    shape = q.shape
    if len(shape) != 4 or k.dim() != 4:
        raise ValueError(f"q and k must be 4-D (got {q.dim()}-D and {k.dim()}-D)")
    B, x, y, D = shape
    if layout == "bhsd":
        Hq, S, Hkv = x, y, k.shape[1]
        want = (B, Hkv, S, D)
    elif layout == "bshd":
        S, Hq, Hkv = x, y, k.shape[2]
        want = (B, S, Hkv, D)
    else:
        raise ValueError(f"layout {layout!r}: 'bhsd' or 'bshd'")
    if k.shape != want:
        raise ValueError(f"k has shape {tuple(k.shape)}, expected {want}")
    dtype = q.dtype
    if k.dtype != dtype:
        raise TypeError(f"k has dtype {k.dtype}, expected {dtype}")
    code = w_code = ft._dtype_code(q)
    on = q.get_device()
    if k.get_device() != on:
        raise ValueError(f"k is on {k.device}, q on {q.device}")
    norm = q_weight is not None
    if norm != (k_weight is not None):
        raise ValueError("give both q_weight and k_weight (norm and rotation), or neither (rotation alone)")
    if norm:
        w = q_weight.dtype
        if w != dtype:
            if w != torch.float32:
                raise TypeError(f"weights of dtype {w} and {k_weight.dtype}: both {dtype} or both float32")
            w_code = ft.FA_F32
        if k_weight.dtype != w:
            raise TypeError(f"weights of dtype {w} and {k_weight.dtype}: both {dtype} or both float32")
        if q_weight.shape != (D,) or k_weight.shape != (D,):
            raise ValueError(f"q_weight, k_weight have shapes {tuple(q_weight.shape)}, {tuple(k_weight.shape)}, expected {(D,)}")
        if not (q_weight.is_contiguous() and k_weight.is_contiguous() and q_weight.get_device() == on == k_weight.get_device()):
            raise ValueError(f"q_weight and k_weight must be contiguous and on {q.device}")
    rot = 0
    if inv_freq is not None:
        if inv_freq.dtype != torch.float32:
            raise TypeError(f"inv_freq has dtype {inv_freq.dtype}, expected torch.float32")
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must be [rotary_dim / 2]")
        rot = 2 * inv_freq.shape[0]
        if inv_freq.get_device() != on or not inv_freq.is_contiguous():
            raise ValueError(f"inv_freq must be contiguous and on {q.device}")
    pos_stride = 0
    if positions is not None:
        if positions.dtype != torch.int64:
            raise TypeError(f"positions has dtype {positions.dtype}, expected torch.int64")
        if positions.shape == (B, S):
            pos_stride = S
        elif positions.shape != (S,):
            raise ValueError(f"positions has shape {tuple(positions.shape)}, expected {(S,)} or {(B, S)}")
        if positions.get_device() != on or not positions.is_contiguous():
            raise ValueError(f"positions must be contiguous and on {q.device}")
    return (B, S, Hq, Hkv, D, code, w_code, rot, 1 if interleaved else 0, 1 if norm else 0, eps, factor,
            offset if offset == 0 else ft._held(offset), pos_stride, 0, 0)


def _same(name: str, t: torch.Tensor, like: torch.Tensor) -> None:
    if t.shape != like.shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(like.shape)}")
    if t.dtype != like.dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {like.dtype}")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, q on {like.device}")


def qk_norm_rope(q, k, inv_freq, positions=None, q_weight=None, k_weight=None, *, eps: float = 1e-6,
                 interleaved: bool = False, factor: float = 1.0, offset: int = 0, layout: str = "bhsd", q_out=None,
                 k_out=None, stream=None):
    """RMS norm of every head of q and k (with weights [D]; without, none) and the rotation of its first
    2 * len(inv_freq) features by the angles position * inv_freq, in one pass: returns (q_out, k_out).

    q: [B, Hq, S, D], k: [B, Hkv, S, D] (layout "bhsd") or [B, S, H, D] ("bshd"), bfloat16 or float32; any strides
    (multiples of 16 bytes) with the D features contiguous, so views of a fused projection's output are read in place.
    positions: int64 [S] or [B, S]; without, token s is at offset + s. interleaved: pairs (2 i, 2 i + 1) instead of
    (i, i + rotary_dim / 2). factor multiplies cosines and sines (see rope_inv_freq).
    """
    p = _params(q, k, inv_freq, positions, q_weight, k_weight, eps, interleaved, factor, offset, layout)
    if q_out is None:
        q_out = ft._like(q, stream)
    else:
        _same("q_out", q_out, q)
    if k_out is None:
        k_out = ft._like(k, stream)
    else:
        _same("k_out", k_out, k)
    c = _Forward(*p, *ft._rows(q, layout), *ft._rows(k, layout), *ft._rows(q_out, layout), *ft._rows(k_out, layout))
    at = ctypes.addressof(c)
    v = at + _PARAMS
    device = q.device
    ft._launch(device, ft.load_library().fa_qk_norm_rope, at, v, v + _VIEW,
               None if q_weight is None else q_weight.data_ptr(), None if k_weight is None else k_weight.data_ptr(),
               None if inv_freq is None else inv_freq.data_ptr(), None if positions is None else positions.data_ptr(),
               v + 2 * _VIEW, v + 3 * _VIEW, ft._stream(device, stream))
    return q_out, k_out


def qk_norm_rope_bwd(dq_out, dk_out, q, k, inv_freq, positions=None, q_weight=None, k_weight=None, *,
                     eps: float = 1e-6, interleaved: bool = False, factor: float = 1.0, offset: int = 0,
                     layout: str = "bhsd", dq=None, dk=None, dq_weight: Optional[torch.Tensor] = None,
                     dk_weight: Optional[torch.Tensor] = None, workspace=None, stream=None):
    """Backward of qk_norm_rope: from the gradients of its outputs and its inputs, returns (dq, dk, dq_weight,
    dk_weight), the weights' in float32 and summed in a fixed order (None without weights). The other arguments are
    the forward's; gradients and inputs may be strided like the forward's, and dq and dk may be parts of one tensor, as the
    gradient of a fused projection's output is."""
    p = _params(q, k, inv_freq, positions, q_weight, k_weight, eps, interleaved, factor, offset, layout)
    _same("dq_out", dq_out, q)
    _same("dk_out", dk_out, k)
    if dq is None:
        dq = ft._like(q, stream)
    else:
        _same("dq", dq, q)
    if dk is None:
        dk = ft._like(k, stream)
    else:
        _same("dk", dk, k)
    c = _Backward(*p, *ft._rows(dq_out, layout), *ft._rows(dk_out, layout), *ft._rows(q, layout), *ft._rows(k, layout),
                  *ft._rows(dq, layout), *ft._rows(dk, layout))
    at = ctypes.addressof(c)
    v = at + _PARAMS
    lib = ft.load_library()
    device = q.device
    ws, ws_bytes = None, 0
    if q_weight is not None:
        D = q.shape[3]
        if dq_weight is None:
            dq_weight = ft._empty((D,), (1,), torch.float32, device, stream)
        if dk_weight is None:
            dk_weight = ft._empty((D,), (1,), torch.float32, device, stream)
        for name, t in (("dq_weight", dq_weight), ("dk_weight", dk_weight)):
            if t.shape != (D,) or t.dtype != torch.float32 or t.device != device or not t.is_contiguous():
                raise ValueError(f"{name} must be float32 {(D,)}, contiguous and on {device}")
        ws_bytes = lib.fa_qk_norm_rope_bwd_workspace_size(at)
        ws = ft._scratch(ws_bytes, device, workspace, stream)
    else:
        dq_weight = dk_weight = None
    ft._launch(device, lib.fa_qk_norm_rope_bwd, at, v, v + _VIEW, v + 2 * _VIEW, v + 3 * _VIEW, ft._ptr(q_weight),
               ft._ptr(k_weight), ft._ptr(inv_freq), ft._ptr(positions), v + 4 * _VIEW, v + 5 * _VIEW,
               ft._ptr(dq_weight), ft._ptr(dk_weight), ft._ptr(ws), ws_bytes, ft._stream(device, stream))
    return dq, dk, dq_weight, dk_weight
