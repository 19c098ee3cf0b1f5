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
        low = max(math.floor(pair(beta_fast)), 0)
        high = min(math.ceil(pair(beta_slow)), rotary_dim - 1)
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        f = f / scale * ramp + f * (1 - ramp)
        factor = 0.1 * math.log(scale) + 1.0
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"scaling {scaling!r}: 'none', 'linear', 'ntk' or 'yarn'")
    return f.to(torch.float32).to(device or "cpu"), factor


def _params(q, k, inv_freq, positions, q_weight, k_weight, eps, interleaved, factor, offset, layout) -> ft.FaRopeParams:
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError(f"q and k must be 4-D (got {q.dim()}-D and {k.dim()}-D)")
    if layout == "bhsd":
        B, Hq, S, D = q.shape
        want = (B, k.shape[1], S, D)
        Hkv = k.shape[1]
    elif layout == "bshd":
        B, S, Hq, D = q.shape
        want = (B, S, k.shape[2], D)
        Hkv = k.shape[2]
    else:
        raise ValueError(f"layout {layout!r}: 'bhsd' or 'bshd'")
    if k.shape != want:
        raise ValueError(f"k has shape {tuple(k.shape)}, expected {want}")
    if k.dtype != q.dtype:
        raise TypeError(f"k has dtype {k.dtype}, expected {q.dtype}")
    code = ft._dtype_code(q)
    device = q.device
    if k.device != device:
        raise ValueError(f"k is on {k.device}, q on {device}")
    w_code = code
    if (q_weight is None) != (k_weight is None):
        raise ValueError("give both q_weight and k_weight (norm and rotation), or neither (rotation alone)")
    if q_weight is not None:
        if q_weight.dtype != k_weight.dtype or q_weight.dtype not in (q.dtype, torch.float32):
            raise TypeError(f"weights of dtype {q_weight.dtype} and {k_weight.dtype}: both {q.dtype} or both float32")
        w_code = ft._dtype_code(q_weight)
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w.shape != (D,):
                raise ValueError(f"{name} has shape {tuple(w.shape)}, expected {(D,)}")
            _small(name, w, device)
    rot = 0
    if inv_freq is not None:
        if inv_freq.dtype != torch.float32:
            raise TypeError(f"inv_freq has dtype {inv_freq.dtype}, expected torch.float32")
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must be [rotary_dim / 2]")
        rot = 2 * inv_freq.shape[0]
        _small("inv_freq", inv_freq, device)
    pos_stride = 0
    if positions is not None:
        if positions.dtype != torch.int64:
            raise TypeError(f"positions has dtype {positions.dtype}, expected torch.int64")
        if positions.shape != (S,) and positions.shape != (B, S):
            raise ValueError(f"positions has shape {tuple(positions.shape)}, expected {(S,)} or {(B, S)}")
        _small("positions", positions, device)
        pos_stride = S if positions.dim() == 2 else 0
    return ft.FaRopeParams(B, S, Hq, Hkv, D, code, w_code, rot, int(bool(interleaved)), int(q_weight is not None), eps,
                           factor, offset, pos_stride, 0)


def _small(name: str, t: torch.Tensor, device) -> None:
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, q on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


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
    lib = ft.load_library()
    p = _params(q, k, inv_freq, positions, q_weight, k_weight, eps, interleaved, factor, offset, layout)
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    else:
        _same("q_out", q_out, q)
    if k_out is None:
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    else:
        _same("k_out", k_out, k)
    views = [ft._view(t, layout) for t in (q, k, q_out, k_out)]
    ft._launch(q.device, lib.fa_qk_norm_rope, p, views[0], views[1], ft._ptr(q_weight), ft._ptr(k_weight),
               ft._ptr(inv_freq) if p.rot else None, ft._ptr(positions), views[2], views[3], ft._stream(q.device, stream))
    return q_out, k_out


def qk_norm_rope_bwd(dq_out, dk_out, q, k, inv_freq, positions=None, q_weight=None, k_weight=None, *,
                     eps: float = 1e-6, interleaved: bool = False, factor: float = 1.0, offset: int = 0,
                     layout: str = "bhsd", dq=None, dk=None, dq_weight: Optional[torch.Tensor] = None,
                     dk_weight: Optional[torch.Tensor] = None, workspace=None, stream=None):
    """Backward of qk_norm_rope: from the gradients of its outputs and its inputs, returns (dq, dk, dq_weight,
    dk_weight), the weights' in float32 and summed in a fixed order (None without weights). The other arguments are
    the forward's; gradients and inputs may be strided like the forward's."""
    lib = ft.load_library()
    p = _params(q, k, inv_freq, positions, q_weight, k_weight, eps, interleaved, factor, offset, layout)
    _same("dq_out", dq_out, q)
    _same("dk_out", dk_out, k)
    if dq is None:
        dq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    else:
        _same("dq", dq, q)
    if dk is None:
        dk = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    else:
        _same("dk", dk, k)
    ws, ws_bytes = None, 0
    if p.norm:
        if dq_weight is None:
            dq_weight = torch.empty(p.D, dtype=torch.float32, device=q.device)
        if dk_weight is None:
            dk_weight = torch.empty(p.D, dtype=torch.float32, device=q.device)
        for name, t in (("dq_weight", dq_weight), ("dk_weight", dk_weight)):
            if t.shape != (p.D,) or t.dtype != torch.float32:
                raise ValueError(f"{name} must be float32 {(p.D,)}")
            _small(name, t, q.device)
        ws_bytes = int(lib.fa_qk_norm_rope_bwd_workspace_size(p))
    else:
        dq_weight = dk_weight = None
    views = [ft._view(t, layout) for t in (dq_out, dk_out, q, k, dq, dk)]
    if ws_bytes:
        ws = ft._scratch(ws_bytes, q.device, workspace, stream)
    ft._launch(q.device, lib.fa_qk_norm_rope_bwd, p, views[0], views[1], views[2], views[3], ft._ptr(q_weight),
               ft._ptr(k_weight), ft._ptr(inv_freq) if p.rot else None, ft._ptr(positions), views[4], views[5],
               ft._ptr(dq_weight), ft._ptr(dk_weight), ft._ptr(ws), ws_bytes, ft._stream(q.device, stream))
    return dq, dk, dq_weight, dk_weight
