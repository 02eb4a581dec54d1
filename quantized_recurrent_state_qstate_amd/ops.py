"""The operators before the recurrence: short causal convolution, and the norm
and rotation of queries and keys.  They need no handle; like a handle's calls
they run in the library's kernels, asynchronously on the current stream of the
tensors' device (or `stream`), and raise if the library is missing.
"""
from __future__ import annotations

import ctypes

from . import _lib
from .api import _empty_like, _ptr, check_rows, check_stream, check_tensor, raw_stream


def _device(name: str, x):
    import torch
    if not isinstance(x, torch.Tensor):
        raise ValueError(f"{name}: expected a torch.Tensor, got {type(x).__name__}")
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"{name}: dtype {x.dtype}, expected torch.bfloat16 or torch.float32")
    return x.device


def _call(fn, name: str, args, device, stream) -> None:
    """Launch on `stream` (None: the device's current one) with the tensors' device current."""
    if device.type != "cuda":
        raise ValueError(f"{name}: tensors on {device}, expected a GPU")
    import torch
    if device.index == torch._C._cuda_getDevice():
        status = fn(ctypes.byref(args), raw_stream(stream, device))
        if status:
            _lib.check(status, name)
    else:
        with torch.cuda.device(device):
            _lib.check(fn(ctypes.byref(args), raw_stream(stream, device)), name)


def _conv(x, weight, bias, window, slot, n, silu, out, stream):
    import torch
    dev = _device("x", x)
    check_stream(stream, dev)
    if x.dim() != 2 or not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("x must be [tokens, C] and weight [W, C]")
    (T, C), W = x.shape, weight.shape[0]
    dtype, slots = x.dtype, 0
    xs = check_rows("x", x, dtype, (T, C), dev)
    check_tensor("weight", weight, torch.float32, W * C, dev)
    if bias is not None:
        check_tensor("bias", bias, torch.float32, C, dev)
    if window is not None:
        if not isinstance(window, torch.Tensor) or window.dim() != 3:
            raise ValueError("window must be [slots, W-1, C]")
        slots = window.shape[0]
        check_tensor("window", window, dtype, slots * (W - 1) * C, dev)
        if window.shape != (slots, W - 1, C):
            raise ValueError(f"window: shape {tuple(window.shape)}, expected {(slots, W - 1, C)}")
    if slot is not None:
        check_tensor("slot", slot, torch.int32, n, dev)
    if out is None:
        out = _empty_like(x, xs == C, stream)
        os = C
    else:
        os = check_rows("out", out, dtype, (T, C), dev)
    a = _lib.Conv(x.data_ptr(), out.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(window), _ptr(slot), None, xs, os,
                  _lib.DTYPE["bf16" if dtype is torch.bfloat16 else "fp32"], T, C, W, n, slots, 1 if silu else 0)
    return a, out, dev


def causal_conv(x, weight, bias=None, *, offsets, window=None, slot=None, silu=True, out=None, stream=None):
    """Causal convolution of each channel over packed prompts: returns out [T, C].

    x [T, C] bf16 or fp32 (its rows may lie in a wider tensor); weight fp32
    [W, C], W = 2..4, the last tap on the token itself; bias fp32 [C] or None.
    offsets int32 [n+1] on the device: sequence i is tokens
    offsets[i]..offsets[i+1]-1; other tokens of `out` are left as they were.
    window [slots, W-1, C] in x's dtype, with slot int32 [n] (None: sequence i
    has window i): the rows before each sequence (all zeros: none), replaced
    by its last W-1 rows; None: sequences begin with zeros.  A sequence whose
    slot is out of range is skipped; two with one slot race."""
    import torch
    if not isinstance(offsets, torch.Tensor) or offsets.numel() < 1:
        raise ValueError("offsets must be an int32 tensor [n+1]")
    n = offsets.numel() - 1
    a, out, dev = _conv(x, weight, bias, window, slot, n, silu, out, stream)
    check_tensor("offsets", offsets, torch.int32, n + 1, dev)
    a.offsets = offsets.data_ptr()
    _call(_lib.lib().qstate_causal_conv, "qstate_causal_conv", a, dev, stream)
    return out


def causal_conv_step(x, weight, bias=None, *, window, slot=None, silu=True, out=None, stream=None):
    """One token for each of n sequences: x [n, C], row i with window slot[i]
    (None: i), which moves on by that token; returns out [n, C].  Otherwise as
    `causal_conv`."""
    if window is None:
        raise ValueError("window must be [slots, W-1, C]")
    n = x.shape[0] if hasattr(x, "shape") and len(x.shape) else 0
    a, out, dev = _conv(x, weight, bias, window, slot, n, silu, out, stream)
    _call(_lib.lib().qstate_causal_conv_step, "qstate_causal_conv_step", a, dev, stream)
    return out


def qk_norm_rotate(q, k=None, *, norm="l2", q_weight=None, k_weight=None, eps=1e-6, position=None, frequency=None,
                   interleaved=False, q_scale=1.0, q_out=None, k_out=None, stream=None):
    """Norm of each query and key head, then the rotation by position, in one
    pass: returns (q_out, k_out).

    q [T, Hq, d], k [T, Hk, d] or None, bf16 or fp32, d a multiple of 8 up to
    512; the rows may lie in a wider tensor if each starts 16-byte aligned.
    norm: "l2" (x / sqrt(sum x^2 + eps)), "rms" (x / sqrt(mean x^2 + eps),
    times q_weight / k_weight fp32 [d] if given) or "none"; a head of zeros
    with eps 0 gives NaN.
    frequency fp64 [rot/2] (radians per position) with position int32 [T]:
    the first `rot` channels turn, in pairs (i, i + rot/2), or (2i, 2i+1) when
    interleaved.  q_scale multiplies q_out.  q_out may be q, k_out may be k."""
    import torch
    dev = _device("q", q)
    check_stream(stream, dev)
    if q.dim() != 3 or (k is not None and (not isinstance(k, torch.Tensor) or k.dim() != 3)):
        raise ValueError("q and k must be [T, heads, dim]")
    (T, hq, d), dtype = q.shape, q.dtype
    hk = kp = ko = rot = 0
    ks = kos = hq * d
    qs = check_rows("q", q, dtype, (T, hq, d), dev)
    if q_out is None:
        q_out = _empty_like(q, qs == hq * d, stream)
        qos = hq * d
    else:
        qos = check_rows("q_out", q_out, dtype, (T, hq, d), dev)
    if k is not None:
        hk = k.shape[1]
        ks = check_rows("k", k, dtype, (T, hk, d), dev)
        if k_out is None:
            k_out = _empty_like(k, ks == hk * d, stream)
            kos = hk * d
        else:
            kos = check_rows("k_out", k_out, dtype, (T, hk, d), dev)
        kp, ko = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    if q_weight is not None:
        check_tensor("q_weight", q_weight, torch.float32, d, dev)
    if k_weight is not None:
        check_tensor("k_weight", k_weight, torch.float32, d, dev)
    if (frequency is None) != (position is None):
        raise ValueError("position and frequency go together")
    if frequency is not None:
        check_tensor("position", position, torch.int32, T, dev)
        check_tensor("frequency", frequency, torch.float64, frequency.numel(), dev)
        rot = 2 * frequency.numel()
    if norm not in _lib.NORM:
        raise ValueError(f"norm {norm!r} (l2, rms or none)")
    a = _lib.Qk(q.data_ptr(), kp, q_out.data_ptr(), ko, _ptr(q_weight), _ptr(k_weight), _ptr(position),
                _ptr(frequency), qs, ks, qos, kos, _lib.DTYPE["bf16" if dtype is torch.bfloat16 else "fp32"], T, hq,
                hk, d, rot, _lib.NORM[norm], 1 if interleaved else 0, eps, q_scale)
    _call(_lib.lib().qstate_qk_norm_rotate, "qstate_qk_norm_rotate", a, dev, stream)
    return q_out, k_out
