"""The operators around the decode step, from their definitions in float64 on
the CPU: convolution, norm and rotation, slot copies, scan token by token."""
from __future__ import annotations

import numpy as np
import torch


def half_step(dtype) -> float:
    """Largest relative error of one rounding to dtype."""
    return float(torch.finfo(dtype).eps) / 2


def conv(x, weight, bias, lengths, windows, silu=True):
    """x [T, C], windows: one [W-1, C] per sequence; returns (out, new windows,
    magnitude sum |w x| + |b|, y before the activation), float64."""
    W = weight.shape[0]
    w = weight.double()
    out = torch.zeros(x.shape, dtype=torch.float64)
    mag, pre, new, a = torch.zeros_like(out), torch.zeros_like(out), [], 0
    for n, win in zip(lengths, windows):
        rows = torch.cat([win.double(), x[a:a + n].double()])
        for j in range(W):
            pre[a:a + n] += rows[j:j + n] * w[j]
            mag[a:a + n] += (rows[j:j + n] * w[j]).abs()
        new.append(rows[n:])
        a += n
    if bias is not None:
        pre[:a] += bias.double()
        mag[:a] += bias.double().abs()
    out = pre * torch.sigmoid(pre) if silu else pre.clone()
    return out, new, mag, pre


def qk(x, norm, weight, eps, position, frequency, interleaved, scale):
    """(y, magnitude of the rotated pair) in float64."""
    y = x.double()
    d = y.shape[-1]
    if norm == "l2":
        y = y / torch.sqrt(y.square().sum(-1, keepdim=True) + eps)
    elif norm == "rms":
        y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / d + eps)
        if weight is not None:
            y = y * weight.double()
    mag = y.abs()
    if frequency is not None:
        half = frequency.numel()
        ang = position.double()[:, None] * frequency.double()
        c, s = ang.cos()[:, None], ang.sin()[:, None]
        i = torch.arange(half)
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b = y[..., lo].clone(), y[..., hi].clone()
        mag, y = mag.clone(), y.clone()
        y[..., lo], y[..., hi] = a * c - b * s, a * s + b * c
        mag[..., lo] = mag[..., hi] = a.abs() + b.abs()
    return y * scale, mag * abs(scale)


def compact_moves(live):
    live = [bool(x) for x in live]
    front = sum(live)
    return list(zip([i for i in range(front, len(live)) if live[i]], [i for i in range(front) if not live[i]]))


def scan(kind, q, k, v, decay, beta, lengths, initial, skip):
    """Token by token in float64.  q, k [T, G, dk], v [T, H, dv], decay [T, H]
    or [T, H, dk].  Returns out, final, and magnitudes for error bounds: out's
    and final's sums of absolute terms (additive), the largest row norm plus
    |v| seen (delta)."""
    q, k, v, decay = (x.double().numpy() for x in (q, k, v, decay))
    T, H, dv = v.shape
    G, dk = k.shape[1:]
    grp = np.arange(H) // (H // G)
    beta = np.ones((T, H)) if beta is None else beta.double().numpy()
    n = len(lengths)
    out, omag = np.zeros((T, H, dv)), np.zeros((T, H, dv))
    final, fmag = np.zeros((n, H, dv, dk)), np.zeros((n, H, dv, dk))
    big = np.zeros((n, H, dv))
    a = 0
    for i, L in enumerate(lengths):
        S = np.zeros((H, dv, dk)) if initial is None else initial[i].double().numpy().copy()
        M = np.abs(S)
        big[i] = np.linalg.norm(S, axis=-1)
        for t in range(a, a + L):
            d = decay[t][:, None, :] if decay.ndim == 3 else decay[t][:, None, None]
            kt, qt = k[t][grp], q[t][grp]
            S, M = S * d, M * d
            u = v[t]
            if kind == "delta":
                u = u - np.einsum("hvk,hk->hv", S, kt)
            u = u * beta[t][:, None]
            S = S + u[..., None] * kt[:, None]
            M = M + np.abs(u)[..., None] * np.abs(kt)[:, None]
            out[t] = np.einsum("hvk,hk->hv", S, qt)
            omag[t] = np.einsum("hvk,hk->hv", M, np.abs(qt))
            big[i] = np.maximum(big[i], np.linalg.norm(S, axis=-1) + np.abs(v[t]))
        final[i], fmag[i] = S, M
        a += L
    if skip is not None:
        s = skip.double().numpy()[:, None]
        out, omag = out + s * v, omag + np.abs(s * v)
    return out, final, omag, fmag, big
