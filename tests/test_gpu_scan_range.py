"""Scans of values far from one: what the recurrence, token by token in fp32,
keeps finite comes out finite and right, whichever way the scan takes.

Tolerances: fp32 throughout, u = 2^-24; a result is a sum of terms each behind
at most 2 roundings a token, dk + 80 more in chunks (see test_gpu_scan.py), of
the sum of their absolute values; then half a step of the output's type.
"""
import sys

import numpy as np
import pytest
import torch

import ops_ref
from quantized_recurrent_state_qstate_amd import QState, StateConfig

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
KINDS = [("additive", "head"), ("additive", "key"), ("delta", "head"), ("delta", "key")]


def make(kind, decay, T, H, G, dk, dv, dtype, seed=0, mu=3.0):
    g = torch.Generator().manual_seed(seed)
    q, k, v = torch.randn(T, G, dk, generator=g), torch.randn(T, G, dk, generator=g), torch.randn(T, H, dv, generator=g)
    k = k / k.norm(dim=-1, keepdim=True)
    d = torch.sigmoid(torch.randn((T, H, dk) if decay == "key" else (T, H), generator=g) + mu)
    b = torch.sigmoid(torch.randn(T, H, generator=g)) * 0.99
    return dict(q=q.to(DT[dtype]), k=k.to(DT[dtype]), v=v.to(DT[dtype]), decay=d, beta=b)


def scan(kind, decay, dtype, a, lengths=None, initial=None, G=None):
    T, H, dv = a["v"].shape
    dk, n = a["k"].shape[2], len(lengths or [T])
    print("[range]", kind, decay, dtype, T, H, dk, dv, lengths, file=sys.stderr, flush=True)
    qs = QState(StateConfig(kind=kind, decay_mode=decay, B=n, H=H, dk=dk, dv=dv, in_dtype=dtype))
    off = None if lengths is None else torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32,
                                                    device=DEV)
    out, final = qs.scan(*(a[x].to(DEV) for x in ("q", "k", "v", "decay", "beta")), offsets=off,
                         initial=None if initial is None else initial.to(DEV))
    torch.cuda.synchronize()
    qs.close()
    return out.cpu().double(), final.cpu().double()


def right(kind, dtype, a, out, final, lengths=None, initial=None):
    """out and final against the recurrence; by the delta rule the errors of S k come back into the state: each token
    adds at most (dk + 16) u of the largest row so far."""
    T, dk = a["k"].shape[0], a["k"].shape[2]
    with np.errstate(over="ignore"):
        o, f, omag, fmag, big = ops_ref.scan(kind, *(a[x] for x in ("q", "k", "v", "decay", "beta")), lengths or [T],
                                             initial, None)
    n = 2 * max(lengths or [T]) + dk + 80
    otol, ftol = n * U * omag, n * U * fmag
    if kind == "delta":
        otol, ftol = otol * (dk + 16), ftol * (dk + 16)
    assert torch.isfinite(out).all() and torch.isfinite(final).all()
    assert (np.abs(out.numpy() - o) <= otol + ops_ref.half_step(DT[dtype]) * np.abs(o) + 1e-38).all()
    assert (np.abs(final.numpy() - f) <= ftol + 1e-38).all()


def test_scan_large_key_behind_small_decays():
    """Additive, a decay a channel: beta k divided by sixteen tokens' decays leaves fp32, the result does not."""
    a = make("additive", "key", 64, 2, 2, 64, 32, "bf16")
    a["decay"][16:32] = 2.0 ** -6
    a["k"][31] = 2.0 ** 32
    a["beta"][31] = 1.0
    a["decay"][32:] = 1.0
    right("additive", "bf16", a, *scan("additive", "key", "bf16", a))


def test_scan_small_query_behind_small_decays():
    """... and q times them vanishes, while the keys divided by them are large."""
    a = make("additive", "key", 64, 2, 2, 64, 32, "bf16")
    a["decay"][16:32] = 2.0 ** -6
    a["decay"][32:] = 1.0
    a["q"][16:32] *= 2.0 ** -44
    right("additive", "bf16", a, *scan("additive", "key", "bf16", a))


@pytest.mark.parametrize("kind,decay", KINDS)
@pytest.mark.parametrize("T", [150, 2600])
def test_scan_overflowing_product_does_not_reach_earlier_tokens(kind, decay, T):
    """A finite key whose product with the state is not: outputs before it stay as they are."""
    bad = T // 2 + 5
    a = make(kind, decay, T, 2, 2, 64, 48, "bf16")
    S0 = torch.randn(1, 2, 48, 64) * 8
    clean, _ = scan(kind, decay, "bf16", a, initial=S0)
    a["k"][bad, 0] = 3e38
    a["q"][bad:] *= 1e-3
    out, _ = scan(kind, decay, "bf16", a, initial=S0)
    assert torch.isfinite(out[:bad]).all() and torch.allclose(out[:bad], clean[:bad], rtol=2 ** -7, atol=1e-3)
    assert torch.isfinite(out[:, 1]).all()


def test_scan_overflowing_sum_before_its_decay():
    """Additive, a decay a head: S q leaves fp32, 2^c S q does not."""
    a = make("additive", "head", 128, 2, 2, 64, 32, "bf16")
    S0 = torch.randn(1, 2, 32, 64) * 2.0 ** 70
    a["q"][40] *= 2.0 ** 60
    a["decay"][:40] = 0.125
    right("additive", "bf16", a, *scan("additive", "head", "bf16", a, initial=S0), initial=S0)


@pytest.mark.parametrize("kind,decay", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scan_growing_decays_of_nothing(kind, decay, dtype):
    """Decays above one whose product leaves fp32, while the state is still zero."""
    a = make(kind, decay, 130, 2, 1, 64, 48, dtype)
    for t in (0, 64):
        a["decay"][t:t + 6] = 1e30
    a["v"][:70] = 0
    right(kind, dtype, a, *scan(kind, decay, dtype, a))


@pytest.mark.parametrize("kind,decay", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scan_growing_decays_of_little(kind, decay, dtype):
    """... or so small that the product with it is not large."""
    a = make(kind, decay, 130, 2, 1, 64, 48, dtype)
    a["decay"][20:24] = 2.0 ** 33
    a["v"][:24] *= 2.0 ** -100
    a["v"][24:30] = 0
    a["decay"][24:30] = 2.0 ** -6
    right(kind, dtype, a, *scan(kind, decay, dtype, a))


@pytest.mark.parametrize("kind,decay", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lengths", [[4096], [100, 3000, 0, 996]])
def test_scan_growing_decays_over_segments(kind, decay, dtype, lengths):
    """Whole segments and pieces whose decays leave fp32, with a state of zero before and in them, then ordinary
    tokens; one head of the two is ordinary throughout."""
    T = sum(lengths)
    a = make(kind, decay, T, 2, 1, 64, 48, dtype, mu=5.0)
    quiet = slice(100, 2600)
    a["decay"][quiet, 0] = 8.0
    a["v"][quiet, 0] = 0
    if len(lengths) == 1:
        a["v"][:100, 0] = 0
    right(kind, dtype, a, *scan(kind, decay, dtype, a, lengths), lengths=lengths)
