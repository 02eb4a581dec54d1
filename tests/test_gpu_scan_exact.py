"""How exact the prompt scans are, against the recurrence in float64.

u = 2^-24.  The scans compute in fp32 and round an output once.  Rounding
errors are taken as independent, each at most u of a value about as large as
the result: a result behind N roundings is off by u sqrt(N / 3) of its size in
the mean square, and the tests allow u sqrt(N), 1.7 times that.  N:
a state's entry has 2 (decay, sum) for each token that is not forgotten, of
which there are n = max_t sum_j prod_{j<i<=t} d_i, and by the delta rule as
many again for S k and beta (v - S k), whose sums over dk channels have dk
roundings more of a row's length / sqrt(dk), which counts as 1; plus 16 for
the joins of chunks and segments.  An output has the sum over dk channels and
64 tokens of a chunk more.

A bf16 output hides what comes before its rounding, but where the terms cancel:
an output below 2^-13 of its head's size is rounded by at most 2^-8 2^-13 of
that size, 2^-21 (times 1 / sqrt 3 in the mean square, as they are spread
evenly below the border), less than a 16-bit operand's 2^-17 by far.
"""
import sys

import numpy as np
import pytest
import torch

from quantized_recurrent_state_qstate_amd import QState, StateConfig

DEV = "cuda"
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
KINDS = [("additive", "head"), ("additive", "key"), ("delta", "head"), ("delta", "key")]


def inputs(kind, decay, T, H, G, dk, dv, dtype, seed, mu):
    g = torch.Generator().manual_seed(seed)
    q, k, v = torch.randn(T, G, dk, generator=g), torch.randn(T, G, dk, generator=g), torch.randn(T, H, dv, generator=g)
    if kind == "delta":
        k = 0.99 * k / k.norm(dim=-1, keepdim=True)
    d = torch.sigmoid(torch.randn((T, H, dk) if decay == "key" else (T, H), generator=g) + mu)
    b = torch.sigmoid(torch.randn(T, H, generator=g))
    return q.to(DT[dtype]), k.to(DT[dtype]), v.to(DT[dtype]), d, b


def remembered(d, lengths):
    """n: the largest number of tokens that a state remembers."""
    most, a = 0.0, 0
    for L in lengths:
        r = torch.zeros_like(d[0], dtype=torch.float64)
        for t in range(a, a + L):
            r = r * d[t].double() + 1
            most = max(most, float(r.max()))
        a += L
    return most


def roundings(kind, dk, n):
    """(of a state's entry, of an output)"""
    s = (4 if kind == "delta" else 2) * n + 16
    return s, s + dk + 64


def bound(N):
    """Of the mean square of what passed N roundings, relative to its size."""
    return U * N ** 0.5


def reference(kind, q, k, v, d, b, lengths, S0):
    """Token by token in float64, elementwise."""
    q, k, v, d, b = (x.double() for x in (q, k, v, d, b))
    H, group = v.shape[1], torch.arange(v.shape[1], device=q.device) // (v.shape[1] // q.shape[1])
    out, final, a = torch.zeros_like(v), [], 0
    for i, L in enumerate(lengths):
        S = S0[i].double().clone()
        for t in range(a, a + L):
            kt, qt = k[t][group][:, None], q[t][group][:, None]
            S *= d[t][:, None] if d.dim() == 3 else d[t][:, None, None]
            u = v[t] - (S * kt).sum(-1) if kind == "delta" else v[t]
            S += (u * b[t][:, None])[..., None] * kt
            out[t] = (S * qt).sum(-1)
        final.append(S)
        a += L
    return out, torch.stack(final)


def state_error(got, want):
    """The error of every head's state, of its size."""
    e, w = (got.double() - want).flatten(2).norm(dim=2), want.flatten(2).norm(dim=2)
    return float((e / w.clamp(min=1e-300)).max())


def scan(kind, decay, lengths, H, G, dk, dv, dtype, mu, seed=0):
    print("[exact]", kind, decay, lengths, H, G, dk, dv, dtype, mu, file=sys.stderr, flush=True)
    q, k, v, d, b = (x.to(DEV) for x in inputs(kind, decay, sum(lengths), H, G, dk, dv, dtype, seed, mu))
    S0 = torch.randn(len(lengths), H, dv, dk, generator=torch.Generator().manual_seed(seed + 1)).to(DEV)
    off = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=DEV)
    qs = QState(StateConfig(kind=kind, decay_mode=decay, B=len(lengths), H=H, dk=dk, dv=dv, in_dtype=dtype))
    out, final = qs.scan(q, k, v, d, b, offsets=off, initial=S0)
    torch.cuda.synchronize()
    want, wfin = reference(kind, q, k, v, d, b, lengths, S0)
    qs.close()
    return out, final, want, wfin, roundings(kind, dk, remembered(d.cpu(), lengths))


@pytest.mark.gpu
@pytest.mark.parametrize("kind,decay", KINDS)
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 128), (256, 64)])
def test_bf16_outputs_that_cancel(kind, decay, dk, dv):
    out, final, want, wfin, (ns, no) = scan(kind, decay, [1024, 333], 8, 4, dk, dv, "bf16", 2.0)
    assert state_error(final, wfin) <= bound(ns)
    size = want.square().mean(-1, keepdim=True).sqrt().expand_as(want)
    err, tol = (out.double() - want).abs() / size, bound(no)
    near = (want.abs() < 2.0 ** -13 * size)
    assert near.sum() >= 30
    rms = float(err[near].square().mean().sqrt())
    print(f"[exact] {int(near.sum())} outputs, off by {rms:.2e} of {tol + 2 ** -21 / 3 ** 0.5:.2e}", file=sys.stderr)
    assert rms <= tol + 2.0 ** -21 / 3 ** 0.5
    # all of them: half a step, and six times the mean square's bound
    assert (err <= 2.0 ** -8 * want.abs() / size + 6 * tol).all()


LONG = [(kind, decay, "bf16", lengths, H, dk, dv)
        for kind, decay in (("delta", "head"), ("additive", "head"), ("additive", "key"))
        for lengths in ([1537], [1024, 1025], [3, 1100, 0, 2600], [1600, 1600, 1600], [63, 4097, 1, 1024])
        for dk, dv, H in ((64, 64, 4), (128, 33, 2), (256, 24, 2))]
LONG += [(kind, decay, dtype, lengths, H, dk, dv)
         for kind, decay, dtype in (("delta", "key", "bf16"), ("delta", "head", "fp32"), ("delta", "key", "fp32"),
                                    ("additive", "head", "fp32"), ("additive", "key", "fp32"))
         for lengths in ([193], [3, 150, 0, 400], [15, 1513, 1, 128])
         for dk, dv, H in ((64, 64, 4), (128, 33, 2), (256, 24, 2))]


@pytest.mark.gpu
@pytest.mark.parametrize("mu", [2.0, 5.0])
@pytest.mark.parametrize("kind,decay,dtype,lengths,H,dk,dv", LONG)
def test_long_sequences(kind, decay, dtype, lengths, H, dk, dv, mu):
    """Segments, pieces and joins: states to fp32's own error, outputs to that and half a step."""
    out, final, want, wfin, (ns, no) = scan(kind, decay, lengths, H, 2, dk, dv, dtype, mu)
    worst = state_error(final, wfin)
    print(f"[exact] states off by {worst:.2e} of {bound(ns):.2e}", file=sys.stderr)
    assert worst <= bound(ns)
    size = want.square().mean(-1, keepdim=True).sqrt()
    half = 2.0 ** -8 if dtype == "bf16" else U
    assert ((out.double() - want).abs() <= half * want.abs() + 6 * bound(no) * size).all()


@pytest.mark.parametrize("mu", [2.0, 5.0])
@pytest.mark.parametrize("kind,decay,dtype,lengths,H,dk,dv", LONG)
def test_the_tolerances_tell(kind, decay, dtype, lengths, H, dk, dv, mu):
    """A state of 16 bits, as from one bf16 piece too few, is refused at each of these sizes; a result of zeros too."""
    *_, d, _ = inputs(kind, decay, sum(lengths), H, 2, dk, 1, dtype, 0, mu)
    ns, no = roundings(kind, dk, remembered(d, lengths))
    S = torch.randn(len(lengths), H, dv, dk, generator=torch.Generator().manual_seed(7))
    hi = S.bfloat16().float()
    cut = hi + (S - hi).bfloat16().float()
    assert state_error(cut, S.double()) > bound(ns)
    assert state_error(torch.zeros_like(S), S.double()) > 1e4 * bound(ns)
    assert 2.0 ** -8 + 6 * bound(no) < 0.01      # zeros for outputs are off by all of them
