"""Batches of many short sequences with a few long ones, which go in launches of
their own: every sequence as if it were scanned by itself.

Both ways are the recurrence in fp32 with one rounding of the output, so they
differ by at most twice what test_gpu_scan_exact.py allows either of them (six
times its mean square for a single value), and a step of the output's type.
"""
import sys

import numpy as np
import pytest
import torch

from quantized_recurrent_state_qstate_amd import QState, StateConfig
from test_gpu_scan_exact import DT, KINDS, bound, inputs, remembered, roundings

pytestmark = pytest.mark.gpu
DEV = "cuda"
LENGTHS = {
    "one prompt": [1] * 120 + [1200] + [1] * 80,
    "the ends": [300] + [1, 0, 2, 63, 64, 65, 3] * 12 + [800],
    "around cells": [5, 59, 64, 1, 127, 0, 0, 65, 9] + [1] * 90 + [500, 64, 64, 1, 1, 1] + [2] * 60,
    "none": [7, 1, 0, 13] * 60,
}


@pytest.mark.parametrize("name", LENGTHS)
@pytest.mark.parametrize("kind,decay", KINDS)
@pytest.mark.parametrize("dtype,H,dk,dv", [("bf16", 4, 64, 64), ("bf16", 4, 128, 24), ("fp32", 2, 64, 40)])
def test_each_sequence_as_by_itself(name, kind, decay, dtype, H, dk, dv):
    lengths = LENGTHS[name]
    n, T, first = len(lengths), sum(lengths), 2
    print("[mixed]", name, kind, decay, dtype, H, dk, dv, n, T, file=sys.stderr, flush=True)
    q, k, v, d, b = inputs(kind, decay, T + 5, H, 2, dk, dv, dtype, 3, 3.0)
    ns, no = roundings(kind, dk, remembered(d, [T + 5]))
    q, k, v, d, b = (x.to(DEV) for x in (q, k, v, d, b))
    S0 = torch.randn(n, H, dv, dk, device=DEV)
    start = first + np.concatenate([[0], np.cumsum(lengths)])
    qs = QState(StateConfig(kind=kind, decay_mode=decay, B=n, H=H, dk=dk, dv=dv, in_dtype=dtype))
    out = torch.full((T + 5, H, dv), -3.0, dtype=DT[dtype], device=DEV)
    final = S0.clone()
    qs.scan(q, k, v, d, b, offsets=torch.tensor(start, dtype=torch.int32, device=DEV), initial=final, final=final,
            out=out)
    torch.cuda.synchronize()
    assert (out[:first] == -3).all() and (out[first + T:] == -3).all()
    for i, L in enumerate(lengths):
        if L == 0:
            assert torch.equal(final[i], S0[i])
            continue
        s = slice(int(start[i]), int(start[i + 1]))
        o, f = qs.scan(q[s], k[s], v[s], d[s], b[s], initial=S0[i:i + 1])
        size = o.float().square().mean(-1, keepdim=True).sqrt()
        tol = 2 * 6 * bound(no) * size + torch.finfo(DT[dtype]).eps * o.float().abs()
        assert ((out[s].float() - o.float()).abs() <= tol).all(), f"sequence {i} of {L}"
        assert (final[i] - f[0]).norm() <= 2 * bound(ns) * f.norm(), f"state {i} of {L}"
    qs.close()
