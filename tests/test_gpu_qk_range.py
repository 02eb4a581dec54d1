"""The norm of queries and keys of very small heads, against the formula in float64.

Tolerance: a sum of d squares and its root is off by at most (d / 2 + 4) u of
itself (u = 2^-24: d roundings of the sum, one of the squares, halved by the
root; the root, the reciprocal, the products), then half a step of the type.
"""
import sys

import pytest
import torch

import ops_ref
from quantized_recurrent_state_qstate_amd import qk_norm_rotate

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("norm", ["l2", "rms"])
@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-38, 1e-30, 1e-24, 1e-20, 1e-6])
@pytest.mark.parametrize("scale", [1.0, 1e-12, 1e-15, 1e-17, 1e-19, 1e-25, 1e-37, 1e-41])
def test_qk_norm_of_tiny_values(dtype, norm, eps, scale):
    """Squares that are subnormal or zero in fp32."""
    print("[qk]", dtype, norm, eps, scale, file=sys.stderr, flush=True)
    d = 72
    x = (torch.randn(5, 3, d, generator=torch.Generator().manual_seed(3)) * scale).to(dtype)
    x[2, 1, 1:] = 0                                      # one channel alone
    x[2, 1, 0] = scale
    out, _ = qk_norm_rotate(x.cuda(), norm=norm, eps=eps)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    want, _ = ops_ref.qk(x, norm, None, eps, None, None, False, 1.0)
    out = out.cpu().double()
    # a result below the normal numbers is off by half a subnormal step (2^-150; bf16 2^-134)
    half = 2.0 ** -150 if dtype is torch.float32 else 2.0 ** -134
    tol = ((d / 2 + 4) * U + ops_ref.half_step(dtype)) * want.abs() + half
    zero = (x == 0).all(-1, keepdim=True).expand_as(out) & (eps == 0)    # 1e-41 is zero in bf16: 0 / 0
    assert torch.isnan(out[zero]).all() and torch.isfinite(out[~zero]).all()
    assert ((out - want).abs() <= tol)[~zero].all()
