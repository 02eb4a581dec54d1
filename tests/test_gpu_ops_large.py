"""Calls of the operators that need 2^32 threads or more in all: the runtime
takes a launch's threads modulo 2^32."""
import sys

import pytest
import torch

from quantized_recurrent_state_qstate_amd import QState, StateConfig, causal_conv, causal_conv_step, qk_norm_rotate

pytestmark = pytest.mark.gpu
DEV = "cuda"


def say(*a):
    print("[large]", *a, file=sys.stderr, flush=True)


def room(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of free GPU memory")


@pytest.mark.parametrize("T", [2 ** 24 - 1, 2 ** 24, 2 ** 24 + 5])
def test_norm_and_rotation_of_many_tokens(T):
    say("qk", T)
    room(4)
    q = torch.ones(T, 1, 16, dtype=torch.bfloat16, device=DEV)
    k = torch.ones(T, 1, 16, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(T, dtype=torch.int32, device=DEV)
    pos[-1] = 1                                          # the last token turns
    freq = torch.full((8,), 0.5, dtype=torch.float64, device=DEV)
    q_out, k_out = qk_norm_rotate(q, k, norm="none", position=pos, frequency=freq, q_scale=2.0,
                                  q_out=torch.zeros_like(q), k_out=torch.zeros_like(k))
    torch.cuda.synchronize()
    assert (q_out[:-1] == 2).all() and (k_out[:-1] == 1).all()
    want, _ = qk_norm_rotate(q[-1:], None, norm="none", position=pos[-1:], frequency=freq, q_scale=2.0)
    assert torch.equal(q_out[-1:], want) and (want != 2).all()


@pytest.mark.parametrize("slots", [True, False])
def test_convolution_of_many_sequences(slots):
    n, C = 2 ** 24 + 3, 8
    say("conv", n)
    room(8)
    x = torch.ones(n, C, dtype=torch.bfloat16, device=DEV)
    x[-1] = 3
    w = torch.ones(3, C, device=DEV)
    window = torch.ones(n, 2, C, dtype=torch.bfloat16, device=DEV)
    slot = torch.arange(n - 1, -1, -1, dtype=torch.int32, device=DEV) if slots else None
    off = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    out = causal_conv(x, w, offsets=off, window=window, slot=slot, silu=False, out=torch.zeros_like(x))
    torch.cuda.synchronize()
    assert (out[:-1] == 3).all() and (out[-1] == 5).all()
    last = 0 if slots else n - 1
    assert (window[last, 1] == 3).all() and (window[last, 0] == 1).all()
    window[last, 1] = 1
    assert (window == 1).all()


def test_convolution_step_of_many_sequences():
    n, C = 2 ** 26 + 7, 8
    say("step", n)
    room(16)
    x = torch.ones(n, C, dtype=torch.bfloat16, device=DEV)
    window = torch.ones(n, 1, C, dtype=torch.bfloat16, device=DEV)
    out = causal_conv_step(x, torch.ones(2, C, device=DEV), window=window, silu=False, out=torch.zeros_like(x))
    torch.cuda.synchronize()
    assert (out == 2).all()


def test_copies_of_many_slots():
    B = 2 ** 23 + 3                                      # two pieces a slot
    say("slots", B)
    room(4)
    qs = QState(StateConfig(B=B, H=1, dk=64, dv=1))
    st = qs.new_state()
    st["codes"].fill_(7)
    src = torch.full((B,), -1, dtype=torch.int32, device=DEV)
    dst = torch.arange(B, dtype=torch.int32, device=DEV)
    dst[0] = B                                           # out of range: slot 0 stays
    qs.copy_slots(st, src, dst)
    torch.cuda.synchronize()
    codes = st["codes"].view(B, -1)
    assert (codes[0] == 7).all() and not codes[1:].any()
    qs.close()
