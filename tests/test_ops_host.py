"""Refusals of the operators around the decode step (no GPU): the C ABI's
argument checks, which end before any HIP call, and the binding's."""
import ctypes

import pytest
import torch

from quantized_recurrent_state_qstate_amd import QState, StateConfig, _lib, causal_conv, causal_conv_step, plan, qk_norm_rotate
from quantized_recurrent_state_qstate_amd.api import _ITEM, _state_dtypes, check_rows

A = 1 << 20        # an address that is never read: every call here is refused first


def conv(**kw):
    c = _lib.Conv(x=A, out=2 * A, weight=3 * A, bias=None, window=4 * A, slot=5 * A, offsets=6 * A, x_stride=64,
                  out_stride=64, dtype=1, tokens=100, channels=64, width=4, n=2, slots=4, silu=1)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CONV = [
    (dict(dtype=2), _lib.QS_EUNSUPPORTED), (dict(dtype=9), _lib.QS_EINVAL),
    (dict(width=1), _lib.QS_EUNSUPPORTED), (dict(width=5), _lib.QS_EUNSUPPORTED),
    (dict(channels=0), _lib.QS_EINVAL), (dict(n=-1), _lib.QS_EINVAL), (dict(slots=-1), _lib.QS_EINVAL),
    (dict(tokens=-1), _lib.QS_EINVAL), (dict(silu=2), _lib.QS_EINVAL),
    (dict(x=None), _lib.QS_EINVAL), (dict(out=None), _lib.QS_EINVAL), (dict(weight=None), _lib.QS_EINVAL),
    (dict(offsets=None), _lib.QS_EINVAL), (dict(x=A + 1), _lib.QS_EINVAL), (dict(weight=3 * A + 2), _lib.QS_EINVAL),
    (dict(x_stride=63), _lib.QS_EINVAL), (dict(out_stride=0), _lib.QS_EINVAL), (dict(x_stride=-64), _lib.QS_EINVAL),
    (dict(out=A), _lib.QS_EINVAL), (dict(out=A + 64), _lib.QS_EINVAL), (dict(window=A), _lib.QS_EINVAL),
    (dict(slot=None, n=5), _lib.QS_EINVAL), (dict(x_stride=1 << 61), _lib.QS_EINVAL),
    (dict(tokens=2 ** 31 - 1, channels=2 ** 20, x_stride=2 ** 20, out_stride=2 ** 20, out=A + (1 << 56),
          window=None),
     _lib.QS_EUNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD_CONV)
def test_conv_refusals(kw, code):
    L = _lib.lib()
    assert L.qstate_causal_conv(ctypes.byref(conv(**kw)), None) == code
    assert L.qstate_last_error().decode() != ""
    if not {"tokens", "offsets"} & set(kw) and "out_stride" not in kw and kw.get("x") != A + 1:
        assert L.qstate_causal_conv_step(ctypes.byref(conv(**kw)), None) == code


def test_conv_null_empty_and_step_needs_windows():
    L = _lib.lib()
    assert L.qstate_causal_conv(None, None) == _lib.QS_EINVAL
    assert L.qstate_causal_conv_step(None, None) == _lib.QS_EINVAL
    assert L.qstate_causal_conv_step(ctypes.byref(conv(window=None)), None) == _lib.QS_EINVAL
    assert L.qstate_causal_conv(ctypes.byref(conv(n=0)), None) == _lib.QS_OK
    assert L.qstate_causal_conv(ctypes.byref(conv(tokens=0)), None) == _lib.QS_OK
    assert L.qstate_causal_conv_step(ctypes.byref(conv(n=0)), None) == _lib.QS_OK


def qk(**kw):
    c = _lib.Qk(q=A, k=2 * A, q_out=3 * A, k_out=4 * A, position=5 * A, frequency=6 * A, q_stride=256, k_stride=128,
                q_out_stride=256, k_out_stride=128, dtype=1, tokens=10, q_heads=4, k_heads=2, dim=64, rot=64, norm=1,
                interleaved=0, eps=1e-6, q_scale=1.0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_QK = [
    (dict(dtype=2), _lib.QS_EUNSUPPORTED), (dict(dim=60), _lib.QS_EUNSUPPORTED), (dict(dim=520), _lib.QS_EUNSUPPORTED),
    (dict(dim=0), _lib.QS_EINVAL), (dict(rot=8), _lib.QS_EUNSUPPORTED), (dict(rot=80), _lib.QS_EINVAL),
    (dict(rot=-16), _lib.QS_EINVAL), (dict(norm=3), _lib.QS_EINVAL), (dict(q_weight=7 * A), _lib.QS_EINVAL),
    (dict(interleaved=2), _lib.QS_EINVAL), (dict(eps=-1.0), _lib.QS_EINVAL), (dict(eps=float("nan")), _lib.QS_EINVAL),
    (dict(q_scale=float("inf")), _lib.QS_EINVAL), (dict(tokens=-1), _lib.QS_EINVAL),
    (dict(q_heads=0, k_heads=0), _lib.QS_EINVAL), (dict(q_heads=-1), _lib.QS_EINVAL),
    (dict(position=None), _lib.QS_EINVAL), (dict(frequency=None), _lib.QS_EINVAL), (dict(q=None), _lib.QS_EINVAL),
    (dict(k_out=None), _lib.QS_EINVAL), (dict(q=A + 8), _lib.QS_EINVAL), (dict(q_stride=255), _lib.QS_EINVAL),
    (dict(k_stride=132), _lib.QS_EINVAL), (dict(norm=2, k_weight=7 * A + 4), _lib.QS_EINVAL),
    (dict(q_out=A, q_out_stride=264), _lib.QS_EINVAL), (dict(k_out=3 * A), _lib.QS_EINVAL),
    (dict(k_out=A), _lib.QS_EINVAL),
]


@pytest.mark.parametrize("kw,code", BAD_QK)
def test_qk_refusals(kw, code):
    assert _lib.lib().qstate_qk_norm_rotate(ctypes.byref(qk(**kw)), None) == code
    assert _lib.lib().qstate_last_error().decode() != ""


def test_qk_null_and_empty():
    assert _lib.lib().qstate_qk_norm_rotate(None, None) == _lib.QS_EINVAL
    assert _lib.lib().qstate_qk_norm_rotate(ctypes.byref(qk(tokens=0)), None) == _lib.QS_OK


def test_handle_calls_refuse_null_handles():
    L = _lib.lib()
    a, n = _lib.Scan(), ctypes.c_uint64()
    assert L.qstate_scan(None, ctypes.byref(a), None, 0, None) == _lib.QS_EINVAL
    assert L.qstate_scan_workspace(None, ctypes.byref(a), ctypes.byref(n)) == _lib.QS_EINVAL
    assert L.qstate_scan_workspace(None, ctypes.byref(a), None) == _lib.QS_EINVAL
    assert L.qstate_copy_slots(None, None, None, 0, 0, None, None, None, 0, None) == _lib.QS_EINVAL
    assert L.qstate_compact_slots(None, None, None, None, None, 0, None) == _lib.QS_EINVAL


def test_binding_checks():
    """Shapes, types, strides and devices are refused before a pointer reaches the library."""
    x, w, win = torch.zeros(10, 32), torch.zeros(4, 32), torch.zeros(3, 3, 32)
    off, slot = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    ok = dict(offsets=off, window=win, slot=slot)
    for args, kw, msg in [
        ((x, w), ok, "expected a GPU"),
        ((x.half(), w), ok, "x: dtype"),
        ((x.t(), w), ok, "x: rows are not contiguous"),
        ((x[0].expand(10, 32), w), ok, "x: rows overlap"),
        ((x, w.bfloat16()), ok, "weight: dtype"),
        ((x, w[:, :31].contiguous()), ok, "weight: 124 elements"),
        ((x, w, torch.zeros(31)), ok, "bias: 31 elements"),
        ((x, w), dict(ok, window=win.bfloat16()), "window: dtype"),
        ((x, w), dict(ok, window=win[:, :2].contiguous()), "window: 192 elements"),
        ((x, w), dict(ok, slot=slot.long()), "slot: dtype"),
        ((x, w), dict(ok, slot=slot[:1]), "slot: 1 elements"),
        ((x, w), dict(ok, offsets=off.long()), "offsets: dtype"),
        ((x, w), dict(ok, offsets=off[:0]), "offsets must be"),
        ((x, w), dict(ok, out=torch.zeros(9, 32)), "out: shape"),
    ]:
        with pytest.raises(ValueError, match=msg):
            causal_conv(*args, **kw)
    with pytest.raises(ValueError, match="window"):
        causal_conv_step(x, w, window=None)
    with pytest.raises(ValueError, match="slot: 2 elements, expected 10"):
        causal_conv_step(x, w, window=win, slot=slot)
    q, k = torch.zeros(5, 4, 64), torch.zeros(5, 2, 64)
    pos, freq = torch.zeros(5, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    for args, kw, msg in [
        ((q, k), {}, "expected a GPU"),
        ((q, k.bfloat16()), {}, "k: dtype"),
        ((q, k[:4]), {}, "k: shape"),
        ((q.transpose(1, 2), k), {}, "rows are not contiguous"),
        ((q, k), dict(norm="max"), "norm 'max'"),
        ((q, k), dict(position=pos), "go together"),
        ((q, k), dict(position=pos.long(), frequency=freq), "position: dtype"),
        ((q, k), dict(position=pos, frequency=freq.float()), "frequency: dtype"),
        ((q, k), dict(norm="rms", q_weight=torch.zeros(63)), "q_weight: 63 elements"),
        ((q,), dict(k_out=k), "k_out without k"),
    ]:
        with pytest.raises(ValueError, match=msg):
            qk_norm_rotate(*args, **kw)
    assert check_rows("x", torch.zeros(4, 10)[:, 2:6], torch.float32, (4, 4), torch.device("cpu")) == 10
    assert check_rows("x", torch.zeros(1, 10)[:, 2:6], torch.float32, (1, 4), torch.device("cpu")) == 4


def test_handle_calls_host_code_under_sanitizers(tmp_path):
    """The scan's, copy's and compaction's argument checks, plans and workspaces, with stand-ins for HIP."""
    import os
    import shutil

    from test_sanitizers import HERE, ROOT, SAN, _run
    gxx, inc = shutil.which("g++"), "/opt/rocm/include"
    if not gxx or not os.path.exists(os.path.join(inc, "hip", "hip_runtime_api.h")):
        pytest.skip("g++ or the HIP headers not available")
    csrc = os.path.join(ROOT, "quantized_recurrent_state_qstate_amd", "csrc")
    exe = str(tmp_path / "ops_driver")
    out = _run([gxx, "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I", inc, "-I", os.path.join(ROOT, "include"),
                "-I", csrc, os.path.join(csrc, "qstate_host.cpp"), os.path.join(csrc, "qstate_ops_host.cpp"),
                os.path.join(HERE, "ops_driver.cpp"), "-o", exe], exe)
    assert "0 failed checks" in out, out


def handle(**kw):
    """A QState without a device: its checks of arguments, on CPU tensors, end before the library is called."""
    qs = QState.__new__(QState)
    qs.cfg, qs.device, qs._h = StateConfig(**kw), torch.device("cpu"), ctypes.c_void_p()
    qs.sizes, qs._scan_bytes = plan(qs.cfg), {}
    qs._buffers = [(n, f"state[{n!r}]", getattr(torch, dt), qs.sizes[n] // _ITEM[dt])
                   for n, dt in _state_dtypes(qs.cfg).items() if qs.sizes[n]]
    return qs


@pytest.mark.parametrize("m", [3, 1 << 20])
def test_the_pool_as_its_own_source_has_no_more_slots(m):
    qs = handle(B=2, H=2, dk=64, dv=16)
    pool = qs.new_state()
    idx = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="state\\['codes'\\]: .* expected at least"):
        qs.copy_slots(pool, idx, idx, source=pool, source_slots=m)


def test_windows_and_states_of_another_layout_are_refused():
    """The right number of elements in the wrong order of dimensions."""
    x, w = torch.zeros(10, 32), torch.zeros(4, 32)
    off, slot = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for window in (torch.zeros(3, 32, 3), torch.zeros(3, 3, 16, 2), torch.zeros(3, 96), torch.zeros(3, 1, 96)):
        with pytest.raises(ValueError, match="window"):
            causal_conv(x, w, offsets=off, window=window, slot=slot)
        with pytest.raises(ValueError, match="window"):
            causal_conv_step(x[:2], w, window=window, slot=slot)
    with pytest.raises(ValueError, match="expected a GPU"):       # nothing else was wrong
        causal_conv(x, w, offsets=off, window=torch.zeros(3, 3, 32), slot=slot)
    for bad in (torch.zeros(32, 4), torch.zeros(128), torch.zeros(4, 32, 1)):
        with pytest.raises(ValueError, match="weight"):
            causal_conv(x, bad, offsets=off)
    qs = handle(kind="delta", B=2, H=4, dk=64, dv=32)
    T, bf = 6, torch.bfloat16
    args = dict(q=torch.zeros(T, 2, 64, dtype=bf), k=torch.zeros(T, 2, 64, dtype=bf), v=torch.zeros(T, 4, 32, dtype=bf),
                decay=torch.zeros(T, 4), offsets=off)
    for name in ("initial", "final"):
        for shape in ((2, 4, 64, 32), (4, 2, 32, 64), (2, 32, 4, 64), (8, 64, 32), (2, 64, 4, 32), (64, 256)):
            with pytest.raises(ValueError, match=f"{name}: shape"):
                qs.scan(**args, **{name: torch.zeros(shape)})
        for shape in ((2, 4, 32, 64), (8, 32, 64), (2, 4, 2048), (2 * 4 * 32 * 64,), (1, 2, 4, 32, 64)):
            with pytest.raises(_lib.QStateError, match="handle is NULL"):    # as far as the library
                qs.scan(**args, **{name: torch.zeros(shape)})


def test_streams_of_another_device_are_refused():
    """A stream is checked before anything is taken on it."""
    from types import SimpleNamespace
    other = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    qs = handle(B=2, H=4, dk=64, dv=32)
    T, bf = 6, torch.bfloat16
    idx, pool = torch.zeros(1, dtype=torch.int32), qs.new_state()
    for call in (lambda: qs.scan(torch.zeros(T, 2, 64, dtype=bf), torch.zeros(T, 2, 64, dtype=bf),
                                 torch.zeros(T, 4, 32, dtype=bf), torch.zeros(T, 4), stream=other),
                 lambda: qs.copy_slots(pool, idx, idx, stream=other),
                 lambda: qs.compact_slots(pool, torch.zeros(2, dtype=torch.uint8), stream=other),
                 lambda: causal_conv(torch.zeros(T, 32), torch.zeros(4, 32), offsets=idx, stream=other),
                 lambda: qk_norm_rotate(torch.zeros(T, 2, 64), stream=other)):
        with pytest.raises(ValueError, match="stream on cuda:1, expected cpu"):
            call()
