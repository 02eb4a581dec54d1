"""Python front end of libqstate: a handle plus torch-owned device buffers.

torch provides device memory and streams only; every computation of the
decode path (dequantize, decay + update, readout, requantize) runs in the
library's kernels through the C ABI of include/qstate.h.
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional

import numpy as np

from . import _lib


@dataclasses.dataclass
class StateConfig:
    """Mirror of qstate_config with readable enumerations."""
    kind: str = "additive"          # additive | delta
    decay_mode: str = "head"        # head | key
    B: int = 1
    H: int = 1
    dk: int = 128
    dv: int = 128
    qbits: int = 8                  # 8 | 4
    hp_dtype: str = "bf16"          # fp32 | bf16 | fp16
    map_mode: str = "none"          # none | head | key
    map: Optional[np.ndarray] = None
    in_dtype: str = "bf16"          # fp32 | bf16
    rounding: str = "stochastic"    # nearest | stochastic
    sr_bits: int = 16
    bdr: bool = False
    bdr_bound: float = 0.0
    lrb_rank: int = 0
    lrb_period: int = 64
    lrb_theta: float = 0.5
    seed: int = 0
    scale_dtype: str = "fp32"       # fp32 | bf16 (bf16: with lrb_dtype bf16 and the low-rank bypass)
    lrb_dtype: str = "fp32"         # fp32 | bf16
    scale_axis: str = "value"       # value | key | head (key and head: ablations, map none, no buffer)

    def to_c(self) -> _lib.Config:
        c = _lib.Config()
        c.abi_version = _lib.ABI_VERSION
        c.kind = _lib.KIND[self.kind]
        c.decay_mode = _lib.DECAY[self.decay_mode]
        c.B, c.H, c.dk, c.dv = self.B, self.H, self.dk, self.dv
        c.qbits = self.qbits
        c.hp_dtype = _lib.DTYPE[self.hp_dtype]
        c.map_mode = _lib.MAP[self.map_mode]
        if self.map is not None:
            self._map_keep = np.ascontiguousarray(self.map, dtype=np.uint8).ravel()
            c.map = self._map_keep.ctypes.data_as(ctypes.POINTER(ctypes.c_uint8))
        c.in_dtype = _lib.DTYPE[self.in_dtype]
        c.rounding = _lib.ROUNDING[self.rounding]
        c.sr_bits = self.sr_bits
        c.bdr = int(self.bdr)
        c.bdr_bound = self.bdr_bound
        c.lrb_rank, c.lrb_period, c.lrb_theta = self.lrb_rank, self.lrb_period, self.lrb_theta
        c.seed = self.seed
        c.scale_dtype = _lib.DTYPE[self.scale_dtype]
        c.lrb_dtype = _lib.DTYPE[self.lrb_dtype]
        c.scale_axis = _lib.AXIS[self.scale_axis]
        return c


def plan(cfg: StateConfig) -> dict:
    """Buffer sizes in bytes (host only; no GPU needed)."""
    c = cfg.to_c()
    s = _lib.Sizes()
    _lib.check(_lib.lib().qstate_plan(ctypes.byref(c), ctypes.byref(s)), "qstate_plan")
    return {n: int(getattr(s, n)) for n, _ in _lib.Sizes._fields_}


def build_map(stat, groups: int, per_group: int, frac: float) -> np.ndarray:
    """Decay-based mixed-precision map: smallest decay-rate units flagged (host)."""
    stat = np.ascontiguousarray(stat, dtype=np.float32).ravel()
    assert stat.size == groups * per_group
    m = np.zeros(groups * per_group, np.uint8)
    _lib.check(_lib.lib().qstate_build_map(stat.ctypes.data, groups, per_group, frac, m.ctypes.data),
               "qstate_build_map")
    return m


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _state_dtypes(cfg: "StateConfig") -> dict:
    """torch dtype name of each state buffer (bf16 scales and factors in the bf16 layout)."""
    sd = "bfloat16" if cfg.scale_dtype == "bf16" else "float32"
    ld = "bfloat16" if cfg.lrb_dtype == "bf16" else "float32"
    return {"codes": "uint8", "scales": sd, "hp": "uint8", "lrb_W": ld, "lrb_U": ld, "lrb_n": "int32"}


_ITEM = {"uint8": 1, "bfloat16": 2, "float32": 4, "int32": 4}


_Tensor: tuple | type = ()          # torch.Tensor, once a check has imported torch


def _tensor_type() -> None:
    global _Tensor
    import torch
    _Tensor = torch.Tensor


def check_tensor(name: str, t, dtype, numel: int, device, at_least: bool = False) -> None:
    """Host-side argument check before a pointer crosses the C ABI: the kernels
    read and write exactly the planned extents, so a tensor of the wrong dtype,
    size, memory layout or device would make them read or write out of bounds
    or get wrong results.  Raises ValueError (checks in that order)."""
    if (isinstance(t, _Tensor) and t.dtype is dtype and t.device == device and t.is_contiguous()
            and (t.numel() == numel or (at_least and t.numel() > numel))):
        return
    _tensor_type()
    if not isinstance(t, _Tensor):
        raise ValueError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if (t.numel() < numel) if at_least else (t.numel() != numel):
        raise ValueError(f"{name}: {t.numel()} elements, expected {'at least ' if at_least else ''}{numel}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")


def check_states(name: str, t, dtype, shape, device) -> None:
    """States of shape [n,H,dv,dk], or with neighbouring dimensions as one: another
    order of them (keys first) has as many elements."""
    numel = shape[0] * shape[1] * shape[2] * shape[3]
    check_tensor(name, t, dtype, numel, device)
    if t.shape == shape or not numel:
        return
    inner, whole = {1}, 1
    for size in reversed(shape):
        whole *= size
        inner.add(whole)
    whole = 1
    for size in reversed(t.shape):
        whole *= size
        if whole not in inner:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def check_state(cfg: "StateConfig", sizes: dict, st: dict, device) -> None:
    """Every buffer the plan sizes > 0 must be present, typed and large enough."""
    import torch
    for n, dt in _state_dtypes(cfg).items():
        nbytes = sizes[n]
        if nbytes == 0:
            continue
        check_tensor(f"state[{n!r}]", st.get(n), getattr(torch, dt), nbytes // _ITEM[dt], device, at_least=True)


def check_inputs(cfg: "StateConfig", n: int, device, q, k, v, decay, beta, out) -> None:
    """Inputs of a step for n batch elements: q, k [n,H,dk] and v [n,H,dv] in
    the configured input dtype, decay fp32 [n,H] (or [n,H,dk] per key), beta
    fp32 [n,H] or None, out fp32 [n,H,dv]."""
    import torch
    ind = torch.bfloat16 if cfg.in_dtype == "bf16" else torch.float32
    nh = n * cfg.H
    check_tensor("q", q, ind, nh * cfg.dk, device)
    check_tensor("k", k, ind, nh * cfg.dk, device)
    check_tensor("v", v, ind, nh * cfg.dv, device)
    check_tensor("decay", decay, torch.float32, nh * (cfg.dk if cfg.decay_mode == "key" else 1), device)
    if beta is not None:
        check_tensor("beta", beta, torch.float32, nh, device)
    check_tensor("out", out, torch.float32, nh * cfg.dv, device)


def check_rows(name: str, t, dtype, shape, device) -> int:
    """A tensor of `shape` whose rows (all dimensions but the first) are
    contiguous, at any stride between them; returns that stride in elements."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.shape == shape and t.device == device:
        if t.is_contiguous():
            return t.stride(0) if shape[0] > 1 else t.numel()
    else:
        _tensor_type()
        if not isinstance(t, _Tensor):
            raise ValueError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
        if t.dtype != dtype:
            raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
        if t.shape != shape:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    st = t.stride()
    if len(st) == 3 and st[2] == 1 and st[1] == shape[2]:
        width = shape[1] * shape[2]
    else:
        width = 1
        for size, stride in zip(reversed(shape[1:]), reversed(st[1:])):
            if size != 1 and stride != width:
                raise ValueError(f"{name}: rows are not contiguous")
            width *= size
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if shape[0] <= 1:
        return width
    if st[0] < width:
        raise ValueError(f"{name}: rows overlap (stride {st[0]} of {width})")
    return st[0]


def _empty(shape, dtype, device, stream):
    """Uninitialised memory for a call on `stream` (None: the current one): taken
    on that stream, so that its reuse waits for the call."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty_like(x, contiguous: bool, stream):
    """`_empty` of x's shape, dtype and device."""
    if stream is not None:
        return _empty(x.shape, x.dtype, x.device, stream)
    if not contiguous:
        return x.new_empty(x.shape)
    import torch
    return torch.empty_like(x)


def check_stream(stream, device) -> None:
    """A stream of the tensors' device, or None."""
    if stream is not None and stream.device != device:
        raise ValueError(f"stream on {stream.device}, expected {device}")


def raw_stream(stream, device) -> int:
    """The hipStream_t of `stream`, or of the device's current stream."""
    if stream is not None:
        return stream.cuda_stream
    import torch
    return torch._C._cuda_getCurrentRawStream(device.index)


class QState:
    """A libqstate handle for one configuration on the current HIP device."""

    def __init__(self, cfg: StateConfig):
        import torch
        self.cfg = cfg
        self._c = cfg.to_c()
        self._h = ctypes.c_void_p()
        s = _lib.Sizes()
        _lib.check(_lib.lib().qstate_init(ctypes.byref(self._c), ctypes.byref(self._h), ctypes.byref(s)),
                   "qstate_init")
        self.sizes = {n: int(getattr(s, n)) for n, _ in _lib.Sizes._fields_}
        self.device = torch.device("cuda", torch.cuda.current_device())
        # the planned buffers: name, what errors call it, dtype, elements
        self._buffers = [(n, f"state[{n!r}]", getattr(torch, dt), self.sizes[n] // _ITEM[dt])
                         for n, dt in _state_dtypes(cfg).items() if self.sizes[n]]
        self._scan_bytes = {}     # workspace sizes by (tokens, sequences, key heads)

    def close(self) -> None:
        if self._h:
            _lib.lib().qstate_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def kernel_name(self) -> str:
        return _lib.lib().qstate_kernel_name(self._h).decode()

    def new_state(self) -> dict:
        """Zero-filled state buffers (the state S = 0), owned by torch."""
        import torch
        z = self.sizes
        dev = self.device

        def buf(nbytes, dtype, item):
            return torch.zeros(max(nbytes // item, 1 if nbytes else 0), dtype=dtype, device=dev)

        dts = {n: getattr(torch, d) for n, d in _state_dtypes(self.cfg).items()}
        return {n: buf(z[n], dts[n], torch.empty((), dtype=dts[n]).element_size()) for n in dts}

    @staticmethod
    def _tensors(st: dict) -> _lib.Tensors:
        t = _lib.Tensors()
        for n in ("codes", "scales", "hp", "lrb_W", "lrb_U", "lrb_n"):
            x = st.get(n)
            setattr(t, n, x.data_ptr() if (x is not None and x.numel() > 0) else None)
        return t

    @staticmethod
    def _stream(stream) -> Optional[int]:
        import torch
        if stream is None:
            stream = torch.cuda.current_stream()
        return stream.cuda_stream

    def quantize(self, S, st: dict, step: int = 0, stream=None) -> None:
        import torch
        c = self.cfg
        check_tensor("S", S, torch.float32, c.B * c.H * c.dv * c.dk, self.device)
        check_state(c, self.sizes, st, self.device)
        t = self._tensors(st)
        _lib.check(_lib.lib().qstate_quantize(self._h, _ptr(S), ctypes.byref(t), step, self._stream(stream)),
                   "qstate_quantize")

    def dequantize(self, st: dict, out=None, stream=None):
        import torch
        c = self.cfg
        if out is None:
            out = torch.empty((c.B, c.H, c.dv, c.dk), dtype=torch.float32, device=self.device)
        check_tensor("out", out, torch.float32, c.B * c.H * c.dv * c.dk, self.device)
        check_state(c, self.sizes, st, self.device)
        t = self._tensors(st)
        _lib.check(_lib.lib().qstate_dequantize(self._h, ctypes.byref(t), _ptr(out), self._stream(stream)),
                   "qstate_dequantize")
        return out

    def step(self, st: dict, q, k, v, decay, beta=None, out=None, step: int = 0, stream=None):
        """One decode step in place on `st`; returns o [B,H,dv] fp32."""
        import torch
        c = self.cfg
        if out is None:
            out = torch.empty((c.B, c.H, c.dv), dtype=torch.float32, device=self.device)
        check_inputs(c, c.B, self.device, q, k, v, decay, beta, out)
        check_state(c, self.sizes, st, self.device)
        t = self._tensors(st)
        inp = _lib.Inputs(_ptr(q), _ptr(k), _ptr(v), _ptr(decay), _ptr(beta))
        _lib.check(_lib.lib().qstate_decode_step(self._h, ctypes.byref(t), ctypes.byref(inp), _ptr(out), step,
                                                 self._stream(stream)), "qstate_decode_step")
        return out

    def step_batch(self, pool: dict, slot, step, q, k, v, decay, beta=None, out=None, stream=None):
        """One decode step for n = len(slot) sequences whose states sit in the
        slots `slot` (int32 [n], device) of `pool` (this handle's B slots),
        each with its own step (uint64 stored as int64 [n], device); inputs
        [n,H,...]; returns o [n,H,dv] fp32."""
        import torch
        c = self.cfg
        n = int(slot.numel())
        if slot.dtype != torch.int32 or step.dtype not in (torch.int64, torch.uint64) or step.numel() != n:
            raise ValueError("slot must be int32 [n] and step 64-bit [n]")
        check_tensor("slot", slot, torch.int32, n, self.device)
        check_tensor("step", step, step.dtype, n, self.device)
        if out is None:
            out = torch.empty((n, c.H, c.dv), dtype=torch.float32, device=self.device)
        check_inputs(c, n, self.device, q, k, v, decay, beta, out)
        check_state(c, self.sizes, pool, self.device)
        t = self._tensors(pool)
        inp = _lib.Inputs(_ptr(q), _ptr(k), _ptr(v), _ptr(decay), _ptr(beta))
        _lib.check(_lib.lib().qstate_decode_step_batch(self._h, ctypes.byref(t), ctypes.byref(inp), _ptr(out), n,
                                                       _ptr(slot), _ptr(step), self._stream(stream)),
                   "qstate_decode_step_batch")
        return out

    def scan(self, q, k, v, decay, beta=None, *, offsets=None, initial=None, final=None, skip=None, out=None,
             stream=None):
        """Run packed prompts through the recurrence: (out, final).

        q, k [T,G,dk] and v [T,H,dv] in the configured input dtype (heads
        h*G//H .. share a query and key head), decay fp32 [T,H] (or [T,H,dk]),
        beta fp32 [T,H] or None; each may be a slice of a wider tensor whose
        trailing dimensions are contiguous.  offsets int32 [n+1] on the device:
        sequence i is tokens offsets[i]..offsets[i+1]-1 (None: one sequence);
        tokens outside every sequence are left as they were in `out`.
        initial fp32 [n,H,dv,dk] or None (zeros); skip fp32 [H] adds skip[h] v
        to the output.  out [T,H,dv] in the input dtype; final fp32
        [n,H,dv,dk] is what `quantize` takes, and may be `initial` itself."""
        import torch
        c = self.cfg
        dev = self.device
        check_stream(stream, dev)
        ind = torch.bfloat16 if c.in_dtype == "bf16" else torch.float32
        if not isinstance(v, torch.Tensor) or v.dim() != 3 or not isinstance(k, torch.Tensor) or k.dim() != 3:
            raise ValueError("k and v must be [T, heads, dim] tensors")
        T, G = v.shape[0], k.shape[1]
        n = 1
        if offsets is not None:
            if not isinstance(offsets, torch.Tensor) or offsets.numel() < 1:
                raise ValueError("offsets must be an int32 tensor [n+1]")
            n = offsets.numel() - 1
            check_tensor("offsets", offsets, torch.int32, n + 1, dev)
        H, dk, dv, f32 = c.H, c.dk, c.dv, torch.float32
        qs = check_rows("q", q, ind, (T, G, dk), dev)
        ks = check_rows("k", k, ind, (T, G, dk), dev)
        vs = check_rows("v", v, ind, (T, H, dv), dev)
        ds = check_rows("decay", decay, f32, (T, H, dk) if c.decay_mode == "key" else (T, H), dev)
        bs = 0 if beta is None else check_rows("beta", beta, f32, (T, H), dev)
        if skip is not None:
            check_tensor("skip", skip, f32, H, dev)
        if initial is not None:
            check_states("initial", initial, f32, (n, H, dv, dk), dev)
        if out is None:
            out = _empty_like(v, vs == H * dv, stream)
            os = H * dv
        else:
            os = check_rows("out", out, ind, (T, H, dv), dev)
        if final is None:
            final = _empty((n, H, dv, dk), f32, dev, stream)
        else:
            check_states("final", final, f32, (n, H, dv, dk), dev)
        a = _lib.Scan(q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(), _ptr(beta), _ptr(skip),
                      _ptr(initial), final.data_ptr(), out.data_ptr(), _ptr(offsets), qs, ks, vs, ds, bs, os, T, n, G)
        L = _lib.lib()
        need = self._scan_bytes.get((T, n, G))
        if need is None:
            z = ctypes.c_uint64()
            _lib.check(L.qstate_scan_workspace(self._h, ctypes.byref(a), ctypes.byref(z)), "qstate_scan_workspace")
            if len(self._scan_bytes) >= 4096:
                self._scan_bytes.clear()
            need = self._scan_bytes[T, n, G] = z.value
        # the call's own: a captured call keeps it in its graph's memory
        ws = _empty((need,), torch.uint8, dev, stream) if need else None
        _lib.check(L.qstate_scan(self._h, ctypes.byref(a), _ptr(ws), need, raw_stream(stream, dev)), "qstate_scan")
        return out, final

    def _checked(self, st: dict, slots: int) -> _lib.Tensors:
        """The buffers of a state of `slots` slots, checked, as the C ABI takes them."""
        B, t = self.cfg.B, _lib.Tensors()
        for name, label, dtype, numel in self._buffers:
            x = st.get(name)
            check_tensor(label, x, dtype, numel if slots == B else numel // B * slots, self.device, at_least=True)
            setattr(t, name, x.data_ptr())
        return t

    def _extra(self, extra, source_extra, src_slots: int):
        """Per-slot buffers that go along: tensors [slots, ...], contiguous, on this device."""
        import torch
        src = list(extra if source_extra is None else source_extra)
        dst = list(extra)
        if len(src) != len(dst) or len(dst) > _lib.MAX_EXTRA:
            raise ValueError(f"{len(dst)} extra buffers and {len(src)} of the source (at most {_lib.MAX_EXTRA})")
        bufs = (_lib.SlotBuffer * max(1, len(dst)))()
        for i, (s, d) in enumerate(zip(src, dst)):
            for t, slots in ((d, self.cfg.B), (s, src_slots)):
                if not isinstance(t, torch.Tensor) or t.dim() < 1 or t.shape[0] < slots or not t.is_contiguous():
                    raise ValueError(f"extra[{i}]: expected a contiguous tensor of at least {slots} slots")
                if t.device != self.device:
                    raise ValueError(f"extra[{i}]: on {t.device}, expected {self.device}")
            if s.dtype != d.dtype or s.shape[1:] != d.shape[1:]:
                raise ValueError(f"extra[{i}]: {s.dtype} {tuple(s.shape[1:])} into {d.dtype} {tuple(d.shape[1:])}")
            bufs[i] = _lib.SlotBuffer(s.data_ptr(), d.data_ptr(), d.element_size() * d[0].numel() if d.shape[0] else 0)
        return bufs, len(dst)

    def copy_slots(self, pool: dict, src_slot, dst_slot, *, source=None, source_slots=None, extra=(),
                   source_extra=None, stream=None) -> None:
        """Slot dst_slot[i] of `pool` becomes slot src_slot[i] of `source` (a
        state of `source_slots` slots of this configuration; None: the pool
        itself), or the zero state when src_slot[i] is -1.  src_slot, dst_slot:
        int32 [n] on the device; elements out of range are skipped.  Forks,
        moves, clears and hand-overs between pools in one launch.
        Destinations must be distinct and, within one pool, must not be
        another element's source.  extra: up to 6 more tensors [B, ...] that
        go along (source_extra: theirs in the source)."""
        import torch
        check_stream(stream, self.device)
        n = int(src_slot.numel())
        check_tensor("src_slot", src_slot, torch.int32, n, self.device)
        check_tensor("dst_slot", dst_slot, torch.int32, n, self.device)
        if source is None:
            if source_slots is not None or source_extra is not None:
                raise ValueError("source_slots and source_extra go with a source")
            source, m = pool, self.cfg.B
        else:
            if source_slots is None:
                raise ValueError("source_slots: the source's number of slots")
            if extra and source_extra is None and source is not pool:
                raise ValueError("extra buffers of another pool need source_extra")
            m = int(source_slots)
        d = self._checked(pool, self.cfg.B)
        s = d if source is pool and m == self.cfg.B else self._checked(source, m)
        bufs, ne = self._extra(extra, source_extra, m) if extra or source_extra else (None, 0)
        _lib.check(_lib.lib().qstate_copy_slots(self._h, ctypes.byref(d), ctypes.byref(s), m, n, _ptr(src_slot),
                                                _ptr(dst_slot), bufs, ne, raw_stream(stream, self.device)),
                   "qstate_copy_slots")

    def compact_slots(self, pool: dict, live, *, extra=(), where=None, stream=None):
        """Move the live slots of `pool` (live: uint8 or bool [B], device) to
        its front: with F of them, the i-th live slot at or behind F goes to
        the i-th free slot before F.  Returns where int32 [B]: the slot each
        slot's state is in now, -1 for free ones.  extra: further tensors
        [B, ...] that go along."""
        import torch
        c = self.cfg
        check_stream(stream, self.device)
        if isinstance(live, torch.Tensor) and live.dtype == torch.bool:
            live = live.view(torch.uint8)
        check_tensor("live", live, torch.uint8, c.B, self.device)
        if where is None:
            where = _empty((c.B,), torch.int32, self.device, stream)
        check_tensor("where", where, torch.int32, c.B, self.device)
        t = self._checked(pool, c.B)
        bufs, ne = self._extra(extra, None, c.B) if extra else (None, 0)
        _lib.check(_lib.lib().qstate_compact_slots(self._h, ctypes.byref(t), _ptr(live), _ptr(where), bufs, ne,
                                                   raw_stream(stream, self.device)), "qstate_compact_slots")
        return where
