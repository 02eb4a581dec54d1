"""The convolution, the norm and rotation of queries and keys, and the slot
copies on the GPU, against their definitions in float64.

Tolerances count roundings: u = 2^-24 for an fp32 operation, half a step of
the output type for the last one.
"""
import sys

import numpy as np
import pytest
import torch

import ops_ref
from quantized_recurrent_state_qstate_amd import QState, StateConfig, causal_conv, causal_conv_step, qk_norm_rotate

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def say(*a):
    print("[ops]", *a, file=sys.stderr, flush=True)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def offsets(lengths, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(lengths)]), dtype=torch.int32, device=DEV)


def wide(x, pad, dtype):
    """x as a slice of a tensor with `pad` more columns on each side."""
    T, C = x.shape
    big = torch.full((T, C + 2 * pad), 7.0, dtype=dtype, device=DEV)
    big[:, pad:pad + C] = x.to(DEV)
    return big[:, pad:pad + C]


# ------------------------------------------------------------------ convolution
def conv_tol(ref, pre, mag, W, dtype, silu):
    # W fused products and the bias: at most W + 1 roundings of partial sums no larger than mag; |act'| < 1.1.
    # act: e^-y from an argument rounded at |y| log2(e) u, one ulp each for exp2 and the reciprocal, a sum and a
    # product: (|y| + 4) 2^-23 of the value; below e^-88 the result is flushed to (minus) zero.
    tol = 1.1 * (W + 1) * U * mag + half_step_of(dtype) * ref.abs()
    if silu:
        tol = tol + (pre.abs() + 4) * 2 * U * ref.abs() + 1e-35
    return tol


def half_step_of(dtype):
    return ops_ref.half_step(dtype)


CONV = [
    # lengths, C, W, dtype, window, bias, silu
    ([1], 64, 4, "bf16", True, True, True),
    ([5], 37, 4, "bf16", True, True, True),
    ([0], 64, 4, "fp32", True, False, True),
    ([1, 2, 3, 0, 4, 1], 64, 4, "fp32", True, True, True),
    ([16, 17, 15, 1, 0, 0, 33], 72, 4, "bf16", True, True, True),
    ([16, 17, 15, 1, 0, 0, 33], 72, 3, "bf16", False, True, False),
    ([130, 2, 64], 515, 2, "fp32", True, False, True),
    ([63, 65], 2304, 4, "bf16", True, True, True),
    ([100], 520, 4, "bf16", False, False, True),
    ([3] * 90 + [0] * 40 + [7] * 3, 24, 4, "fp32", True, True, True),
]


@pytest.mark.parametrize("case", CONV, ids=lambda c: f"{len(c[0])}x{sum(c[0])}_{c[1]}_{c[2]}_{c[3]}")
@pytest.mark.parametrize("strided", [False, True])
def test_conv_prompts(case, strided):
    lengths, C, W, dt, with_window, with_bias, silu = case
    say("conv", case, strided)
    dtype, g, T = DT[dt], gen(1), sum(lengths)
    first, behind, n = (2, 3, len(lengths)) if strided else (0, 0, len(lengths))
    x = torch.randn(T, C, generator=g).to(dtype)
    w, b = torch.randn(W, C, generator=g), torch.randn(C, generator=g) if with_bias else None
    slots = n + 3
    slot = torch.randperm(slots, generator=g)[:n].to(torch.int32)
    win = torch.randn(slots, W - 1, C, generator=g).to(dtype)
    rows = torch.cat([torch.full((first, C), 9.0), x.float(), torch.full((behind, C), 9.0)]).to(dtype)
    xd = wide(rows, 5 if C % 8 else 8, dtype) if strided else rows.to(DEV)
    out = torch.full((first + T + behind, C), -3.0, dtype=dtype, device=DEV)
    if strided:
        out = wide(out, 16, dtype)
    wind = win.to(DEV)
    kw = dict(window=wind, slot=slot.to(DEV)) if with_window else {}
    got = causal_conv(xd, w.to(DEV), None if b is None else b.to(DEV), offsets=offsets(lengths, first), silu=silu,
                      out=out, **kw)
    assert got is out
    torch.cuda.synchronize()
    before = [win[slot[i]] if with_window else torch.zeros(W - 1, C) for i in range(n)]
    ref, new, mag, pre = ops_ref.conv(x, w, b, lengths, before, silu)
    o = out.cpu().double()
    err = (o[first:first + T] - ref).abs()
    assert (err <= conv_tol(ref, pre, mag, W, dtype, silu)).all(), f"worst {err.max()}"
    assert (o[:first] == -3).all() and (o[first + T:] == -3).all(), "rows outside the sequences were written"
    want = win.clone()
    if with_window:
        for i in range(n):
            want[slot[i]] = new[i].to(dtype)
    assert torch.equal(wind.cpu(), want), "windows"


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("C,n,W", [(64, 1, 4), (37, 3, 4), (2304, 8, 4), (520, 5, 2), (72, 4, 3)])
def test_conv_step(dt, C, n, W):
    say("conv step", dt, C, n, W)
    dtype, g = DT[dt], gen(2)
    x, w, b = torch.randn(n, C, generator=g).to(dtype), torch.randn(W, C, generator=g), torch.randn(C, generator=g)
    win = torch.randn(n + 2, W - 1, C, generator=g).to(dtype)
    slot = torch.randperm(n + 2, generator=g)[:n].to(torch.int32)
    wind = win.to(DEV)
    out = causal_conv_step(x.to(DEV), w.to(DEV), b.to(DEV), window=wind, slot=slot.to(DEV))
    torch.cuda.synchronize()
    ref, new, mag, pre = ops_ref.conv(x, w, b, [1] * n, [win[i] for i in slot], True)
    assert ((out.cpu().double() - ref).abs() <= conv_tol(ref, pre, mag, W, dtype, True)).all()
    for i in range(n):
        win[slot[i]] = new[i].to(dtype)
    assert torch.equal(wind.cpu(), win)


def test_conv_skips_slots_out_of_range():
    g, C = gen(3), 40
    x, w = torch.randn(30, C, generator=g).to(DEV), torch.randn(4, C, generator=g).to(DEV)
    win = torch.randn(3, 3, C, generator=g).to(DEV)
    keep = win.clone()
    slot = torch.tensor([1, -1, 3], dtype=torch.int32, device=DEV)
    out = torch.full((30, C), -3.0, device=DEV)
    causal_conv(x, w, offsets=offsets([10, 10, 10]), window=win, slot=slot, out=out)
    one = torch.full((3, C), -3.0, device=DEV)
    causal_conv_step(x[:3], w, window=win, slot=torch.tensor([7, -5, 3], dtype=torch.int32, device=DEV), out=one)
    torch.cuda.synchronize()
    assert (out[10:] == -3).all() and (out[:10] != -3).any()
    assert torch.equal(win[[0, 2]], keep[[0, 2]]) and torch.equal(win[1], x[7:10])
    assert (one == -3).all()


def test_conv_prompt_then_tokens_is_one_prompt():
    """A prompt in two calls and then token by token is the prompt in one call."""
    g, C, T = gen(4), 96, 41
    x = torch.randn(T, C, generator=g).to(torch.bfloat16).to(DEV)
    w, b = torch.randn(4, C, generator=g).to(DEV), torch.randn(C, generator=g).to(DEV)
    win = torch.zeros(2, 3, C, dtype=torch.bfloat16, device=DEV)
    one = causal_conv(x, w, b, offsets=offsets([T]))
    slot = torch.tensor([1], dtype=torch.int32, device=DEV)
    parts = [causal_conv(x[:2], w, b, offsets=offsets([2]), window=win, slot=slot),
             causal_conv(x[2:35], w, b, offsets=offsets([33]), window=win, slot=slot)]
    parts += [causal_conv_step(x[t:t + 1], w, b, window=win, slot=slot) for t in range(35, T)]
    assert torch.equal(torch.cat(parts), one) and torch.equal(win[1], x[-3:]) and not win[0].any()


# ------------------------------------------------------------------ norm and rotation
QK = [
    # T, Hq, Hk, d, rot, norm, weight, interleaved, far
    (1, 1, 1, 8, 0, "l2", False, False, 0),
    (3, 4, 2, 64, 64, "rms", True, False, 1 << 20),
    (17, 32, 32, 128, 128, "rms", True, False, 262144),
    (17, 6, 3, 128, 64, "l2", False, True, 1 << 20),
    (2, 3, 1, 72, 48, "rms", False, False, 4096),
    (5, 2, 2, 72, 64, "none", False, True, 100000),
    (600, 3, 2, 256, 256, "l2", False, False, 1 << 20),
    (4, 5, 0, 512, 512, "rms", True, False, 5000),
    (4, 70, 3, 264, 32, "l2", False, True, 5000),
]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("case", QK, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("form", ["plain", "strided", "inplace"])
def test_qk_norm_rotate(case, dt, form):
    T, hq, hk, d, rot, norm, weight, inter, far = case
    say("qk", case, dt, form)
    dtype, g = DT[dt], gen(5)
    rows = torch.randn(T, (hq + hk) * d, generator=g) * 3
    rows[0, :d] = 0                                     # a head of zeros stays zeros
    rows = rows.to(dtype)
    both = wide(rows, 16, dtype) if form == "strided" else rows.to(DEV)
    q, k = both[:, :hq * d].unflatten(1, (hq, d)), both[:, hq * d:].unflatten(1, (hk, d)) if hk else None
    qw, kw = (torch.randn(d, generator=g), torch.randn(d, generator=g)) if weight else (None, None)
    pos = freq = None
    if rot:
        pos = torch.randint(far // 2, far, (T,), generator=g, dtype=torch.int32)
        pos[-1] = -3
        freq = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    dev = lambda x: None if x is None else x.to(DEV)
    kwargs = dict(q_out=q, k_out=k) if form == "inplace" else {}
    qo, ko = qk_norm_rotate(q, k, norm=norm, q_weight=dev(qw), k_weight=dev(kw), eps=1e-6, position=dev(pos),
                            frequency=dev(freq), interleaved=inter, q_scale=0.25, **kwargs)
    torch.cuda.synchronize()
    cq, ck = rows[:, :hq * d].unflatten(1, (hq, d)), rows[:, hq * d:].unflatten(1, (hk, d)) if hk else None
    for name, got, x, w, scale in (("q", qo, cq, qw, 0.25), ("k", ko, ck, kw, 1.0)):
        if x is None:
            assert got is None
            continue
        ref, mag = ops_ref.qk(x, norm, w, 1e-6, pos, freq, inter, scale)
        # the sum of squares: 8 in a lane and 6 joins, all positive: 14 u, halved by the root; root, division,
        # weight, scale: 4 u; rotation: the turn as fp32 is half an ulp of 1/2 off (2 pi 2^-25 rad < 4 u), sine
        # and cosine 2 ulp (4 u), two products and a sum (3 u): 22 u of |a| + |b|
        tol = 24 * U * mag + half_step_of(dtype) * ref.abs() + 1e-38
        err = (got.cpu().double() - ref).abs()
        assert (err <= tol).all(), f"{name}: worst {(err / tol).max():.2f} of its tolerance"


# ------------------------------------------------------------------ slots
POOLS = {
    "int8": dict(H=3, dk=64, dv=40, qbits=8),
    "int8_heads_bf16": dict(H=4, dk=128, dv=64, qbits=8, map_mode="head", hp_dtype="bf16"),
    "int8_keys_fp16": dict(H=2, dk=64, dv=7, qbits=8, map_mode="key", hp_dtype="fp16"),
    "int4_buffer": dict(H=3, dk=64, dv=33, qbits=4, rounding="nearest", lrb_rank=5),
    "int4_buffer_bf16": dict(H=3, dk=64, dv=33, qbits=4, rounding="nearest", lrb_rank=3, scale_dtype="bf16",
                             lrb_dtype="bf16"),
    "big": dict(H=8, dk=128, dv=128, qbits=8),
}


def pool_of(name, B):
    kw = dict(POOLS[name])
    r = np.random.default_rng(9)
    if kw.get("map_mode") == "head":
        kw["map"] = (np.arange(kw["H"]) % 2).astype(np.uint8)
    elif kw.get("map_mode") == "key":
        kw["map"] = (r.random((kw["H"], kw["dk"])) < 0.2).astype(np.uint8)
    return QState(StateConfig(B=B, **kw))


def fill(st, seed):
    r = np.random.default_rng(seed)
    for x in st.values():
        if x.numel():
            b = x.view(torch.uint8).view(-1)
            b.copy_(torch.from_numpy(r.integers(0, 256, b.numel(), dtype=np.uint8)))
    return st


def slot_rows(st, B):
    """Every buffer as bytes [B, bytes per slot] on the CPU."""
    return {k: x.view(torch.uint8).view(B, -1).cpu().clone() for k, x in st.items() if x.numel()}


@pytest.mark.parametrize("name", list(POOLS))
def test_copy_slots_within_a_pool(name):
    say("copy", name)
    B = 9
    qs = pool_of(name, B)
    st = fill(qs.new_state(), 1)
    extra = torch.arange(B * 3 * 37, device=DEV, dtype=torch.int32).to(torch.bfloat16).view(B, 3, 37)
    want, wx = slot_rows(st, B), extra.cpu().clone()
    moves = [(2, 5), (2, 0), (-1, 7), (4, 4), (3, 9), (9, 1), (-2, 1), (3, -1), (8, 6)]
    src, dst = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in zip(*moves))
    qs.copy_slots(st, src, dst, extra=[extra])
    torch.cuda.synchronize()
    for a, b in [(2, 5), (2, 0), (-1, 7), (8, 6)]:
        for x in want.values():
            x[b] = x[a] if a >= 0 else 0
        wx[b] = wx[a] if a >= 0 else 0
    got = slot_rows(st, B)
    for k in want:
        assert torch.equal(got[k], want[k]), k
    assert torch.equal(extra.cpu(), wx)
    qs.copy_slots(st, src[:0], dst[:0])
    assert all(torch.equal(slot_rows(st, B)[k], want[k]) for k in want)
    qs.close()


@pytest.mark.parametrize("name", ["int8_heads_bf16", "int4_buffer_bf16"])
def test_copy_slots_between_pools(name):
    small, big = pool_of(name, 2), pool_of(name, 6)
    a, b = fill(small.new_state(), 2), fill(big.new_state(), 3)
    want, have = slot_rows(b, 6), slot_rows(a, 2)
    src = torch.tensor([1, 0, 1, 2], dtype=torch.int32, device=DEV)
    dst = torch.tensor([0, 5, 1, 2], dtype=torch.int32, device=DEV)
    big.copy_slots(b, src, dst, source=a, source_slots=2)
    torch.cuda.synchronize()
    got = slot_rows(b, 6)
    for k in want:
        want[k][0], want[k][5], want[k][1] = have[k][1], have[k][0], have[k][1]
        assert torch.equal(got[k], want[k]), k
    with pytest.raises(ValueError, match="codes"):      # the source is smaller than said
        big.copy_slots(b, src, dst, source=a, source_slots=3)
    small.close(), big.close()


@pytest.mark.parametrize("B,frac", [(1, 0.0), (1, 1.0), (2, 0.5), (5, 0.4), (70, 0.5), (70, 0.0), (70, 1.0), (300, 0.1),
                                    (300, 0.9), (700, 0.5)])
def test_compact_slots(B, frac):
    say("compact", B, frac)
    qs = pool_of("int8_keys_fp16", B)
    st = fill(qs.new_state(), 4)
    extra = torch.randn(B, 11, device=DEV)
    live = torch.rand(B, generator=gen(B)) < frac
    want, wx = slot_rows(st, B), extra.cpu().clone()
    where = qs.compact_slots(st, live.to(DEV), extra=[extra])
    torch.cuda.synchronize()
    at = [i if x else -1 for i, x in enumerate(live.tolist())]
    for a, b in ops_ref.compact_moves(live.tolist()):
        at[a] = b
        for x in list(want.values()) + [wx]:
            x[b] = x[a]
    assert where.cpu().tolist() == at
    got = slot_rows(st, B)
    for k in want:
        assert torch.equal(got[k], want[k]), k
    assert torch.equal(extra.cpu(), wx)
    qs.close()
