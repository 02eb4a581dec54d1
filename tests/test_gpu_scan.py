"""The scan of prompts on the GPU against the recurrence in float64, token by
token, and a whole serving run: convolution, norm, scan, hand-over into a
pool's slots, decode.

Tolerances count roundings (u = 2^-24).  Additive recurrences: the scan sums
terms u_j k_j e^{...} q, each with its decay; whatever the order, a term
passes at most 2 roundings a token (decay, sum) and, in a chunked order, a
handful more; so the error is at most (2 t + dk + 16) u times the sum of the
terms' absolute values.  For bf16 inputs the products may take an operand as
a sum of two bf16 numbers: 2^-17 each, at most two such operands: 2^-16 of
that sum more for the output, none for the state.  Delta rule: with unit keys,
beta <= 1 and decays <= 1 a step does not enlarge a row's error, and adds at
most (dk + 16) u of the row's norm plus |v|.  Last, half a step of the output.
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
    print("[scan]", *a, file=sys.stderr, flush=True)


def offsets(lengths, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(lengths)]), dtype=torch.int32, device=DEV)


def inputs(kind, decay, lengths, H, G, dk, dv, dtype, seed=0, mu=3.0, beta=True):
    g = torch.Generator().manual_seed(seed)
    T = sum(lengths)
    q = torch.randn(T, G, dk, generator=g) * dk ** -0.5
    k = torch.randn(T, G, dk, generator=g)
    k = k / k.norm(dim=-1, keepdim=True)
    v = torch.randn(T, H, dv, generator=g)
    d = torch.sigmoid(torch.randn((T, H, dk) if decay == "key" else (T, H), generator=g) + mu)
    b = torch.sigmoid(torch.randn(T, H, generator=g)) if beta else None
    q, k, v = (x.to(DT[dtype]) for x in (q, k, v))
    if kind == "delta":                                 # rounding may push a key above length one
        b = b * 0.99
    return q, k, v, d, b


def check(kind, dtype, lengths, dk, out, final, ref):
    o, f, omag, fmag, big = ref
    t = np.concatenate([np.arange(1, L + 1) for L in lengths] + [np.zeros(0)])[:, None, None]
    n = np.array(lengths)[:, None, None, None]
    half = ops_ref.half_step(DT[dtype])
    split = 2.0 ** -16 if dtype == "bf16" else 0.0
    if kind == "additive":
        otol, ftol = ((2 * t + dk + 16) * U + split) * omag, (2 * n + 16) * U * fmag
    else:
        seq = np.repeat(np.arange(len(lengths)), lengths)
        otol = ((t + 1) * (dk + 16) * U + split) * (big[seq] + 1) + 4 * U * omag
        ftol = (n + 1) * (dk + 16) * U * (big[..., None] + 1)
    oerr, ferr = np.abs(out.cpu().double().numpy() - o), np.abs(final.cpu().double().numpy() - f)
    assert (oerr <= otol + half * np.abs(o)).all(), \
        f"out: {(oerr / (otol + half * np.abs(o) + 1e-300)).max():.2f} of its tolerance"
    assert (ferr <= ftol + 1e-38).all(), f"final: {(ferr / (ftol + 1e-38)).max():.2f} of its tolerance"


def run(kind, decay, lengths, H, G, dk, dv, dtype, initial=False, skip=False, strided=False, mu=3.0, beta=True,
        seed=0):
    say(kind, decay, lengths, H, G, dk, dv, dtype, initial, skip, strided)
    q, k, v, d, b = inputs(kind, decay, lengths, H, G, dk, dv, dtype, seed, mu, beta)
    n, T = len(lengths), sum(lengths)
    g = torch.Generator().manual_seed(seed + 1)
    S0 = torch.randn(n, H, dv, dk, generator=g) * 0.5 if initial else None
    sk = torch.randn(H, generator=g) if skip else None
    first = 3 if strided else 0
    qs = QState(StateConfig(kind=kind, decay_mode=decay, B=max(n, 1), H=H, dk=dk, dv=dv, in_dtype=dtype))
    dev = lambda x: None if x is None else x.to(DEV)
    if strided:                                         # slices of one wide tensor, rows before and behind
        pad = lambda x: torch.cat([torch.full((first, *x.shape[1:]), 5.0).to(x.dtype), x,
                                   torch.full((4, *x.shape[1:]), 5.0).to(x.dtype)])
        qw, kw, vw = H * dv + 8, H * dv + 8 + G * dk, 0
        big = torch.zeros(T + 7, H * dv + 8 + 2 * G * dk, dtype=DT[dtype], device=DEV)
        big[:, qw:qw + G * dk], big[:, kw:kw + G * dk] = dev(pad(q).flatten(1)), dev(pad(k).flatten(1))
        big[:, :H * dv] = dev(pad(v).flatten(1))
        qd, kd = big[:, qw:qw + G * dk].unflatten(1, (G, dk)), big[:, kw:kw + G * dk].unflatten(1, (G, dk))
        vd = big[:, :H * dv].unflatten(1, (H, dv))
        gates = torch.zeros(T + 7, 3 * H, device=DEV)
        if b is not None:
            gates[:, H:2 * H] = dev(pad(b))
        if decay == "head":
            gates[:, :H] = dev(pad(d))
        bd = gates[:, H:2 * H] if b is not None else None
        dd = gates[:, :H] if decay == "head" else dev(pad(d))
        out = torch.full((T + 7, H, dv), -3.0, dtype=DT[dtype], device=DEV)
        final = dev(S0) if initial else None            # in place
        out, final = qs.scan(qd, kd, vd, dd, bd, offsets=offsets(lengths, first), initial=final, final=final,
                             skip=dev(sk), out=out)
        torch.cuda.synchronize()
        assert (out[:first] == -3).all() and (out[first + T:] == -3).all(), "rows outside the sequences were written"
        out = out[first:first + T]
    else:
        out, final = qs.scan(dev(q), dev(k), dev(v), dev(d), dev(b), offsets=offsets(lengths), initial=dev(S0),
                             skip=dev(sk))
        torch.cuda.synchronize()
    check(kind, dtype, lengths, dk, out, final, ops_ref.scan(kind, q, k, v, d, b, lengths, S0, sk))
    qs.close()


KINDS = [("additive", "head"), ("additive", "key"), ("delta", "head"), ("delta", "key")]


@pytest.mark.parametrize("kind,decay", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (256, 33), (64, 1), (128, 200)])
def test_scan_sizes(kind, decay, dtype, dk, dv):
    run(kind, decay, [1, 0, 16, 17, 70], 2, 1, dk, dv, dtype, initial=True, skip=dv != 33)


@pytest.mark.parametrize("kind,decay", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lengths", [[1], [0], [64], [65], [129, 63, 128], [300], [5] * 20, [0, 0, 200, 0]])
def test_scan_lengths(kind, decay, dtype, lengths):
    run(kind, decay, lengths, 4, 2, 64, 64, dtype)


@pytest.mark.parametrize("kind,decay", KINDS)
@pytest.mark.parametrize("dtype,dv", [("bf16", 64), ("bf16", 31), ("fp32", 64), ("fp32", 5)])
def test_scan_strided_in_place_and_rows_outside(kind, decay, dtype, dv):
    run(kind, decay, [33, 0, 130], 4, 4, 128, dv, dtype, initial=True, skip=True, strided=True)


@pytest.mark.parametrize("kind,decay", KINDS)
@pytest.mark.parametrize("mu", [-6.0, 0.0, 9.0])
def test_scan_fast_and_slow_decays(kind, decay, mu):
    run(kind, decay, [200, 65], 2, 2, 128, 64, "bf16", initial=True, mu=mu)


@pytest.mark.parametrize("kind,decay", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scan_zero_decays_forget_everything(kind, decay, dtype):
    """A decay of zero (a document's end) cuts the past off exactly: what follows equals a scan that starts there."""
    q, k, v, d, b = inputs(kind, decay, [150], 2, 1, 64, 48, dtype)
    cut = 70
    d[cut] = 0.0
    d[20:23] = 0.0
    qs = QState(StateConfig(kind=kind, decay_mode=decay, B=1, H=2, dk=64, dv=48, in_dtype=dtype))
    S0 = torch.randn(1, 2, 48, 64)
    out, final = qs.scan(*(x.to(DEV) for x in (q, k, v, d, b)), initial=S0.to(DEV))
    torch.cuda.synchronize()
    check(kind, dtype, [150], 64, out, final, ops_ref.scan(kind, q, k, v, d, b, [150], S0, None))
    ref = ops_ref.scan(kind, q[cut:], k[cut:], v[cut:], d[cut:], b[cut:], [150 - cut], None, None)
    check(kind, dtype, [150 - cut], 64, out[cut:], final, ref)
    qs.close()


@pytest.mark.parametrize("kind,decay", KINDS)
def test_scan_in_two_calls_is_one_scan(kind, decay):
    """Chunked prefill: the state handed from one call to the next."""
    dk, dv, H, T = 128, 64, 4, 200
    q, k, v, d, b = (x.to(DEV) for x in inputs(kind, decay, [T], H, 2, dk, dv, "bf16"))
    qs = QState(StateConfig(kind=kind, decay_mode=decay, B=1, H=H, dk=dk, dv=dv))
    a = 77
    o1, S = qs.scan(q[:a], k[:a], v[:a], d[:a], b[:a])
    o2, S = qs.scan(q[a:], k[a:], v[a:], d[a:], b[a:], initial=S, final=S)
    torch.cuda.synchronize()
    ref = ops_ref.scan(kind, *(x.cpu() for x in (q, k, v, d, b)), [T], None, None)
    check(kind, "bf16", [T], dk, torch.cat([o1, o2]), S, ref)
    qs.close()


@pytest.mark.parametrize("kind,decay", KINDS)
def test_scan_is_the_decode_step_many_times(kind, decay):
    """With fp32 storage (every head protected) the decode step is the same recurrence, token by token."""
    H, dk, dv, T = 2, 64, 64, 20
    q, k, v, d, b = (x.to(DEV) for x in inputs(kind, decay, [T], H, H, dk, dv, "bf16"))
    qs = QState(StateConfig(kind=kind, decay_mode=decay, B=1, H=H, dk=dk, dv=dv, map_mode="head", hp_dtype="fp32",
                            map=np.ones(H, np.uint8)))
    out, final = qs.scan(q, k, v, d, b)
    st = qs.new_state()
    steps = torch.cat([qs.step(st, q[t:t + 1], k[t:t + 1], v[t:t + 1], d[t:t + 1].clone(), b[t:t + 1], step=t)
                       for t in range(T)])
    S = qs.dequantize(st)
    torch.cuda.synchronize()
    ref = ops_ref.scan(kind, *(x.cpu() for x in (q, k, v, d, b)), [T], None, None)
    check(kind, "bf16", [T], dk, out, final, ref)
    check(kind, "fp32", [T], dk, steps, S, ref)
    qs.close()


def test_serving_run():
    """Prompts of a delta-rule layer through convolution, norm, scan and hand-over into slots of a pool, then decode
    steps, a fork and a compaction: every output against the whole computation in float64 from the same stored state."""
    g = torch.Generator().manual_seed(11)
    H, dk, dv, W, B = 4, 64, 64, 4, 6
    C = 3 * H * dk
    lengths, steps = [37, 5, 90], 4
    slots = [4, 0, 2]
    n, T = len(lengths), sum(lengths)
    bf = torch.bfloat16
    x = torch.randn(T, C, generator=g).to(bf).to(DEV)
    w = (torch.randn(W, C, generator=g) * 0.5).to(DEV)
    slot = torch.tensor(slots, dtype=torch.int32, device=DEV)
    cfg = dict(kind="delta", decay_mode="head", H=H, dk=dk, dv=dv, map_mode="head", hp_dtype="fp32",
               map=np.ones(H, np.uint8))
    pool_qs, some_qs = QState(StateConfig(B=B, **cfg)), QState(StateConfig(B=n, **cfg))
    pool, window = pool_qs.new_state(), torch.zeros(B, W - 1, C, dtype=bf, device=DEV)

    def qkv(rows):
        q, k = qk_norm_rotate(rows[:, :H * dk].unflatten(1, (H, dk)), rows[:, H * dk:2 * H * dk].unflatten(1, (H, dk)),
                              q_scale=dk ** -0.5)
        return q, k, rows[:, 2 * H * dk:].unflatten(1, (H, dv))

    def gates(m):
        return (torch.sigmoid(torch.randn(m, H, generator=g) + 3).to(DEV),
                (torch.sigmoid(torch.randn(m, H, generator=g)) * 0.99).to(DEV))

    q, k, v = qkv(causal_conv(x, w, offsets=offsets(lengths), window=window, slot=slot))
    d, b = gates(T)
    out, S = some_qs.scan(q, k, v, d, b, offsets=offsets(lengths))
    check("delta", "bf16", lengths, dk, out, S,
          ops_ref.scan("delta", *(t.cpu() for t in (q, k, v, d, b)), lengths, None, None))
    temp = some_qs.new_state()
    some_qs.quantize(S, temp)
    pool_qs.copy_slots(pool, torch.arange(n, dtype=torch.int32, device=DEV), slot, source=temp, source_slots=n)
    # fork the second sequence, drop the first
    pool_qs.copy_slots(pool, torch.tensor([0], dtype=torch.int32, device=DEV),
                       torch.tensor([5], dtype=torch.int32, device=DEV), extra=[window])
    live = torch.tensor([1, 0, 1, 0, 0, 1], dtype=torch.uint8, device=DEV)
    where = pool_qs.compact_slots(pool, live, extra=[window])
    assert where.tolist() == [0, -1, 2, -1, -1, 1]
    now = torch.tensor([0, 2, 1], dtype=torch.int32, device=DEV)      # second prompt, third prompt, the fork
    states = pool_qs.dequantize(pool)[[0, 2, 1]].cpu()
    assert torch.equal(states, S.cpu()[[1, 2, 1]])                    # fp32 storage: nothing was lost
    last = window[now.long()].cpu()
    assert torch.equal(last[0], x[39:42].cpu()) and torch.equal(last[0], last[2]) and torch.equal(last[1], x[-3:].cpu())
    qs_, ks_, vs_, ds_, bs_, os_ = [], [], [], [], [], []
    for t in range(steps):
        xt = torch.randn(3, C, generator=g).to(bf).to(DEV)
        rows = causal_conv_step(xt, w, window=window, slot=now)
        q, k, v = qkv(rows)
        d, b = gates(3)
        o = pool_qs.step_batch(pool, now, torch.full((3,), t, dtype=torch.int64, device=DEV), q.contiguous(),
                               k.contiguous(), v.contiguous(), d, b)
        for keep, val in zip((qs_, ks_, vs_, ds_, bs_, os_), (q, k, v, d, b, o)):
            keep.append(val.cpu())
    for i in range(3):
        one = [torch.stack([s[i] for s in seq]) for seq in (qs_, ks_, vs_, ds_, bs_)]
        ref = ops_ref.scan("delta", *one, [steps], states[i:i + 1], None)
        got = torch.stack([s[i] for s in os_])
        check("delta", "fp32", [steps], dk, got, pool_qs.dequantize(pool)[now[i]][None], ref)
    pool_qs.close(), some_qs.close()


@pytest.mark.parametrize("kind,decay", KINDS)
@pytest.mark.parametrize("where,value", [("v", float("nan")), ("v", float("inf")), ("k", float("nan")),
                                         ("decay", float("nan")), ("beta", float("inf")), ("q", float("nan"))])
def test_scan_later_tokens_do_not_reach_earlier_ones(kind, decay, where, value):
    """A value that is not finite at a token leaves every earlier output as it is, and every other sequence."""
    lengths, bad = [150, 40], (70, 75)
    q, k, v, d, b = inputs(kind, decay, lengths, 2, 2, 64, 48, "bf16")
    args = dict(q=q, k=k, v=v, decay=d, beta=b)
    qs = QState(StateConfig(kind=kind, decay_mode=decay, B=2, H=2, dk=64, dv=48))
    clean, cfin = qs.scan(*(x.to(DEV) for x in (q, k, v, d, b)), offsets=offsets(lengths))
    x = args[where].clone()
    for t in bad:
        x[t].view(-1)[3 if x[t].numel() > 3 else 0] = value
    args[where] = x
    out, fin = qs.scan(*(args[n].to(DEV) for n in ("q", "k", "v", "decay", "beta")), offsets=offsets(lengths))
    torch.cuda.synchronize()
    same = lambda a, c: torch.allclose(a.float(), c.float(), rtol=2 ** -7, atol=1e-3)
    assert torch.isfinite(out[:bad[0]]).all() and same(out[:bad[0]], clean[:bad[0]])
    assert torch.isfinite(out[150:]).all() and same(out[150:], clean[150:]) and torch.equal(fin[1], cfin[1])
    assert not torch.isfinite(out[bad[0]:150]).all()
    if where == "v":                                    # only that head's value row
        ok = torch.ones(2, 48, dtype=torch.bool)
        ok[0, 3] = False
        assert torch.isfinite(out[:, ok]).all() and same(out[:, ok], clean[:, ok])
    if where == "q":                                    # nothing of it stays
        assert torch.equal(fin, cfin)
    qs.close()


@pytest.mark.parametrize("kind", ["additive", "delta"])
def test_scan_long_and_many_heads(kind):
    """Long enough to be cut into segments, over cells' and sequences' boundaries."""
    run(kind, "head", [700, 1, 0, 1300, 64, 47], 4, 2, 64, 40, "bf16", initial=True, skip=True, mu=5.0)
    run(kind, "head", [2048], 2, 1, 128, 64, "bf16", mu=6.0)


@pytest.mark.parametrize("kind,decay", KINDS)
def test_scan_in_place_over_many_segments(kind, decay):
    """final may be initial: the state before a sequence's first segment is read from it while the last segment, a
    single token here, is done long before."""
    dk, dv, H, T = 64, 64, 32, 4097
    q, k, v, d, b = (x.to(DEV) for x in inputs(kind, decay, [T], H, 1, dk, dv, "bf16", mu=6.0))
    qs = QState(StateConfig(kind=kind, decay_mode=decay, B=1, H=H, dk=dk, dv=dv))
    S0 = torch.randn(1, H, dv, dk, device=DEV) * 100
    out, fin = qs.scan(q, k, v, d, b, initial=S0)
    for _ in range(5):
        S = S0.clone()
        o, f = qs.scan(q, k, v, d, b, initial=S, final=S)
        torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(f, fin)
    qs.close()


@pytest.mark.parametrize("decay", ["head", "key"])
@pytest.mark.parametrize("dk,dv,H", [(64, 64, 4), (128, 33, 2), (256, 5, 2), (64, 100, 32)])
def test_scan_fp32_in_segments(decay, dk, dv, H):
    """Additive fp32 prompts long enough to be cut, in place, with sequences that end inside a segment."""
    run("additive", decay, [300, 0, 1, 700, 64, 129], H, 2, dk, dv, "fp32", initial=True, skip=True, strided=True,
        mu=5.0)


@pytest.mark.parametrize("kind,decay", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scan_many_rows_of_short_sequences(kind, decay, dtype):
    """More rows than one a lane is taken for, lengths that are not whole groups of tokens."""
    run(kind, decay, [9, 0, 1, 18, 3, 15, 11], 32, 8, 64, 100, dtype, initial=True, skip=True)


@pytest.mark.parametrize("kind,decay", KINDS)
def test_scan_fp32_later_tokens_do_not_reach_earlier_ones(kind, decay):
    lengths, bad = [150, 180], 71
    q, k, v, d, b = (x.to(DEV) for x in inputs(kind, decay, lengths, 2, 2, 64, 48, "fp32"))
    qs = QState(StateConfig(kind=kind, decay_mode=decay, B=2, H=2, dk=64, dv=48, in_dtype="fp32"))
    clean, cfin = qs.scan(q, k, v, d, b, offsets=offsets(lengths))
    v[bad, 0, 3] = float("inf")
    out, fin = qs.scan(q, k, v, d, b, offsets=offsets(lengths))
    torch.cuda.synchronize()
    ok = torch.ones_like(out, dtype=torch.bool)
    ok[bad:150, 0, 3] = False
    assert torch.equal(out[ok], clean[ok]) and not torch.isfinite(out[~ok]).any()
    assert torch.equal(fin[1], cfin[1]) and torch.equal(fin[0, 1], cfin[0, 1]) and not torch.isfinite(fin[0, 0, 3]).all()
    qs.close()


@pytest.mark.parametrize("kind,decay", KINDS)
def test_scan_fp32_infinite_last_value(kind, decay):
    """What the last token leaves in the state is stored as it is, whatever the length."""
    for T in (1, 5, 16, 18):
        q, k, v, d, b = (x.to(DEV) for x in inputs(kind, decay, [T], 1, 1, 64, 8, "fp32"))
        v[T - 1, 0, 2] = float("inf")
        qs = QState(StateConfig(kind=kind, decay_mode=decay, B=1, H=1, dk=64, dv=8, in_dtype="fp32"))
        _, fin = qs.scan(q, k, v, d, b)
        torch.cuda.synchronize()
        assert torch.equal(fin[0, 0, 2], torch.where(k[T - 1, 0] > 0, 1.0, -1.0) * float("inf"))
        assert torch.isfinite(fin[0, 0, [0, 1, 3, 4, 5, 6, 7]]).all()
        qs.close()


@pytest.mark.parametrize("lengths", [[1537], [1024, 1025], [3, 1100, 0, 2600], [1600, 1600, 1600], [63, 4097, 1, 1024]])
@pytest.mark.parametrize("dk,dv,H", [(64, 64, 4), (128, 33, 2), (256, 24, 2)])
def test_scan_delta_in_pieces(lengths, dk, dv, H):
    """Long sequences of few heads by the delta rule, in place: cut into pieces of whole chunks, or not, by their length;
    last pieces of one token, sequences that begin inside a cell."""
    run("delta", "head", lengths, H, 2, dk, dv, "bf16", initial=True, skip=True, strided=True, mu=5.0)
    run("delta", "head", lengths, H, 1, dk, dv, "bf16", mu=2.0)


@pytest.mark.parametrize("dtype,decay", [("fp32", "head"), ("fp32", "key"), ("bf16", "key")])
@pytest.mark.parametrize("lengths", [[193], [128, 129], [3, 150, 0, 400], [200, 200, 200], [15, 513, 1, 128]])
@pytest.mark.parametrize("dk,dv,H", [(64, 64, 4), (128, 33, 2), (256, 24, 2), (64, 100, 16)])
def test_scan_delta_in_pieces_token_by_token(dtype, decay, lengths, dk, dv, H):
    run("delta", decay, lengths, H, 2, dk, dv, dtype, initial=True, skip=True, strided=True, mu=5.0)
    run("delta", decay, lengths, H, 1, dk, dv, dtype, mu=2.0)


@pytest.mark.parametrize("where,value", [("v", float("nan")), ("v", float("inf")), ("k", float("nan")),
                                         ("decay", float("nan")), ("decay", 0.0), ("beta", float("inf"))])
@pytest.mark.parametrize("dtype,decay", [("bf16", "head"), ("fp32", "head"), ("bf16", "key")])
def test_scan_delta_in_pieces_odd_values(where, value, dtype, decay):
    """As in a sequence in one piece: a value that is not finite reaches its head (v: its row) from its token on, and a
    decay of zero cuts off what was before."""
    T, bad, H, dv = 2600, 1300, 2, 48
    names = ("q", "k", "v", "decay", "beta")
    args = dict(zip(names, (x.to(DEV) for x in inputs("delta", decay, [T], H, 2, 64, dv, dtype, mu=6.0))))
    qs = QState(StateConfig(kind="delta", decay_mode=decay, B=1, H=H, dk=64, dv=dv, in_dtype=dtype))
    S0 = torch.randn(1, H, dv, 64, device=DEV)
    scan = lambda a, S, t0=0: qs.scan(*(a[n][t0:] for n in names), initial=S)
    clean, cfin = scan(args, S0)
    args[where] = args[where].clone()
    if where == "decay":
        args[where][bad].view(H, -1)[0] = value
    else:
        args[where][bad].view(-1)[3 if where in ("v", "k") else 0] = value
    out, fin = scan(args, S0)
    torch.cuda.synchronize()
    same = lambda a, c: torch.allclose(a.float(), c.float(), rtol=2 ** -7, atol=1e-3)
    assert torch.isfinite(out[:bad]).all() and same(out[:bad], clean[:bad])
    assert torch.isfinite(out[:, 1]).all() and same(out[:, 1], clean[:, 1]) and same(fin[0, 1], cfin[0, 1])
    if where == "v":
        ok = torch.arange(dv, device=DEV) != 3
        assert torch.isfinite(out[:, 0, ok]).all() and same(out[:, 0, ok], clean[:, 0, ok])
        assert same(fin[0, 0, ok], cfin[0, 0, ok])
        assert not torch.isfinite(out[bad:, 0, 3]).any() and not torch.isfinite(fin[0, 0, 3]).any()
    elif value == 0.0:
        o, f = scan(args, None, bad)
        torch.cuda.synchronize()
        assert same(out[bad:, 0], o[:, 0]) and torch.allclose(fin[0, 0], f[0, 0], rtol=1e-5, atol=1e-6)
    else:
        assert not torch.isfinite(out[bad:, 0]).any() and not torch.isfinite(fin[0, 0]).any()
    qs.close()


@pytest.mark.parametrize("kind,decay", KINDS)
@pytest.mark.parametrize("dk,dv", [(64, 24), (128, 72), (128, 136)])
def test_scan_what_lies_between_value_rows_does_not_matter(kind, decay, dk, dv):
    """v as a slice of a wider tensor: the elements behind its last head, and another head's, change no bit."""
    T, H = 300, 2
    q, k, v, d, b = (x.to(DEV) for x in inputs(kind, decay, [T], H, 1, dk, dv, "bf16"))
    qs = QState(StateConfig(kind=kind, decay_mode=decay, B=1, H=H, dk=dk, dv=dv))

    def scan(behind, second):
        wide = torch.full((T, H * dv + 64), behind, dtype=torch.bfloat16, device=DEV)
        wide[:, :H * dv] = v.flatten(1)
        if second is not None:
            wide[:, dv:H * dv] = second
        out = qs.scan(q, k, wide[:, :H * dv].unflatten(1, (H, dv)), d, b)
        torch.cuda.synchronize()
        return out

    nan = float("nan")
    (o, f), (o1, f1), (o2, f2) = scan(0.0, None), scan(nan, None), scan(0.0, nan)
    assert torch.equal(o, o1) and torch.equal(f, f1)
    assert torch.equal(o[:, 0], o2[:, 0]) and torch.equal(f[:, 0], f2[:, 0])
    qs.close()
