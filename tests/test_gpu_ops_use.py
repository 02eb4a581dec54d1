"""How the operators are used: captured into graphs and replayed between eager
work, on other streams, several at once, on tensors beyond 2^31 elements, and
with what the binding refuses."""
import sys

import numpy as np
import pytest
import torch

from quantized_recurrent_state_qstate_amd import QState, StateConfig, causal_conv, causal_conv_step, qk_norm_rotate
from quantized_recurrent_state_qstate_amd._lib import QStateError

pytestmark = pytest.mark.gpu
DEV = "cuda"


def say(*a):
    print("[use]", *a, file=sys.stderr, flush=True)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def scan_inputs(kind, decay, lengths, H, G, dk, dv, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    T = sum(lengths)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)
    q, k, v = rnd(T, G, dk), torch.nn.functional.normalize(rnd(T, G, dk), dim=-1), rnd(T, H, dv)
    d = torch.sigmoid(rnd(T, H, dk) + 3 if decay == "key" else rnd(T, H) + 3)
    off = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=DEV)
    return dict(q=q.bfloat16(), k=k.bfloat16(), v=v.bfloat16(), decay=d, beta=torch.sigmoid(rnd(T, H)), offsets=off)


def make(op):
    """(run, fresh): run(buffers) makes the calls and returns outputs; fresh() their in/out buffers."""
    g = torch.Generator(device=DEV).manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)
    if op.startswith("scan"):
        kind, decay = op.split("_")[1:]
        qs = QState(StateConfig(kind=kind, decay_mode=decay, B=3, H=4, dk=128, dv=64))
        inp = scan_inputs(kind, decay, [700, 0, 333], 4, 2, 128, 64)
        return lambda s: list(qs.scan(**inp, initial=s[0], final=s[0])), lambda: [torch.ones(3, 4, 64, 128, device=DEV)]
    if op == "conv":
        x, w, b = rnd(90, 64).bfloat16(), rnd(4, 64), rnd(64)
        off = torch.tensor([0, 50, 51, 90], dtype=torch.int32, device=DEV)
        return (lambda s: [causal_conv(x, w, b, offsets=off, window=s[0]),
                           causal_conv_step(x[:3], w, b, window=s[0]), s[0]],
                lambda: [torch.ones(3, 3, 64, device=DEV).bfloat16()])
    if op == "qk":
        q, k = rnd(40, 8, 128).bfloat16(), rnd(40, 4, 128).bfloat16()
        pos = torch.arange(40, dtype=torch.int32, device=DEV)
        freq = 10000.0 ** (-torch.arange(64, device=DEV, dtype=torch.float64) / 64)
        return lambda s: list(qk_norm_rotate(q, k, norm="rms", position=pos, frequency=freq)), lambda: []
    qs = QState(StateConfig(B=6, H=3, dk=64, dv=40))
    live = torch.tensor([0, 1, 0, 1, 1, 1], dtype=torch.uint8, device=DEV)
    src, dst = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([3, -1, 3], [0, 1, 2]))
    vals = rnd(6, 3, 40, 64)

    def fresh():
        st = qs.new_state()
        qs.quantize(vals, st)
        return [st]

    def run(s):
        qs.copy_slots(s[0], src, dst)
        return [qs.compact_slots(s[0], live), s[0]["codes"], s[0]["scales"]]
    return run, fresh


OPS = ["conv", "qk", "slots", "scan_additive_head", "scan_additive_key", "scan_delta_head", "scan_delta_key"]


@pytest.mark.parametrize("op", OPS)
def test_graph_replays_match_eager(op):
    say("graph", op)
    run, fresh = make(op)
    bg, be = fresh(), fresh()
    run(fresh())                                        # loads the kernels
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            og = run(bg)
    torch.cuda.synchronize()
    for rep in range(3):
        graph.replay()
        torch.cuda.synchronize()
        _ = (torch.randn(1 << 18, device=DEV) * 2.0).sum().item()
        oe = run(be)
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(og, oe)):
            assert same(x, y), f"{op}: replay {rep}, output {i}"


@pytest.mark.parametrize("op", OPS)
def test_same_bits_every_time_and_on_another_stream(op):
    say("stream", op)
    run, fresh = make(op)
    first = [x.clone() for x in run(fresh())]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for s in (s1, s2, s1, s2):                          # two streams at work at once, each with its own buffers
        with torch.cuda.stream(s):
            s.wait_stream(torch.cuda.default_stream())
            got.append(run(fresh()))
    torch.cuda.synchronize()
    for outs in got:
        assert all(same(x, y) for x, y in zip(first, outs))


def test_stream_argument():
    """Work put on a stream by argument, with the inputs made there."""
    s = torch.cuda.Stream()
    inp = scan_inputs("additive", "head", [900], 4, 2, 128, 64)
    qs = QState(StateConfig(B=1, H=4, dk=128, dv=64))
    want, wfin = qs.scan(**inp)
    x, w = torch.randn(100, 64, device=DEV), torch.randn(4, 64, device=DEV)
    off = torch.tensor([0, 100], dtype=torch.int32, device=DEV)
    cw = causal_conv(x, w, offsets=off)
    torch.cuda.synchronize()
    got, fin = qs.scan(**inp, stream=s)
    cg = causal_conv(x, w, offsets=off, stream=s)
    s.synchronize()
    assert same(got, want) and same(fin, wfin) and same(cg, cw)


def test_slots_beyond_4_gib():
    B, H, dk, dv = 16384, 32, 128, 128                  # 524 KB of codes a slot: 8.6 GB
    qs = QState(StateConfig(B=8, H=H, dk=dk, dv=dv))
    per = qs.sizes["codes"] // 8
    qs.close()
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB of free GPU memory")
    say("slots", B * per)
    qs = QState(StateConfig(B=B // 8, H=H, dk=dk, dv=dv))      # 2^35 elements bound a handle: the source is the big one
    pool = qs.new_state()
    big = {"codes": torch.empty(B * per, dtype=torch.uint8, device=DEV),
           "scales": torch.empty(B * H * dv, device=DEV)}
    pat = torch.randint(0, 255, (per,), dtype=torch.uint8, device=DEV)
    big["codes"][(B - 1) * per:] = pat
    big["scales"][(B - 1) * H * dv:] = 3.0
    src = torch.tensor([B - 1, B], dtype=torch.int32, device=DEV)
    dst = torch.tensor([B // 8 - 1, 0], dtype=torch.int32, device=DEV)
    qs.copy_slots(pool, src, dst, source=big, source_slots=B)
    torch.cuda.synchronize()
    c = pool["codes"].view(B // 8, per)
    assert torch.equal(c[-1], pat) and not c[:-1].any() and (pool["scales"].view(B // 8, -1)[-1] == 3).all()
    qs.close()


def test_rows_beyond_2_31_elements():
    T, C = 200000, 12288                                # 2.46e9 elements
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of free GPU memory")
    say("conv", T, C)
    x = torch.empty(T, C, dtype=torch.bfloat16, device=DEV)
    n = 1000
    x[-n:] = torch.randn(n, C, device=DEV).bfloat16()
    w = torch.randn(4, C, device=DEV)
    off = torch.tensor([0, T - n, T], dtype=torch.int32, device=DEV)
    out = causal_conv(x, w, offsets=off)
    want = causal_conv(x[-n:], w, offsets=torch.tensor([0, n], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert same(out[-n:], want)
    q = x.view(T, 96, 128)
    qo, _ = qk_norm_rotate(q, q_out=out.view(T, 96, 128))
    qw, _ = qk_norm_rotate(q[-n:])
    torch.cuda.synchronize()
    assert same(qo[-n:], qw)
    # the scan's v and out: the last sequence's tokens lie behind 2^31 elements
    for kind, decay in (("additive", "head"), ("additive", "key"), ("delta", "head")):
        say("scan", kind, decay)
        H, dv, dk = 96, 128, 64
        qs = QState(StateConfig(kind=kind, decay_mode=decay, B=1, H=H, dk=dk, dv=dv))
        inp = scan_inputs(kind, decay, [n], H, 1, dk, dv)
        first = T - n
        small, sfin = qs.scan(**{**inp, "v": q[-n:]})
        wide = {}
        for name in ("q", "k", "decay", "beta"):
            y = inp[name]
            wide[name] = torch.empty(T, *y.shape[1:], dtype=y.dtype, device=DEV)
            wide[name][first:] = y
        off = torch.tensor([first, T], dtype=torch.int32, device=DEV)
        o, fin = qs.scan(wide["q"], wide["k"], q, wide["decay"], wide["beta"], offsets=off, out=out.view(T, H, dv))
        torch.cuda.synchronize()
        # cut into other segments and chunks: the same up to the order of sums
        assert torch.allclose(o[first:].float(), small.float(), rtol=2 ** -6, atol=2 ** -6)
        assert torch.allclose(fin, sfin, rtol=1e-4, atol=1e-4)
        qs.close()
        del wide


def test_binding_refusals_with_a_handle():
    qs = QState(StateConfig(B=2, H=4, dk=64, dv=32))
    inp = scan_inputs("additive", "head", [40, 40], 4, 2, 64, 32)
    st = qs.new_state()
    idx = torch.zeros(1, dtype=torch.int32, device=DEV)
    bad = [
        (dict(q=inp["q"].float()), "q: dtype"), (dict(k=inp["k"][:, :1]), "q: shape"),
        (dict(v=inp["v"][:79]), "q: shape"), (dict(decay=inp["decay"].double()), "decay: dtype"),
        (dict(beta=inp["beta"][:, :3]), "beta: shape"), (dict(offsets=inp["offsets"].long()), "offsets: dtype"),
        (dict(offsets=inp["offsets"].cpu()), "offsets: on cpu"), (dict(skip=torch.zeros(3, device=DEV)), "skip: 3"),
        (dict(initial=torch.zeros(1, 4, 32, 64, device=DEV)), "initial: 8192"),
        (dict(out=torch.zeros(80, 4, 32, device=DEV)), "out: dtype"),
        (dict(final=torch.zeros(2, 4, 32, 64, device=DEV).double()), "final: dtype"),
    ]
    for kw, msg in bad:
        with pytest.raises(ValueError, match=msg):
            qs.scan(**{**inp, **kw})
    with pytest.raises(QStateError, match="does not divide"):
        qs.scan(**{**inp, "q": torch.zeros(80, 3, 64, device=DEV).bfloat16(), "k": torch.zeros(80, 3, 64, device=DEV).bfloat16()})
    with pytest.raises(QStateError, match="overlaps"):
        qs.scan(**inp, out=inp["v"])
    for call, msg in [
        (lambda: qs.copy_slots(st, idx.long(), idx), "src_slot: dtype"),
        (lambda: qs.copy_slots(st, idx, idx.repeat(2)), "dst_slot: 2 elements"),
        (lambda: qs.copy_slots(st, idx, idx, source=st), "source_slots"),
        (lambda: qs.copy_slots(st, idx, idx, source_slots=2), "go with a source"),
        (lambda: qs.copy_slots(dict(st, codes=st["codes"][:-1]), idx, idx), "codes"),
        (lambda: qs.copy_slots(st, idx, idx, extra=[torch.zeros(1, 3, device=DEV)]), "at least 2 slots"),
        (lambda: qs.copy_slots(st, idx, idx, extra=[torch.zeros(2, 3)]), "on cpu"),
        (lambda: qs.copy_slots(st, idx, idx, extra=[torch.zeros(2, 3, device=DEV)] * 7), "at most 6"),
        (lambda: qs.compact_slots(st, torch.zeros(3, dtype=torch.uint8, device=DEV)), "live: 3"),
        (lambda: qs.compact_slots(st, torch.zeros(2, device=DEV)), "live: dtype"),
    ]:
        with pytest.raises(ValueError, match=msg):
            call()
    qs.close()


def test_qk_norm_of_huge_values():
    """Squares that overflow fp32 still give unit heads."""
    x = torch.randn(6, 2, 64, generator=torch.Generator().manual_seed(1))
    for scale, norm in ((1e37, "l2"), (1e37, "rms"), (1e25, "l2"), (1.0, "l2")):
        y = (x * scale).to(DEV)
        out, _ = qk_norm_rotate(y, norm=norm, eps=0.0)
        ref = (x * scale).double()
        m = ref.square().sum(-1, keepdim=True) / (64 if norm == "rms" else 1)
        assert torch.allclose(out.cpu().double(), ref / m.sqrt(), rtol=1e-5, atol=1e-6)
