"""The operators around the decode step, as they are measured: the short causal
convolution (prompts and single tokens), the scan of a prompt into a state, the
norm and rotation of queries and keys, and the copying and compacting of state
slots.

Sizes follow this package's own workloads: mamba2 (32 heads of 64 x 128, 2048 +
2 * 128 convolved channels), gdn (32 heads of 128 x 128, 3 * 4096 convolved
channels), gla_int4's recurrence and gla_small.  `own` false computes everything
with elementary torch operations in 32 bits (logarithms of decays and rotation
angles in 64); `own` true calls the package."""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one token for each of 8 running sequences, the channels of a mamba2 layer: latency
        dict(name="conv_token", op="conv_step", n=8, slots=256, C=2304, W=4, bias=True, dtype="bf16"),
        # a batch of prompts of uneven length (one empty, one of a single token) in fp32
        dict(name="conv_prompt_ragged", op="conv", n=13, T=4011, slots=16, C=2304, W=4, bias=True, dtype="fp32"),
        # a long prompt through the three convolved projections of a gdn layer
        dict(name="conv_prompt_long", op="conv", n=1, T=16384, slots=4, C=12288, W=4, bias=False, dtype="bf16"),
        # one token for each of 64 sequences: norm with weights, rotation far into a long context
        dict(name="qk_token", op="qk", T=64, Hq=32, Hk=32, d=128, rot=128, norm="rms", interleaved=False, far=262144,
             dtype="bf16"),
        # the queries and keys of a prompt, cut out of one projection
        dict(name="qk_prompt", op="qk", T=8192, Hq=32, Hk=32, d=128, rot=64, norm="l2", interleaved=True, far=8192,
             dtype="bf16"),
        # one prefix state forked into seven more sequences (mamba2 slots: int8 heads and bf16 heads)
        dict(name="slots_fork", op="fork", B=256, H=32, P=8, dv=64, dk=128, n=7, sources=1),
        # half of a gdn pool's sequences have ended: the live ones move to the front
        dict(name="slots_compact", op="compact", B=256, H=32, P=0, dv=128, dk=128, live=128),
        # the smallest scan: gla_small's 32 tokens in fp32
        dict(name="scan_gla_small", op="scan", kind="additive", decay="key", n=1, T=32, H=2, G=2, dk=64, dv=64,
             dtype="fp32", initial=False, skip=False),
        # a batch of short prompts of a mamba2 layer, keys and queries shared by all heads
        dict(name="scan_mamba2_ragged", op="scan", kind="additive", decay="head", n=32, T=8011, H=32, G=1, dk=128, dv=64,
             dtype="bf16", initial=False, skip=True),
        # one long prompt of a mamba2 layer, continued from a state
        dict(name="scan_mamba2_long", op="scan", kind="additive", decay="head", n=1, T=16384, H=32, G=1, dk=128, dv=64,
             dtype="bf16", initial=True, skip=True),
        # four prompts of a gdn layer, each key head shared by two value heads
        dict(name="scan_gdn", op="scan", kind="delta", decay="head", n=4, T=8192, H=32, G=16, dk=128, dv=128,
             dtype="bf16", initial=True, skip=False),
        # two prompts of a gla layer: a decay for every key channel
        dict(name="scan_gla", op="scan", kind="additive", decay="key", n=2, T=2048, H=32, G=32, dk=128, dv=128,
             dtype="bf16", initial=False, skip=False),
    ]


def _log_int(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["conv_step", "conv", "qk", "fork", "compact", "scan", "scan", "scan", "scan"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "conv_step":
        n = _log_int(rng, 1, 256)
        return dict(op=op, n=n, slots=n + rng.randint(0, 64), C=_log_int(rng, 64, 8192), W=rng.choice([2, 3, 4]),
                    bias=rng.random() < 0.5, dtype=dtype)
    if op == "conv":
        n = _log_int(rng, 1, 64)
        return dict(op=op, n=n, T=_log_int(rng, 64, 8192), slots=n + rng.randint(0, 8), C=_log_int(rng, 64, 8192),
                    W=rng.choice([2, 3, 4]), bias=rng.random() < 0.5, dtype=dtype)
    if op == "qk":
        d = rng.choice([64, 128, 256, 8 * rng.randint(4, 32)])
        Hk = rng.choice([1, 2, 4, 8, 16, 32])
        return dict(op=op, T=_log_int(rng, 1, 4096), Hq=Hk * rng.choice([1, 2]), Hk=Hk, d=d,
                    rot=rng.choice([0, d // 16 * 16, d // 32 * 16]), norm=rng.choice(["l2", "rms", "none"]),
                    interleaved=rng.random() < 0.5, far=_log_int(rng, 4096, 1 << 20), dtype=dtype)
    if op in ("fork", "compact"):
        dv, dk, H = rng.choice([64, 96, 128]), rng.choice([64, 128]), rng.choice([8, 16, 32])
        B = rng.randint(16, 128)
        base = dict(op=op, B=B, H=H, P=rng.choice([0, H // 4]), dv=dv, dk=dk)
        if op == "compact":
            return dict(base, live=rng.randint(1, B - 1))
        n = rng.randint(1, B // 2)
        return dict(base, n=n, sources=rng.randint(1, min(n, B // 4)))
    kind, decay = rng.choice([("additive", "head"), ("delta", "head"), ("additive", "key"), ("delta", "key")])
    H = rng.choice([2, 4, 8, 16, 32])
    dk = rng.choice([64, 128, 256])
    dv = rng.choice([64, 128, rng.randint(16, 128)])
    T = _log_int(rng, 32, 4096 if decay == "head" else 1024)
    return dict(op="scan", kind=kind, decay=decay, n=_log_int(rng, 1, 16), T=T, H=H, G=rng.choice([1, H // 2, H]),
                dk=dk, dv=dv, dtype=dtype, initial=rng.random() < 0.5, skip=rng.random() < 0.3)


def _lengths(case):
    """The sequences' lengths: uneven, of sum T; from four sequences on one is empty and one has a single token."""
    n, T = case["n"], case["T"]
    r = random.Random(1000003 * n + T)
    cuts = sorted(r.randint(0, T) for _ in range(n - 1))
    got = [b - a for a, b in zip([0] + cuts, cuts + [T])]
    if n >= 4:
        spare = got[0] + got[1]
        got[0], got[1] = 0, min(1, spare)
        got[2] += spare - got[1]
    return got


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = dict(case=case)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=DEV).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    def slots_of(n, of):
        return torch.randperm(of, generator=g, device=DEV)[:n].to(torch.int32)

    op = case["op"]
    if op in ("conv", "conv_step"):
        dt, C, W = DTYPE[case["dtype"]], case["C"], case["W"]
        rows = case["n"] if op == "conv_step" else case["T"]
        s["x"] = normal(rows, C, dtype=dt)
        s["weight"] = normal(W, C) / math.sqrt(W)
        s["bias"] = normal(C) * 0.5 if case["bias"] else None
        s["window"] = normal(case["slots"], W - 1, C, dtype=dt)
        s["slot"] = slots_of(case["n"], case["slots"])
        if op == "conv":
            s["lengths"] = _lengths(case)
            s["offsets"] = _offsets(s["lengths"])
    elif op == "qk":
        dt, T, d = DTYPE[case["dtype"]], case["T"], case["d"]
        Hq, Hk = case["Hq"], case["Hk"]
        both = normal(T, (Hq + Hk) * d, dtype=dt)                    # one projection's rows
        s["q"], s["k"] = both[:, :Hq * d].unflatten(1, (Hq, d)), both[:, Hq * d:].unflatten(1, (Hk, d))
        s["q_weight"] = s["k_weight"] = None
        if case["norm"] == "rms":
            s["q_weight"], s["k_weight"] = 1 + 0.2 * normal(d), 1 + 0.2 * normal(d)
        s["position"] = s["frequency"] = None
        if case["rot"]:
            start = torch.randint(0, max(1, case["far"] - T), (1,), generator=g, device=DEV)
            s["position"] = (start + torch.arange(T, device=DEV)).to(torch.int32)
            i = torch.arange(case["rot"] // 2, device=DEV, dtype=torch.float64)
            s["frequency"] = 10000.0 ** (-2.0 * i / case["rot"])
    elif op in ("fork", "compact"):
        B, H, P, dv, dk = (case[x] for x in ("B", "H", "P", "dv", "dk"))
        # int8 codes of the H - P quantized heads, a scale for each row, bf16 rows of the P protected heads
        s["codes"] = torch.randint(-127, 128, (B, (H - P) * dv * dk), generator=g, device=DEV, dtype=torch.int8)
        s["scales"] = uniform(B, H * dv) * 0.05
        s["hp"] = normal(B, P * dv * dk, dtype=torch.bfloat16)
        order = torch.randperm(B, generator=g, device=DEV).to(torch.int32)
        if op == "fork":
            n, m = case["n"], case["sources"]
            s["src"] = order[:m].repeat((n + m - 1) // m)[:n].contiguous()
            s["dst"] = order[m:m + n].contiguous()
        else:
            s["live"] = torch.zeros(B, dtype=torch.uint8, device=DEV)
            s["live"][order[:case["live"]].long()] = 1
        if own:
            import numpy as np
            from quantized_recurrent_state_qstate_amd import QState, StateConfig
            m = (np.arange(H) < P).astype(np.uint8)
            s["handle"] = QState(StateConfig(B=B, H=H, dk=dk, dv=dv, qbits=8, map_mode="head" if P else "none",
                                             map=m if P else None))
    else:
        dt, T, H, G, dk, dv = DTYPE[case["dtype"]], case["T"], case["H"], case["G"], case["dk"], case["dv"]
        delta, key = case["kind"] == "delta", case["decay"] == "key"
        # value, key and query rows next to each other, as the convolution before them writes them
        rows = normal(T, H * dv + 2 * G * dk)
        v, k, q = rows.split([H * dv, G * dk, G * dk], dim=1)
        if delta:
            k = torch.nn.functional.normalize(k.unflatten(1, (G, dk)), dim=-1).flatten(1)
        elif key:
            k, q = k * 0.125, q * 0.125
        rows = torch.cat([v, k, q], 1).to(dt)
        s["v"] = rows[:, :H * dv].unflatten(1, (H, dv))
        s["k"] = rows[:, H * dv:H * dv + G * dk].unflatten(1, (G, dk))
        s["q"] = rows[:, H * dv + G * dk:].unflatten(1, (G, dk))
        if key:
            s["decay"] = torch.sigmoid(normal(T, H, dk) + 5.0)
            s["beta"] = torch.sigmoid(normal(T, H)) if delta else None
        elif delta:
            s["decay"], s["beta"] = torch.sigmoid(normal(T, H) + 4.0), torch.sigmoid(normal(T, H))
        else:
            step = torch.nn.functional.softplus(normal(T, H) * 0.5 - 2.0)
            s["decay"], s["beta"] = torch.exp(-step * torch.exp(2.0 * uniform(H))), step
        s["skip"] = normal(H) if case["skip"] else None
        s["initial"] = normal(case["n"], H, dv, dk) * 0.3 if case["initial"] else None
        s["lengths"] = _lengths(case)
        s["offsets"] = _offsets(s["lengths"])
        if own:
            from quantized_recurrent_state_qstate_amd import QState, StateConfig
            s["handle"] = QState(StateConfig(kind=case["kind"], decay_mode=case["decay"], B=max(1, case["n"]), H=H,
                                             dk=dk, dv=dv, in_dtype=case["dtype"]))
    return s


def _offsets(lengths):
    sums = [0]
    for x in lengths:
        sums.append(sums[-1] + x)
    return torch.tensor(sums, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    return (OWN if own else PLAIN)[op](s)


def _own_conv(s):
    from quantized_recurrent_state_qstate_amd import causal_conv
    out = causal_conv(s["x"], s["weight"], s["bias"], offsets=s["offsets"], window=s["window"], slot=s["slot"])
    return {"out": out, "window": s["window"]}


def _own_conv_step(s):
    from quantized_recurrent_state_qstate_amd import causal_conv_step
    out = causal_conv_step(s["x"], s["weight"], s["bias"], window=s["window"], slot=s["slot"])
    return {"out": out, "window": s["window"]}


def _own_qk(s):
    from quantized_recurrent_state_qstate_amd import qk_norm_rotate
    c = s["case"]
    q, k = qk_norm_rotate(s["q"], s["k"], norm=c["norm"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6,
                          position=s["position"], frequency=s["frequency"], interleaved=c["interleaved"],
                          q_scale=c["d"] ** -0.5)
    return {"q": q, "k": k}


def _pool(s):
    """The slots' buffers as the handle knows them (its codes and protected rows are bytes)."""
    return {"codes": s["codes"].view(torch.uint8).view(-1), "scales": s["scales"].view(-1),
            "hp": s["hp"].view(torch.uint8).view(-1)}


def _own_fork(s):
    s["handle"].copy_slots(_pool(s), s["src"], s["dst"])
    return {"codes": s["codes"], "scales": s["scales"], "hp": s["hp"]}


def _own_compact(s):
    where = s["handle"].compact_slots(_pool(s), s["live"])
    return {"codes": s["codes"], "scales": s["scales"], "hp": s["hp"], "where": where}


def _own_scan(s):
    out, final = s["handle"].scan(s["q"], s["k"], s["v"], s["decay"], s["beta"], offsets=s["offsets"],
                                  initial=s["initial"], skip=s["skip"])
    return {"out": out, "final": final}


def _silu(y):
    return y / (1 + torch.exp(-y))


def _plain_conv(s):
    x, weight, bias, offsets, window = s["x"], s["weight"], s["bias"], s["offsets"].long(), s["window"]
    T, C = x.shape
    W, N, slot = weight.shape[0], window.shape[0], s["slot"].long()
    table = torch.cat([window.view(N * (W - 1), C), x])              # rows before a sequence are its window's
    t = torch.arange(T, device=x.device)
    seq = torch.searchsorted(offsets[1:], t, right=True)

    def rows(p, i):
        before = p - offsets[i]
        return torch.where(before < 0, slot[i] * (W - 1) + W - 1 + before, N * (W - 1) + p)

    y = sum(weight[j] * table[rows(t - (W - 1 - j), seq)].float() for j in range(W))
    y = _silu(y if bias is None else y + bias)
    i = torch.arange(offsets.numel() - 1, device=x.device)[:, None]
    last = rows(offsets[1:, None] - (W - 1) + torch.arange(W - 1, device=x.device), i)
    window[slot] = table[last]
    return {"out": y.to(x.dtype), "window": window}


def _plain_conv_step(s):
    x, bias, window, slot = s["x"], s["bias"], s["window"], s["slot"].long()
    rows = torch.cat([window[slot], x[:, None]], 1)
    y = (rows.float() * s["weight"]).sum(1)
    y = _silu(y if bias is None else y + bias)
    window[slot] = rows[:, 1:]
    return {"out": y.to(x.dtype), "window": window}


def _plain_qk(s):
    c = s["case"]
    d, rot = c["d"], c["rot"]
    if rot:
        angle = s["position"].double()[:, None] * s["frequency"]
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def one(x, weight, scale):
        y = x.float()
        if c["norm"] == "l2":
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) + 1e-6)
        elif c["norm"] == "rms":
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight
        if rot:
            part = y[..., :rot]
            a, b = (part[..., 0::2], part[..., 1::2]) if c["interleaved"] else part.chunk(2, -1)
            a, b = a * cos - b * sin, a * sin + b * cos
            part = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
            y = torch.cat([part, y[..., rot:]], -1)
        return (y * scale).to(x.dtype)

    return {"q": one(s["q"], s["q_weight"], d ** -0.5), "k": one(s["k"], s["k_weight"], 1.0)}


def _plain_fork(s):
    src, dst = s["src"].long(), s["dst"].long()
    got = {n: s[n] for n in ("codes", "scales", "hp")}
    for x in got.values():
        x[dst] = x[src]
    return got


def _plain_compact(s):
    live = s["live"] != 0
    B = live.numel()
    at = torch.arange(B, device=live.device)
    front = at < live.sum()                                          # where the live slots end up
    src, dst = (live & ~front).nonzero()[:, 0], (front & ~live).nonzero()[:, 0]
    where = at.clone()
    where[src] = dst
    where = torch.where(live, where, torch.full_like(at, -1))
    got = {n: s[n] for n in ("codes", "scales", "hp")}
    for x in got.values():
        x[dst] = x[src]
    return dict(got, where=where.to(torch.int32))


def _plain_scan(s):
    """Chunks of L tokens: with c the running sum of log decays from a chunk's start,
    S_i = e^{c_i} S + sum_{j<=i} e^{c_i - c_j} u_j k_j^T, so a chunk is a few masked products;
    the states between chunks follow from one product with the decays between chunks
    (additive), or chunk by chunk (delta rule, where u depends on the state)."""
    c, offsets = s["case"], s["offsets"].long()
    delta, key, dt = c["kind"] == "delta", c["decay"] == "key", DTYPE[c["dtype"]]
    T, H, G, dk, dv, n = c["T"], c["H"], c["G"], c["dk"], c["dv"], c["n"]
    L = 16 if key else 64
    counts = [(x + L - 1) // L for x in s["lengths"]]
    N, most, dev = sum(counts), max(counts + [0]), offsets.device
    count = torch.tensor(counts, device=dev)
    first = torch.cumsum(count, 0) - count
    seq = torch.repeat_interleave(torch.arange(n, device=dev), count, output_size=N)
    token = offsets[seq, None] + (torch.arange(N, device=dev) - first[seq])[:, None] * L + torch.arange(L, device=dev)
    real = token < offsets[seq + 1, None]
    at = token.clamp(max=T - 1)

    def chunks(x, empty=0.0):                                        # [T, heads, ...] -> [N, heads, L, ...]
        y = x.float()[at]
        y = torch.where(real.view(N, L, *[1] * (y.dim() - 2)), y, torch.full_like(y, empty))
        return y.transpose(1, 2)

    def heads(x):
        return x.repeat_interleave(H // G, 1) if G < H else x

    q, k, v = heads(chunks(s["q"])), heads(chunks(s["k"])), chunks(s["v"])
    beta = 1.0 if s["beta"] is None else chunks(s["beta"])[..., None]
    d = chunks(s["decay"], 1.0).double().log()
    cum = torch.cumsum(d if key else d[..., None], 2)                # [N, H, L, dk or 1]
    total = cum[:, :, -1]                                            # [N, H, dk or 1]
    grow, rest = cum.exp().float(), (total[:, :, None] - cum).exp().float()
    low = torch.ones(L, L, device=dev).tril()

    def pairs(a):                                                    # sum over channels of a_i k_j e^{c_i - c_j}, j <= i
        if not key:
            gap = (cum - cum.transpose(2, 3)).clamp(max=0).float()
            return (a @ k.transpose(2, 3)) * gap.exp() * low
        gap = (cum[:, :, :, None] - cum[:, :, None]).clamp(max=0).float()
        return (a[:, :, :, None] * k[:, :, None] * gap.exp()).sum(-1) * low

    seen, u = pairs(q), v * beta
    start = s["initial"] if s["initial"] is not None else torch.zeros(n, H, dv, dk, device=dev)
    if not delta:
        local = (u * 1.0).transpose(2, 3) @ (k * rest)               # [N, H, dv, dk]
        run_ = torch.cumsum(total, 0)                                # logs over all chunks, one sequence after another
        begin = run_ - total
        same = seq[:, None] == seq[None]
        order = torch.arange(N, device=dev)
        before = same & (order[:, None] > order[None])
        base = (begin - begin[first[seq]]).exp().float()             # from a sequence's start to a chunk's
        if key:
            between = (begin[:, None] - run_[None]).clamp(max=0).float().exp() * before[..., None, None]
            carry = between.permute(2, 3, 0, 1) @ local.permute(1, 3, 0, 2)      # [H, dk, N, dv]
            carry = carry.permute(2, 0, 3, 1)
        else:
            between = (begin[:, None] - run_[None]).clamp(max=0).float().exp()[..., 0] * before[..., None]
            carry = (between.permute(2, 0, 1) @ local.permute(1, 0, 2, 3).reshape(H, N, dv * dk)).view(H, N, dv, dk).transpose(0, 1)
        states = carry + base[:, :, None] * start[seq]
        o = seen @ u + (q * grow) @ states.transpose(2, 3)
        end = total.exp().float()[:, :, None] * states + local
        final = start.clone()
        has = count > 0
        final[has] = end[(first + count - 1)[has]]
    else:
        a = pairs(k) * beta * low.tril(-1)
        eye = torch.eye(L, device=dev)
        inverse, power = eye - a, a @ a                              # (I + a)^-1 = (I - a)(I + a^2)(I + a^4)...
        for _ in range(int(math.log2(L)) - 1):
            inverse, power = inverse @ (eye + power), power @ power
        u0, kin = inverse @ u, inverse @ (k * grow * beta)

        def padded(x):                                               # a chunk of nothing for sequences that have ended
            return torch.cat([x, torch.zeros_like(x[:1])])

        u0, kin, seen, qin, kout = padded(u0), padded(kin), padded(seen), padded(q * grow), padded(k * rest)
        hold = torch.cat([total.exp().float(), torch.ones_like(total[:1]).float()])
        state, o = start, torch.zeros(N + 1, H, L, dv, device=dev)
        for i in range(most):
            which = torch.where(i < count, first + i, N)
            w = u0[which] - kin[which] @ state.transpose(2, 3)
            o[which] = seen[which] @ w + qin[which] @ state.transpose(2, 3)
            state = hold[which][:, :, None] * state + w.transpose(2, 3) @ kout[which]
        final, o = state, o[:N]
    o = o.transpose(1, 2)[real]                                      # [T, H, dv], sequences in order
    if s["skip"] is not None:
        o = o + s["skip"][:, None] * s["v"].float()
    return {"out": o.to(dt), "final": final}


OWN = {"conv": _own_conv, "conv_step": _own_conv_step, "qk": _own_qk, "fork": _own_fork, "compact": _own_compact,
       "scan": _own_scan}
PLAIN = {"conv": _plain_conv, "conv_step": _plain_conv_step, "qk": _plain_qk, "fork": _plain_fork,
         "compact": _plain_compact, "scan": _plain_scan}


# ---------------------------------------------------------------- bytes and operations
def work(case):
    c, op = case, case["op"]
    size = 2 if c.get("dtype") == "bf16" else 4
    if op in ("conv", "conv_step"):
        rows = c["n"] if op == "conv_step" else c["T"]
        C, W, n = c["C"], c["W"], c["n"]
        return {"bytes": 2 * rows * C * size + 2 * n * (W - 1) * C * size + (W + c["bias"]) * C * 4 + 8 * n,
                "flops": rows * C * (2 * W + 5)}
    if op == "qk":
        values = c["T"] * (c["Hq"] + c["Hk"]) * c["d"]
        return {"bytes": 2 * values * size + 4 * c["T"] * bool(c["rot"]), "flops": 8 * values}
    if op in ("fork", "compact"):
        slot = (c["H"] - c["P"]) * c["dv"] * c["dk"] + 4 * c["H"] * c["dv"] + 2 * c["P"] * c["dv"] * c["dk"]
        if op == "fork":
            return {"bytes": slot * (c["sources"] + c["n"]) + 8 * c["n"], "flops": 0}
        moved = max(1, round(c["live"] * (c["B"] - c["live"]) / c["B"]))     # live slots behind the front, on average
        return {"bytes": 2 * slot * moved + 5 * c["B"], "flops": 0}
    T, H, G, dk, dv, n = (c[x] for x in ("T", "H", "G", "dk", "dv", "n"))
    rows = T * (2 * G * dk + 2 * H * dv) * size
    gates = 4 * T * H * ((dk if c["decay"] == "key" else 1) + (c["kind"] == "delta" or c["decay"] == "head"))
    states = 4 * n * H * dv * dk * (1 + c["initial"])
    return {"bytes": rows + gates + states, "flops": T * H * dv * dk * (7 if c["kind"] == "delta" else 5)}


# ---------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("conv", "conv_step"):
        W, w, slot = case["W"], s["weight"].double(), s["slot"].tolist()
        lengths = [1] * case["n"] if op == "conv_step" else s["lengths"]
        out, window, a = torch.empty_like(s["x"], dtype=torch.float64), s["window"].double(), 0
        for n, i in zip(lengths, slot):
            rows = torch.cat([window[i], s["x"][a:a + n].double()])
            y = torch.zeros_like(rows[:n])
            for j in range(W):
                y += rows[j:j + n] * w[j]
            if s["bias"] is not None:
                y += s["bias"].double()
            out[a:a + n] = y * torch.sigmoid(y)
            window[i] = rows[n:]
            a += n
        return {"out": out, "window": window}
    if op == "qk":
        rot, got = case["rot"], {}
        for name, scale in (("q", case["d"] ** -0.5), ("k", 1.0)):
            x = s[name].double()
            if case["norm"] != "none":
                m = x.square().sum(-1, keepdim=True) / (case["d"] if case["norm"] == "rms" else 1)
                x = x * (m + 1e-6) ** -0.5
            if case["norm"] == "rms":
                x = x * s[name + "_weight"].double()
            y = x.clone()
            if rot:
                i = torch.arange(rot // 2, device=DEV)
                lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
                turn = torch.polar(torch.ones(1, device=DEV, dtype=torch.float64),
                                   torch.outer(s["position"].double(), s["frequency"]))[:, None]
                z = torch.complex(x[..., lo], x[..., hi]) * turn
                y[..., lo], y[..., hi] = z.real, z.imag
            got[name] = y * scale
        return got
    if op in ("fork", "compact"):
        got = {n: s[n].double() for n in ("scales", "hp")}
        if op == "fork":
            moves = list(zip(s["src"].tolist(), s["dst"].tolist()))
        else:
            live = s["live"].tolist()
            front = sum(live)
            moves = list(zip([i for i in range(front, case["B"]) if live[i]], [i for i in range(front) if not live[i]]))
        for a, b in moves:
            for x in got.values():
                x[b] = x[a]
        return dict(got, codes=None, where=None) if op == "compact" else dict(got, codes=None)
    # one token of every sequence after the other
    H, G, n = case["H"], case["G"], case["n"]
    lengths, offsets, T = s["lengths"], s["offsets"].long(), case["T"]
    S = torch.zeros(n, H, case["dv"], case["dk"], device=DEV, dtype=torch.float64)
    if s["initial"] is not None:
        S += s["initial"].double()
    out = torch.zeros(T, H, case["dv"], device=DEV, dtype=torch.float64)
    group = torch.arange(H, device=DEV) // (H // G)
    order = sorted(range(n), key=lambda i: -lengths[i])              # the longest first: the running ones are a prefix
    S, head = S[order], offsets[:-1][torch.tensor(order, device=DEV)]
    for i in range(max(lengths)):
        m = sum(lengths[j] > i for j in order)
        t = head[:m] + i
        d = s["decay"][t].double()
        k, q, u = s["k"][t].double()[:, group], s["q"][t].double()[:, group], s["v"][t].double()
        S[:m] *= d[:, :, None] if case["decay"] == "key" else d[:, :, None, None]
        if case["kind"] == "delta":
            u = u - (S[:m] * k[:, :, None]).sum(-1)
        if s["beta"] is not None:
            u = u * s["beta"][t].double()[..., None]
        S[:m] += u[..., None] * k[:, :, None]
        out[t] = (S[:m] * q[:, :, None]).sum(-1)
    final = torch.empty_like(S)
    final[order] = S
    if s["skip"] is not None:
        out += s["skip"].double()[:, None] * s["v"].double()
    return {"out": out, "final": final}
