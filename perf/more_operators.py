"""What the operators around a softmax block over a 4-bit cache are measured on.

A block reads the residual stream, and leaves its output there, and between the two its attention reads a cache
whose keys and values are held in 4 bits (blocks of 32 elements of a head share one power of two):

    residual_norm            norm of a block's output, its scaled sum with the residual stream and the norm before
                             the next block, in one pass
    gated_norm               per-head norm of a mixer's output times its activated gate
    cache_write_fp4_varlen   new keys and values into the 4-bit cache; cache_read_fp4_varlen gives back what it
                             stands for
    attention_fp4_varlen     causal attention with grouped heads of packed sequences over that cache

`listed()` gives the cases, `draw(rng)` more of the same ranges, `prepare(case, seed)` their inputs on the GPU,
`run(state)` one pass (elementary torch operations in 32 bits, or the package's kernels where `own` is true),
`work(case)` the bytes and operations a pass cannot do without and `exact(case, seed)` the result in 64 bits.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6

# The 4-bit values (bit 3 is the sign) and the shared powers of two: a block's largest element is at most 6 of them.
# They are such that every value of a block is a number of its type (4 * 2^126 would not be).
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = 32
POWERS = {"f32": (-126, 125), "bf16": (-126, 125), "f16": (-23, 13)}


# ---- cases ---------------------------------------------------------------------------------------
# Lengths are drawn from the case itself (`lengths` seeds them): `q_lo`..`q_hi` new tokens a sequence,
# `past_lo`..`past_hi` tokens already in the cache.  `gaps` makes the first, the middle and the last sequence
# empty.  `heads_major` keeps the cache as [heads, rows, ...] instead of [rows, heads, ...].
def _residual(name, kind, N, C, post, stream, channels):
    return dict(name=name, op="residual", type=kind, N=N, C=C, post=post, stream=stream, channels=channels)


def _gated(name, kind, N, H, V, activation, gate_first, packed):
    return dict(name=name, op="gated", type=kind, N=N, H=H, V=V, activation=activation, gate_first=gate_first,
                packed=packed)


def _cached(name, op, kind, B, q, past, H, HK, D, lengths, heads_major=True, gaps=False, lse=False):
    return dict(name=name, op=op, type=kind, B=B, q_lo=q[0], q_hi=q[1], past_lo=past[0], past_hi=past[1], H=H, HK=HK,
                D=D, heads_major=heads_major, lengths=lengths, gaps=gaps, lse=lse)


def listed():
    return [
        # one decode step of a full batch: the residual stream is taken on to the next block
        _residual("residual_decode", "bf16", 256, 4096, False, "bf16", False),
        # the prompts of a prefill batch, norms before and after the block, the stream kept in single precision
        _residual("residual_prefill", "bf16", 24748, 4096, True, "f32", True),
        # one decode step's recurrent output behind its gate
        _gated("gated_decode", "bf16", 256, 32, 128, "silu", False, True),
        # a ragged half-precision batch with narrow heads, the gate inside the norm
        _gated("gated_ragged", "f16", 9111, 16, 64, "sigmoid", True, False),
        # one decode step of 64 sequences: a launch's latency counts
        _cached("store_decode", "store", "bf16", 64, (1, 1), (0, 100), 16, 2, 256, 11),
        # the prompts of a prefill batch, written to a fresh cache and read back
        _cached("store_prefill", "store", "bf16", 8, (512, 4096), (0, 0), 32, 8, 128, 103, heads_major=False),
        # the smallest call: one token of one conversation
        _cached("fp4_single", "attention", "f16", 1, (1, 1), (1022, 1022), 16, 4, 64, 21),
        # one token of one sequence over a very long cache
        _cached("fp4_long_cache", "attention", "bf16", 1, (1, 1), (131071, 131071), 16, 2, 256, 22),
        # a decode step of a full batch with contexts of every length
        _cached("fp4_decode", "attention", "bf16", 256, (1, 1), (0, 4095), 32, 8, 128, 102),
        # a verification step: four drafted tokens and the last accepted one, per sequence
        _cached("fp4_verify", "attention", "bf16", 64, (5, 5), (1000, 8000), 16, 2, 256, 24, heads_major=False),
        # prompts continued over what the cache holds
        _cached("fp4_continued", "attention", "bf16", 8, (512, 4096), (0, 3000), 32, 8, 128, 103),
        # the same in single precision, ragged, empty ones among them
        _cached("fp4_ragged_f32", "attention", "f32", 64, (0, 300), (0, 1000), 16, 4, 64, 105, heads_major=False, gaps=True,
                lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# No drawn case moves or computes more than these (all of them below the largest listed case's).
_SCORES = 3 << 30    # H * B * longest query * longest key: the plain form's score matrix
_GATHER = 1 << 30    # B * longest key * HK * D: the plain form's padded keys
_ELEMENTS = 1 << 26  # of a norm's input, of the new keys, and of a cache that is read back


def draw(rng):
    while True:
        op = rng.choice(["residual", "gated", "store", "attention", "attention", "attention", "attention"])
        kind = rng.choice(["bf16", "bf16", "f16", "f32"])
        if op == "residual":
            N, C = _log(rng, 1, 30000), 8 * rng.choice([rng.randrange(8, 1200), 512, 256, 640, 1024, 288])
            if N * C > _ELEMENTS:
                continue
            c = _residual("", kind, N, C, rng.random() < 0.5, rng.choice([kind, "f32"]), rng.random() < 0.3)
        elif op == "gated":
            N, H = _log(rng, 1, 30000), rng.choice([1, 2, 4, 6, 8, 12, 16, 32, 64])
            V = rng.choice([64, 128, 256, 512, 1024, 8 * rng.randrange(1, 129)])
            if N * H * V > _ELEMENTS:
                continue
            c = _gated("", kind, N, H, V, rng.choice(["silu", "silu", "sigmoid"]), rng.random() < 0.4, rng.random() < 0.5)
        else:
            HK = rng.choice([1, 2, 3, 4, 8])
            H = HK * rng.choice([1, 2, 3, 4, 5, 8, 16])
            D = rng.choice([64, 128, 256, 64, 128, 256, 32, 96, 160, 192, 224])
            form = rng.choice(["token", "block", "prompt"])
            if form == "token":
                B, q = _log(rng, 1, 256), (1, 1)
            elif form == "block":
                hi = rng.randrange(2, 10)
                B, q = _log(rng, 1, 96), (rng.randrange(1, hi), hi)
            else:
                hi = _log(rng, 16, 8192)
                B, q = _log(rng, 1, 64), (max(0, hi // rng.choice([1, 2, 8]) - rng.randrange(2)), hi)
            past_hi = rng.choice([_log(rng, 1, 100), _log(rng, 1, 4000), _log(rng, 100, 100000)])
            past = (past_hi // rng.choice([1, 2, 16]), past_hi)
            if op == "store":
                past = (min(past[0], 100), min(past[1], 100))
                if B * (q[1] + past[1]) * HK * D > _ELEMENTS:
                    continue
            S = past[1] + q[1]
            if H * B * q[1] * S > _SCORES or B * S * HK * D > _GATHER:
                continue
            c = _cached("", op, kind, B, q, past, H, HK, D, rng.randrange(1 << 20), rng.random() < 0.6,
                        rng.random() < 0.3, op == "attention" and rng.random() < 0.5)
        del c["name"]
        return c


def _sizes(case):
    """(new tokens, tokens already cached) of every sequence."""
    rng = random.Random(case["lengths"])
    T = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    past = [rng.randint(case["past_lo"], case["past_hi"]) for _ in range(case["B"])]
    if case["gaps"] and case["B"] > 2:
        for b in (0, case["B"] // 2, case["B"] - 1):
            T[b] = 0
    if sum(T) == 0:
        T[-1] = 1
    return T, past


# ---- inputs --------------------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rng = random.Random(seed)
    dt = TYPES[case["type"]]

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=gen, device=dev, dtype=dtype)

    def ints(v, dtype=torch.int32):
        return torch.tensor(v, dtype=dtype, device=dev)

    if case["op"] == "residual":
        N, C = case["N"], case["C"]
        s = dict(case=case, x=normal(N, C), residual=3 * normal(N, C, dtype=TYPES[case["stream"]]),
                 weight=1 + 0.2 * normal(C, dtype=torch.float32), post_weight=None, channel_scale=None, scale=0.7)
        if case["post"]:
            s["post_weight"] = 1 + 0.2 * normal(C, dtype=torch.float32)
        if case["channels"]:
            s["channel_scale"] = 0.1 + 0.05 * normal(C, dtype=torch.float32)
        s["out"], s["residual_out"] = torch.empty_like(s["x"]), torch.empty_like(s["residual"])
        return s
    if case["op"] == "gated":
        N, H, V = case["N"], case["H"], case["V"]
        s = dict(case=case, x=normal(N, H, V), weight=1 + 0.2 * normal(V, dtype=torch.float32))
        if case["packed"]:  # the gate is the last part of the projection's packed row
            s["gate"] = normal(N, (H + 1) * V)[:, V:].unflatten(1, (H, V))
        else:
            s["gate"] = normal(N, H, V)
        s["out"] = torch.empty((N, H, V), dtype=dt, device=dev)
        return s

    T, past = _sizes(case)
    B, N, H, HK, D = case["B"], sum(T), case["H"], case["HK"], case["D"]
    offsets = [0]
    for t in T:
        offsets.append(offsets[-1] + t)
    # every sequence owns a run of the cache's rows, in no order
    kv_len = [p + t for p, t in zip(past, T)]
    order = list(range(B))
    rng.shuffle(order)
    begin, rows = [0] * B, 0
    for b in order:
        begin[b] = rows
        rows += kv_len[b]
    s = dict(case=case, T=T, N=N, offsets=ints(offsets), kv_begin=ints(begin, torch.int64), kv_len=ints(kv_len),
             past=ints(past), longest_q=max(T), longest_kv=max(kv_len), rows=rows)

    def held(width):
        if case["heads_major"]:
            return torch.empty((HK, rows, width), dtype=torch.uint8, device=dev).permute(1, 0, 2)
        return torch.empty((rows, HK, width), dtype=torch.uint8, device=dev)

    # the cache as earlier steps left it: four tensors, codes and powers of the keys and of the values
    cache = []
    step = max(1, (1 << 27) // (HK * D))
    for _ in range(2):
        codes, powers = held(D // 2), held(D // BLOCK)
        for r in range(0, rows, step):
            n = min(step, rows - r)
            codes[r : r + n], powers[r : r + n] = _to_fp4(normal(n, HK, D), case["type"])
        cache += [codes, powers]
    s["cache"] = tuple(cache)
    if case["op"] == "store":
        row = normal(N, (H + 2 * HK) * D)  # the values are a part of the projection's packed row, the keys are not
        s["k"], s["v"] = normal(N, HK, D), row[:, (H + HK) * D :].view(N, HK, D)
        s["whole"], s["first"] = ints([0, rows]), ints([0], torch.int64)
    else:
        s["q"] = 1.5 * normal(N, H, D)  # normed and weighted queries: some rows attend sharply
    return s


# ---- one pass ------------------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if not own:
        return {"residual": _plain_residual, "gated": _plain_gated, "store": _plain_store,
                "attention": _plain_attention}[case["op"]](s)
    import gated_delta_rule_varlen_amd as gdn

    if case["op"] == "residual":
        return gdn.residual_norm(s["x"], s["residual"], weight=s["weight"], post_weight=s["post_weight"], scale=s["scale"],
                                 channel_scale=s["channel_scale"], eps=EPS, out=s["out"], residual_out=s["residual_out"])
    if case["op"] == "gated":
        return gdn.gated_norm(s["x"], s["gate"], weight=s["weight"], eps=EPS, activation=case["activation"],
                              gate_first=case["gate_first"], out=s["out"])
    if case["op"] == "store":
        gdn.cache_write_fp4_varlen(s["k"], s["v"], s["offsets"], cache=s["cache"], past=s["past"], kv_begin=s["kv_begin"])
        # what the whole cache stands for, as one run of its rows
        return gdn.cache_read_fp4_varlen(s["cache"], s["whole"], N=s["rows"], kv_begin=s["first"], dtype=s["k"].dtype)
    out = gdn.attention_fp4_varlen(s["q"], s["cache"], s["offsets"], kv_len=s["kv_len"], kv_begin=s["kv_begin"],
                                   max_q=s["longest_q"], return_lse=case["lse"])
    return out if case["lse"] else out[0]


def _to_fp4(x, kind):
    """(codes, powers) of x [..., D]: two codes a byte, the first in the low half, and a byte 127 + e for the block's 2^e."""
    lo, hi = POWERS[kind]
    y = x.float().unflatten(-1, (-1, BLOCK))
    top = y.abs().amax(-1)
    part, power = torch.frexp(top)  # top = part * 2^power, 1/2 <= part < 1
    e = torch.where(part > 0.75, power - 2, power - 3)  # the least e with top <= 6 * 2^e
    e = torch.where(top == 0, lo, e).clamp(lo, hi).int()
    y = y * ((127 - e) << 23).view(torch.float32)[..., None]  # times 2^-e, which is exact
    a = y.abs()
    # to the nearest value, a tie to the even code
    code = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).byte()
    code = (code | (torch.signbit(y).byte() << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).byte()


def _from_fp4(codes, powers):
    """The values of the codes, in 32 bits (exact)."""
    table = torch.tensor(VALUES + tuple(-x for x in VALUES), device=codes.device)
    y = table[torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).int()]
    return (y.unflatten(-1, (-1, BLOCK)) * (powers.int() << 23).view(torch.float32)[..., None]).flatten(-2)


def _normed(y, weight):
    return y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * weight


def _plain_residual(s):
    t = s["x"].float()
    if s["post_weight"] is not None:
        t = _normed(t, s["post_weight"])
    t = t * s["scale"]
    if s["channel_scale"] is not None:
        t = t * s["channel_scale"]
    h = s["residual"].float() + t
    s["out"].copy_(_normed(h, s["weight"]))
    s["residual_out"].copy_(h)
    return s["out"], s["residual_out"]


def _plain_gated(s):
    x, z = s["x"].float(), s["gate"].float()
    act = 1 / (1 + torch.exp(-z))
    if s["case"]["activation"] == "silu":
        act = act * z
    s["out"].copy_(_normed(x * act, s["weight"]) if s["case"]["gate_first"] else _normed(x, s["weight"]) * act)
    return s["out"]


def _token_places(s):
    """(sequence, index in the sequence) of every packed token."""
    off = s["offsets"].long()
    t = torch.arange(s["N"], device=off.device)
    b = torch.searchsorted(off, t, right=True) - 1
    return b, t - off[b]


def _plain_store(s):
    b, i = _token_places(s)
    row = s["kv_begin"][b] + s["past"].long()[b] + i
    kc, kp, vc, vp = s["cache"]
    kc[row], kp[row] = _to_fp4(s["k"], s["case"]["type"])
    vc[row], vp[row] = _to_fp4(s["v"], s["case"]["type"])
    return _from_fp4(kc, kp).to(s["k"].dtype), _from_fp4(vc, vp).to(s["k"].dtype)


def _plain_attention(s):
    case = s["case"]
    B, H, HK, D = case["B"], case["H"], case["HK"], case["D"]
    G, Tm, Sm, N = H // HK, s["longest_q"], s["longest_kv"], s["N"]
    dev = s["q"].device
    off, n_kv = s["offsets"].long(), s["kv_len"].long()
    T = off[1:] - off[:-1]
    i, j = torch.arange(Tm, device=dev), torch.arange(Sm, device=dev)
    kc, kp, vc, vp = s["cache"]
    # the batch padded to its longest query and its longest key run
    q = s["q"][(off[:-1, None] + i).clamp(max=N - 1)].float()  # [B, Tm, H, D]
    q = q.view(B, Tm, HK, G, D).permute(0, 2, 3, 1, 4).reshape(B, HK, G * Tm, D)
    at = (s["kv_begin"][:, None] + torch.minimum(j, (n_kv - 1).clamp(min=0)[:, None])).clamp(max=s["rows"] - 1)
    k = _from_fp4(kc[at], kp[at]).permute(0, 2, 3, 1).contiguous()  # [B, HK, D, Sm]
    scores = (q @ k).mul_(1 / math.sqrt(D)).view(B, HK, G, Tm, Sm)
    del k
    last = (n_kv - T)[:, None] + i  # [B, Tm]: the last key each query sees
    hidden = (j > last[..., None]) | (i >= T[:, None])[..., None]
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    v = _from_fp4(vc[at], vp[at]).permute(0, 2, 1, 3).contiguous()
    scores = scores.view(B, HK, G * Tm, Sm)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total, o = p.sum(-1, keepdim=True), p @ v
    b, t = _token_places(s)

    def packed(x):  # [B, HK, G * Tm, n] -> [N, H, n]
        return x.view(B, HK, G, Tm, -1).permute(0, 3, 1, 2, 4)[b, t].reshape(N, H, -1)

    top, total, o = packed(top), packed(total), packed(o)
    out = (o / torch.where(total == 0, 1.0, total)).to(s["q"].dtype)
    return (out, (top + total.log()).squeeze(-1)) if case["lse"] else out


# ---- what a pass cannot do without ---------------------------------------------------------------
def work(case):
    es = SIZE[case["type"]]
    if case["op"] == "residual":
        N, C = case["N"], case["C"]
        vectors = 1 + case["post"] + case["channels"]
        return {"bytes": 2 * N * C * (es + SIZE[case["stream"]]) + 4 * C * vectors,
                "flops": N * C * (6 + 3 * case["post"] + case["channels"])}
    if case["op"] == "gated":
        n = case["N"] * case["H"] * case["V"]
        return {"bytes": 3 * n * es + 4 * case["V"], "flops": 9 * n}
    T, past = _sizes(case)
    N, H, HK, D = sum(T), case["H"], case["HK"], case["D"]
    held = D // 2 + D // BLOCK  # bytes of a head's keys or values in the cache
    if case["op"] == "store":
        rows = N + sum(past)
        return {"bytes": 2 * HK * (N * (D * es + held) + rows * (held + D * es)) + case["B"] * 20,
                "flops": 2 * HK * D * (3 * N + rows)}
    keys = sum(p + t for p, t in zip(past, T) if t)
    pairs = sum(t * p + t * (t + 1) // 2 for p, t in zip(past, T))
    return {"bytes": 2 * N * H * D * es + 2 * keys * HK * held + (4 * N * H if case["lse"] else 0) + case["B"] * 16,
            "flops": 4 * D * H * pairs}


# ---- the definition in 64 bits -------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "residual":
        y = s["x"].double()
        if case["post"]:
            y = s["post_weight"].double() * y / torch.sqrt((y * y).sum(1, keepdim=True) / case["C"] + EPS)
        c = torch.full((case["C"],), s["scale"], dtype=torch.float64, device="cuda")
        if case["channels"]:
            c = c * s["channel_scale"].double()
        stream = torch.addcmul(s["residual"].double(), y, c[None, :])
        del y
        size = torch.linalg.vector_norm(stream, dim=1, keepdim=True).square() / case["C"]
        return stream * s["weight"].double() / torch.sqrt(size + EPS), stream
    if case["op"] == "gated":
        x, z = s["x"].double(), s["gate"].double()
        g = torch.sigmoid(z)
        if case["activation"] == "silu":
            g = z * g
        inner = x * g if case["gate_first"] else x
        size = torch.linalg.vector_norm(inner, dim=2, keepdim=True).square() / case["V"]
        y = inner * s["weight"].double() / torch.sqrt(size + EPS)
        return y if case["gate_first"] else y * g
    T, past = _sizes(case)
    start = [sum(T[:b]) for b in range(len(T) + 1)]
    begin = s["kv_begin"].tolist()
    if case["op"] == "store":
        k, v = (_exact_values(s["cache"][2 * x], s["cache"][2 * x + 1]) for x in range(2))
        for new, held in ((s["k"], k), (s["v"], v)):
            near = _exact_nearest(new.double(), POWERS[case["type"]])
            for b, t in enumerate(T):
                held[begin[b] + past[b] : begin[b] + past[b] + t] = near[start[b] : start[b + 1]]
        return k, v
    H, HK, D = case["H"], case["HK"], case["D"]
    G = H // HK
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, t in enumerate(T):
        if t == 0:
            continue
        run_ = slice(begin[b], begin[b] + past[b] + t)
        for h in range(HK):
            k, v = (_exact_values(s["cache"][2 * x][run_, h], s["cache"][2 * x + 1][run_, h]) for x in range(2))
            for a in range(0, t, 2048):  # a block of queries at a time
                e = min(t, a + 2048)
                seen = past[b] + e
                q = s["q"][start[b] + a : start[b] + e, h * G : (h + 1) * G].double()
                x = torch.tensordot(q, k[:seen], dims=([2], [1])) / math.sqrt(D)  # [e - a, G, seen]
                later = torch.arange(seen, device="cuda") > (past[b] + torch.arange(a, e, device="cuda"))[:, None]
                x = x.masked_fill(later[:, None, :], -math.inf)
                lse[start[b] + a : start[b] + e, h * G : (h + 1) * G] = torch.logsumexp(x, -1)
                out[start[b] + a : start[b] + e, h * G : (h + 1) * G] = torch.softmax(x, -1) @ v[:seen]
    return (out, lse) if case["lse"] else out


def _exact_values(codes, powers):
    """What codes and powers stand for, from the meaning of a code's bits: sign, two of exponent, one of fraction."""
    y = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.float64, device=codes.device)
    for half in range(2):
        c = (codes >> (4 * half)) & 15
        exponent, fraction = ((c >> 1) & 3).double(), (c & 1).double()
        size = torch.where(exponent == 0, 0.5 * fraction, torch.exp2(exponent - 1) * (1 + 0.5 * fraction))
        y[..., half::2] = torch.where(c >= 8, -size, size)
    return y * torch.exp2(powers.double() - 127).repeat_interleave(BLOCK, dim=-1)


def _exact_nearest(x, powers):
    """The nearest value of x [..., D] that its block of 32 can hold, ties to the even code."""
    y = x.reshape(*x.shape[:-1], -1, BLOCK)
    top = y.abs().amax(-1, keepdim=True)
    unit = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0**-200) / 6)))
    # the logarithm may be off by a little: the least power of two that holds the largest element
    unit = torch.where(top > 6 * unit, 2 * unit, torch.where(top <= 3 * unit, 0.5 * unit, unit))
    unit = unit.clamp(2.0 ** powers[0], 2.0 ** powers[1])
    size = (y / unit).abs()
    best = torch.zeros_like(size)
    for code in range(1, 8):
        middle = (VALUES[code - 1] + VALUES[code]) / 2
        best = torch.where(size >= middle if code % 2 == 0 else size > middle, VALUES[code], best)
    return (torch.copysign(best, y) * unit).reshape(x.shape)
