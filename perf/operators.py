"""What the softmax-attention operators of this package are measured on.

Three operators, the ones a softmax-attention layer needs beside the recurrent layers:

    qk_norm_rope_varlen        per-head RMS norm of q and k, rotary positions, and the write of the new
                               keys and values into the cache, in one pass
    attention_varlen           causal attention with grouped heads of packed sequences (whole prompts,
                               prompts continued over a cache, draft blocks, single tokens)
    attention_prefix_varlen    the same for a batch whose sequences all start with one shared prefix

`listed()` gives the cases, `draw(rng)` more of the same ranges, `prepare(case, seed)` their inputs on the
GPU, `run(state)` one pass (elementary torch operations in 32 bits, or the package's kernels where
`own` is true), `work(case)` the bytes and operations a pass cannot do without and `exact(case, seed)`
the result in 64 bits.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ---- cases ---------------------------------------------------------------------------------------
# Lengths are drawn from the case itself (`lengths` seeds them): `q_lo`..`q_hi` new tokens a sequence,
# `past_lo`..`past_hi` tokens already in the cache.  `gaps` makes the first, the middle and the last
# sequence empty.  `heads_major` keeps the cache as [heads, rows, D] instead of [rows, heads, D].
def _rope(name, kind, B, q, past, H, HK, D, rot, interleaved, far, lengths, gaps=False):
    return dict(name=name, op="rope", type=kind, B=B, q_lo=q[0], q_hi=q[1], past_lo=past[0], past_hi=past[1], H=H,
                HK=HK, D=D, rot=rot, interleaved=interleaved, far=far, lengths=lengths, gaps=gaps)


def _attn(name, kind, B, q, past, H, HK, D, lengths, prefix=0, heads_major=False, gaps=False, lse=False):
    return dict(name=name, op="prefix" if prefix else "attention", type=kind, B=B, q_lo=q[0], q_hi=q[1],
                past_lo=past[0], past_hi=past[1], H=H, HK=HK, D=D, prefix=prefix, heads_major=heads_major,
                lengths=lengths, gaps=gaps, lse=lse)


def listed():
    return [
        # one decode step of 64 sequences: a launch's latency counts, little is moved
        _rope("rope_decode", "bf16", 64, (1, 1), (0, 2047), 16, 2, 256, 64, False, 0, 11),
        # the prompts of a prefill batch, written to a fresh cache
        _rope("rope_prefill", "bf16", 8, (512, 4096), (0, 0), 32, 8, 128, 128, False, 0, 103),
        # ragged prompts with empty ones among them, neighbouring pairs rotated, far positions
        _rope("rope_ragged", "f16", 64, (0, 300), (0, 40), 16, 4, 64, 64, True, 1 << 20, 105, gaps=True),
        # the smallest call: one token of one conversation
        _attn("attn_single", "f16", 1, (1, 1), (1022, 1022), 16, 4, 64, 21),
        # one token of one sequence over a very long cache
        _attn("attn_long_cache", "bf16", 1, (1, 1), (131071, 131071), 16, 2, 256, 22),
        # a decode step of a full batch with contexts of every length
        _attn("attn_decode", "bf16", 256, (1, 1), (0, 4095), 32, 8, 128, 102),
        # a verification step: four drafted tokens and the last accepted one, per sequence
        _attn("attn_verify", "bf16", 64, (5, 5), (1000, 8000), 16, 2, 256, 24, heads_major=True),
        # the prompts of a prefill batch
        _attn("attn_prefill", "bf16", 8, (512, 4096), (0, 0), 32, 8, 128, 103),
        # one long prompt
        _attn("attn_long_prompt", "bf16", 1, (16384, 16384), (0, 0), 16, 2, 256, 104),
        # prompts continued over what the cache holds, in single precision, empty ones among them
        _attn("attn_ragged_f32", "f32", 64, (0, 300), (0, 1000), 16, 4, 64, 105, gaps=True, lse=True),
        # a decode step of a batch that shares a long system prompt
        _attn("prefix_decode", "bf16", 256, (1, 1), (0, 511), 32, 8, 128, 31, prefix=8192),
        # a few short drafts behind a shared prompt of odd length
        _attn("prefix_small", "f16", 8, (1, 4), (0, 90), 16, 4, 64, 32, prefix=1001, lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# No drawn case moves or computes more than these (all of them below the largest listed case's).
_SCORES = 3 << 30    # H * B * longest query * longest key: the plain form's score matrix
_GATHER = 1 << 30    # B * longest key * HK * D: the plain form's padded keys
_TOKENS = 1 << 27    # rotated elements


def draw(rng):
    while True:
        op = rng.choice(["rope", "attention", "attention", "prefix"])
        kind = rng.choice(["bf16", "bf16", "f16", "f32"])
        HK = rng.choice([1, 2, 3, 4, 8])
        H = HK * rng.choice([1, 2, 3, 4, 5, 8, 16])
        D = rng.choice([64, 128, 256, 64, 128, 256, 32, 72, 80, 96, 192])
        lengths = rng.randrange(1 << 20)
        gaps = rng.random() < 0.3
        form = rng.choice(["token", "block", "prompt"])
        if op == "prefix" and form == "prompt":
            form = rng.choice(["token", "block"])
        if form == "token":
            B, q = _log(rng, 1, 256), (1, 1)
        elif form == "block":
            hi = rng.randrange(2, 10)
            B, q = _log(rng, 1, 96), (rng.randrange(1, hi), hi)
        else:
            hi = _log(rng, 16, 8192)
            B, q = _log(rng, 1, 64), (max(0, hi // rng.choice([1, 2, 8]) - rng.randrange(2)), hi)
        past_hi = rng.choice([0 if form == "prompt" else _log(rng, 1, 100), _log(rng, 1, 4000), _log(rng, 100, 100000)])
        past = (past_hi // rng.choice([1, 2, 16]), past_hi)
        if op == "rope":
            past = (min(past[0], 100), min(past[1], 100))
            if B * q[1] * (H + 2 * HK) * D > _TOKENS:
                continue
            rot = rng.choice([D, D // 2, 2 * rng.randrange(1, D // 2 + 1)])
            c = _rope("", kind, B, q, past, H, HK, D, rot, rng.random() < 0.4, rng.choice([0, 1 << 12, 1 << 22]), lengths,
                      gaps)
        else:
            prefix = _log(rng, 16, 16384) if op == "prefix" else 0
            if op == "prefix":
                past = (min(past[0], 2000), min(past[1], 2000))
            S = past[1] + q[1]
            if H * B * q[1] * (S + prefix) > _SCORES or B * S * HK * D > _GATHER:
                continue
            c = _attn("", kind, B, q, past, H, HK, D, lengths, prefix=prefix, heads_major=rng.random() < 0.4, gaps=gaps,
                      lse=rng.random() < 0.5)
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
    T, past = _sizes(case)
    B, N, H, HK, D = case["B"], sum(T), case["H"], case["HK"], case["D"]

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=gen, device=dev, dtype=dtype)

    def ints(v, dtype=torch.int32):
        return torch.tensor(v, dtype=dtype, device=dev)

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
    s = dict(case=case, T=T, N=N, offsets=ints(offsets), kv_begin=ints(begin, torch.int64), longest_q=max(T),
             longest_kv=max(kv_len))
    if case["op"] == "rope":
        # q, k and v are parts of the projection's packed row
        row = normal(N, (H + 2 * HK) * D)
        s["q"] = row[:, : H * D].view(N, H, D)
        s["k"] = row[:, H * D : (H + HK) * D].view(N, HK, D)
        s["v"] = row[:, (H + HK) * D :].view(N, HK, D)
        s["q_weight"] = 1 + 0.2 * normal(D, dtype=torch.float32)
        s["k_weight"] = 1 + 0.2 * normal(D, dtype=torch.float32)
        i = torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64)
        s["inv_freq"] = (1e6 ** (-i / case["rot"])).float()
        s["past"] = ints(past)
        s["positions"] = ints([p + (rng.randrange(case["far"]) if case["far"] else 0) for p in past])
        s["q_out"] = torch.empty((N, H, D), dtype=dt, device=dev)
        s["k_cache"], s["v_cache"] = normal(rows, HK, D), normal(rows, HK, D)
        return s
    s["q"] = 1.5 * normal(N, H, D)  # normed and weighted queries: some rows attend sharply
    s["kv_len"] = ints(kv_len)
    for n in ("k", "v"):
        s[n] = normal(HK, rows, D).permute(1, 0, 2) if case["heads_major"] else normal(rows, HK, D)
        if case["op"] == "prefix":
            s["prefix_" + n] = normal(case["prefix"], HK, D)
    return s


# ---- one pass ------------------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if case["op"] == "rope":
        if own:
            import gated_delta_rule_varlen_amd as gdn

            return gdn.qk_norm_rope_varlen(s["q"], s["k"], s["v"], s["offsets"], inv_freq=s["inv_freq"],
                                           q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6,
                                           interleaved=case["interleaved"], past=s["past"], positions=s["positions"],
                                           kv_begin=s["kv_begin"], q_out=s["q_out"], k_out=s["k_cache"],
                                           v_out=s["v_cache"])
        return _plain_rope(s)
    if own:
        import gated_delta_rule_varlen_amd as gdn

        if case["op"] == "prefix":
            out = gdn.attention_prefix_varlen(s["q"], s["prefix_k"], s["prefix_v"], s["k"], s["v"], s["offsets"],
                                              kv_len=s["kv_len"], kv_begin=s["kv_begin"], max_q=s["longest_q"],
                                              return_lse=case["lse"])
        else:
            out = gdn.attention_varlen(s["q"], s["k"], s["v"], s["offsets"], kv_len=s["kv_len"],
                                       kv_begin=s["kv_begin"], max_q=s["longest_q"], return_lse=case["lse"])
        return out if case["lse"] else out[0]
    return _plain_attention(s)


def _token_places(s):
    """(sequence, index in the sequence) of every packed token."""
    off = s["offsets"].long()
    t = torch.arange(s["N"], device=off.device)
    b = torch.searchsorted(off, t, right=True) - 1
    return b, t - off[b]


def _plain_rope(s):
    case = s["case"]
    rot = case["rot"]
    b, i = _token_places(s)
    angle = (s["positions"].long()[b] + i).double()[:, None] * s["inv_freq"].double()  # 64 bits: far positions
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]

    def norm_rotate(x, weight):
        y = x.float()
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight
        if case["interleaved"]:
            lo, hi = y[..., 0:rot:2], y[..., 1:rot:2]
            turned = torch.stack((lo * cos - hi * sin, lo * sin + hi * cos), dim=-1).flatten(-2)
        else:
            lo, hi = y[..., : rot // 2], y[..., rot // 2 : rot]
            turned = torch.cat((lo * cos - hi * sin, lo * sin + hi * cos), dim=-1)
        return torch.cat((turned, y[..., rot:]), dim=-1).to(x.dtype)

    row = s["kv_begin"][b] + s["past"].long()[b] + i
    s["q_out"].copy_(norm_rotate(s["q"], s["q_weight"]))
    s["k_cache"][row] = norm_rotate(s["k"], s["k_weight"])
    s["v_cache"][row] = s["v"]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _softmax_parts(scores, v):
    """Largest score, sum of exponentials and their product with v, of rows that may be empty."""
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    return top, p.sum(-1, keepdim=True), p @ v


def _plain_attention(s):
    case = s["case"]
    B, H, HK, D = case["B"], case["H"], case["HK"], case["D"]
    G, Tm, Sm, N = H // HK, s["longest_q"], s["longest_kv"], s["N"]
    scale = 1 / math.sqrt(D)
    dev = s["q"].device
    off, n_kv = s["offsets"].long(), s["kv_len"].long()
    T = off[1:] - off[:-1]
    i, j = torch.arange(Tm, device=dev), torch.arange(Sm, device=dev)
    # the batch padded to its longest query and its longest key run
    q = s["q"][(off[:-1, None] + i).clamp(max=N - 1)].float()  # [B, Tm, H, D]
    q = q.view(B, Tm, HK, G, D).permute(0, 2, 3, 1, 4).reshape(B, HK, G * Tm, D)
    at = (s["kv_begin"][:, None] + torch.minimum(j, (n_kv - 1).clamp(min=0)[:, None])).clamp(max=len(s["k"]) - 1)
    k = s["k"][at].float().permute(0, 2, 3, 1).contiguous()  # [B, HK, D, Sm]
    scores = (q @ k).mul_(scale).view(B, HK, G, Tm, Sm)
    del k
    last = (n_kv - T)[:, None] + i  # [B, Tm]: the last key each query sees
    hidden = (j > last[..., None]) | (i >= T[:, None])[..., None]
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    v = s["v"][at].float().permute(0, 2, 1, 3).contiguous()
    top, total, o = _softmax_parts(scores.view(B, HK, G * Tm, Sm), v)
    b, t = _token_places(s)

    def packed(x):  # [B, HK, G * Tm, n] -> [N, H, n]
        return x.view(B, HK, G, Tm, -1).permute(0, 3, 1, 2, 4)[b, t].reshape(N, H, -1)

    top, total, o = packed(top), packed(total), packed(o)
    if case["op"] == "prefix":
        # every token against the shared prefix at once
        qp = s["q"].float().view(N, HK, G, D).permute(1, 0, 2, 3).reshape(HK, N * G, D)
        ps = (qp @ s["prefix_k"].float().permute(1, 2, 0).contiguous()).mul_(scale)
        ptop, ptotal, po = _softmax_parts(ps, s["prefix_v"].float().permute(1, 0, 2).contiguous())
        ptop, ptotal, po = (x.view(HK, N, G, -1).permute(1, 0, 2, 3).reshape(N, H, -1) for x in (ptop, ptotal, po))
        both = torch.maximum(top, ptop)
        w, pw = (top - both).exp(), (ptop - both).exp()
        top, total, o = both, total * w + ptotal * pw, o * w + po * pw
    out = (o / torch.where(total == 0, 1.0, total)).to(s["q"].dtype)
    return (out, (top + total.log()).squeeze(-1)) if case["lse"] else out


# ---- what a pass cannot do without ---------------------------------------------------------------
def work(case):
    T, past = _sizes(case)
    N, H, HK, D, es = sum(T), case["H"], case["HK"], case["D"], SIZE[case["type"]]
    if case["op"] == "rope":
        return {"bytes": 2 * N * (H + 2 * HK) * D * es + 2 * D * 4 + case["rot"] * 2 + case["B"] * 20,
                "flops": N * (H + HK) * (4 * D + 3 * case["rot"])}
    keys = sum(p + t for p, t in zip(past, T) if t) + case["prefix"]
    pairs = sum(t * (p + case["prefix"]) + t * (t + 1) // 2 for p, t in zip(past, T))
    return {"bytes": 2 * N * H * D * es + 2 * keys * HK * D * es + (4 * N * H if case["lse"] else 0) + case["B"] * 16,
            "flops": 4 * D * H * pairs}


# ---- the definition in 64 bits -------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    T, past = _sizes(case)
    start = [sum(T[:b]) for b in range(len(T) + 1)]
    begin = s["kv_begin"].tolist()
    if case["op"] == "rope":
        return _exact_rope(case, s, T, past, start, begin)
    H, HK, D, P = case["H"], case["HK"], case["D"], case["prefix"]
    G = H // HK
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, t in enumerate(T):
        if t == 0:
            continue
        n = past[b] + t
        for h in range(HK):
            k, v = (s[x][begin[b] : begin[b] + n, h].double() for x in ("k", "v"))
            if P:
                k, v = (torch.cat((s["prefix_" + x][:, h].double(), y)) for x, y in (("k", k), ("v", v)))
            for a in range(0, t, 2048):  # a block of queries at a time
                e = min(t, a + 2048)
                seen = P + past[b] + e
                q = s["q"][start[b] + a : start[b] + e, h * G : (h + 1) * G].double()
                x = torch.tensordot(q, k[:seen], dims=([2], [1])) / math.sqrt(D)  # [e - a, G, seen]
                later = torch.arange(seen, device="cuda") > (P + past[b] + torch.arange(a, e, device="cuda"))[:, None]
                x = x.masked_fill(later[:, None, :], -math.inf)
                lse[start[b] + a : start[b] + e, h * G : (h + 1) * G] = torch.logsumexp(x, -1)
                out[start[b] + a : start[b] + e, h * G : (h + 1) * G] = torch.softmax(x, -1) @ v[:seen]
    return (out, lse) if case["lse"] else out


def _exact_rope(case, s, T, past, start, begin):
    rot, half = case["rot"], case["rot"] // 2
    first = s["positions"].tolist()
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    q_out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    # element i of a rotated pair's place, and its partner's
    pair = torch.arange(half, device="cuda")
    one, two = (2 * pair, 2 * pair + 1) if case["interleaved"] else (pair, pair + half)
    for b, t in enumerate(T):
        if t == 0:
            continue
        pos = torch.arange(first[b], first[b] + t, device="cuda", dtype=torch.float64)
        turn = torch.polar(torch.ones((t, half), dtype=torch.float64, device="cuda"),
                           pos[:, None] * s["inv_freq"].double()[None, :])
        for name, w in (("q", s["q_weight"]), ("k", s["k_weight"])):
            x = s[name][start[b] : start[b] + t].double()
            x = w.double() * x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["D"] + 1e-6)
            z = torch.complex(x[..., one].contiguous(), x[..., two].contiguous()) * turn[:, None, :]
            x[..., one], x[..., two] = z.real, z.imag
            if name == "q":
                q_out[start[b] : start[b] + t] = x
            else:
                k_cache[begin[b] + past[b] : begin[b] + past[b] + t] = x
        v_cache[begin[b] + past[b] : begin[b] + past[b] + t] = s["v"][start[b] : start[b] + t].double()
    return q_out, k_cache, v_cache
