"""Timed cases of the prompt side's operators: rotary positions, the RMS norm with the residual's
addition (bf16/fp16 or 8-bit outputs with scales) and attention over packed prompts and caches.

`own` false: each operator in its plain form, elementary torch operations in 32 bits (angles in 64),
rounded once at the end.  `own` true: the calls a user makes of the package.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_E4M3 = torch.float8_e4m3fn
_E4M3_MOST = 448.0
_LEAST_AMAX = 2.0 ** -100  # an all-zero row or group still gets a positive scale
_GROUP = 128


# ------------------------------------------------------------------------------------- cases

def _rope(tokens, heads, kv_heads, head_dim, rotary, interleaved, scaling, factor, reach, dtype, fused):
    return {"op": "rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "rotary": rotary,
            "interleaved": interleaved, "scaling": scaling, "factor": factor, "reach": reach, "type": dtype, "fused": fused}


def _norm(rows, width, scales, residual, dtype):
    return {"op": "norm", "rows": rows, "width": width, "scales": scales, "residual": residual, "type": dtype}


def _attend(kind, count, longest, cached, heads, kv_heads, head_dim, dtype, lse, mix):
    return {"op": "attend", "kind": kind, "count": count, "longest": longest, "cached": cached, "heads": heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "type": dtype, "lse": lse, "mix": mix}


def listed():
    named = {
        # one new token for each of 16 requests, whole heads rotated: a serving step, latency counts
        "rope_single_tokens": _rope(16, 32, 8, 128, 128, False, "none", 1.0, 8192, "bf16", False),
        # a packed batch of long prompts whose positions go past the trained length
        "rope_prompts_scaled": _rope(8192, 32, 8, 128, 128, False, "parts", 8.0, 131072, "bf16", False),
        # half of each 96-wide head rotated, neighbouring pairs, q and k as slices of one fused projection
        "rope_part_interleaved": _rope(30011, 28, 4, 96, 48, True, "linear", 4.0, 65536, "fp16", True),
        # a serving step's rows at the hidden width, straight to 8 bits with one scale a row
        "norm_single_tokens": _norm(8, 5376, "row", True, "bf16"),
        # an odd number of rows of a width that is no multiple of a warp's vectors, 16-bit output
        "norm_odd_rows": _norm(1023, 2000, "none", True, "fp16"),
        # a prompt batch, one scale for each 128 channels
        "norm_prompt_groups": _norm(8192, 4096, "group", True, "bf16"),
        # every token of a five-second clip at the hidden width, one scale a row
        "norm_clip_rows": _norm(124992, 5376, "row", True, "bf16"),
        # two dozen short prompts packed behind one another, grouped heads, views of a fused projection
        "attend_short_prompts": _attend("prompts", 24, 300, 0, 32, 8, 128, "bf16", False, 1),
        # one long prompt
        "attend_long_prompt": _attend("prompts", 1, 16384, 0, 32, 8, 128, "bf16", False, 1),
        # pieces of three prompts against what is cached of them, seven heads a group, with log-sum-exps
        "attend_chunks": _attend("chunks", 3, 509, 12000, 28, 4, 96, "bf16", True, 2),
        # single tokens over short caches, every head its own keys: latency counts
        "attend_single_short": _attend("single", 8, 1, 900, 16, 16, 64, "fp16", False, 3),
        # single tokens over long ragged caches kept with one capacity for all
        "attend_single_long": _attend("single", 47, 1, 16384, 32, 8, 128, "bf16", False, 4),
    }
    return [dict(c, name=name) for name, c in named.items()]


def _spread(rng, lo, hi):
    """Log-uniform whole number of [lo, hi]."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rope", "norm", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "rope":
        head_dim = rng.choice([64, 96, 128])
        kv = rng.choice([1, 2, 4, 8])
        return _rope(_spread(rng, 1, 40000), kv * rng.randint(1, 8), kv, head_dim, 2 * rng.randint(8, head_dim // 2),
                     rng.random() < 0.5, rng.choice(["none", "linear", "base", "parts"]), rng.choice([2.0, 4.0, 8.0]),
                     _spread(rng, 1000, 1000000), dtype, rng.random() < 0.5)
    if op == "norm":
        return _norm(_spread(rng, 1, 60000), 8 * _spread(rng, 8, 1024), rng.choice(["none", "row", "group"]),
                     rng.random() < 0.8, dtype)
    head_dim = rng.choice([64, 96, 128])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 7, 8])
    kind = rng.choice(["prompts", "chunks", "single"])
    lse, mix = rng.random() < 0.3, rng.randint(1, 1 << 20)
    most = 16384 * 16384 * 32 // (2 * heads)  # pairs of (query, key) that the plain form may hold for one head
    if kind == "single":
        cached = _spread(rng, 16, 16384)
        return _attend(kind, min(_spread(rng, 1, 64), max(1, (1 << 29) // (cached * kv * head_dim))), 1, cached, heads,
                       kv, head_dim, dtype, lse, mix)
    longest = _spread(rng, 16, 6000 if kind == "prompts" else 1024)
    cached = 0 if kind == "prompts" else _spread(rng, 16, 12000)
    count = min(_spread(rng, 1, 32), max(1, most // (longest * (longest + cached))))
    return _attend(kind, count, longest, cached, heads, kv, head_dim, dtype, lse, mix)


def _ragged(count, longest, rng):
    """`count` lengths from 1 to `longest`, the longest among them, many short and few long."""
    got = [max(1, int(longest * rng.random() ** 2)) for _ in range(count - 1)] + [longest]
    rng.shuffle(got)
    return got


def _lengths(case):
    """(queries, keys) of each sequence: whole numbers that a serving program knows when it plans the step."""
    rng = random.Random(case["mix"])
    if case["kind"] == "single":
        return [1] * case["count"], _ragged(case["count"], case["cached"], rng)
    queries = _ragged(case["count"], case["longest"], rng)
    if case["kind"] == "prompts":
        return queries, list(queries)
    return queries, [n + c for n, c in zip(queries, _ragged(case["count"], case["cached"], rng))]


# ------------------------------------------------------------------------------------- inputs

def _starts(lengths):
    total = [0]
    for n in lengths:
        total.append(total[-1] + n)
    return torch.tensor(total, dtype=torch.int32, device="cuda")


def _sequences(case):
    """Shapes and the device's index arrays: starts of queries and of keys, keys in use of each sequence."""
    lq, lk = _lengths(case)
    state = {"starts_q": _starts(lq), "max_q": max(lq), "max_k": max(lk), "tokens": sum(lq), "lengths_k": None}
    if case["kind"] == "single":  # a cache with one capacity for all: keys start at its multiples
        room = -(-case["cached"] // 64) * 64
        state |= {"rows_k": room * case["count"], "starts_k": _starts([room] * case["count"]),
                  "lengths_k": torch.tensor(lk, dtype=torch.int32, device="cuda")}
    else:
        state |= {"rows_k": sum(lk), "starts_k": _starts(lk)}
    return state


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = _TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    state = dict(case)
    if case["op"] == "rope":
        n, h, kv, d = (case[x] for x in ("tokens", "heads", "kv_heads", "head_dim"))
        if case["fused"]:
            qkv = normal(n, h + 2 * kv, d)
            state |= {"q": qkv[:, :h], "k": qkv[:, h:h + kv]}
        else:
            state |= {"q": normal(n, h, d), "k": normal(n, kv, d)}
        state["positions"] = torch.randint(0, case["reach"], (n,), generator=g, device="cuda", dtype=torch.int32)
    elif case["op"] == "norm":
        n, c = case["rows"], case["width"]
        # a residual stream: rows of unlike size, some channels far larger than the others
        big = 1.0 + 20.0 * (torch.rand(c, generator=g, device="cuda") < 0.01)
        state["x"] = torch.empty(n, c, device="cuda", dtype=dtype)
        for i in range(0, n, 16384):
            part = state["x"][i:i + 16384]
            part.copy_(torch.randn(part.shape, generator=g, device="cuda") * big * (0.5 + torch.rand(len(part), 1, generator=g, device="cuda")))
        state["f"] = normal(n, c) if case["residual"] else None
        state["gamma"] = 1.0 + 0.1 * torch.randn(c, generator=g, device="cuda")
    else:
        state |= _sequences(case)
        h, kv, d = (case[x] for x in ("heads", "kv_heads", "head_dim"))
        if case["kind"] == "prompts":
            qkv = normal(state["tokens"], h + 2 * kv, d)
            state |= {"q": qkv[:, :h], "k": qkv[:, h:h + kv], "v": qkv[:, h + kv:]}
        else:
            state |= {"q": normal(state["tokens"], h, d), "k": normal(state["rows_k"], kv, d), "v": normal(state["rows_k"], kv, d)}
    return state


# ------------------------------------------------------------------------------------- one pass

_THETA = 500000.0
_TRAINED = 8192  # length that scaled positions were trained with
_SLOW, _FAST = 1.0, 32.0  # turns over the trained length: below, a frequency is divided; above, it is kept
_EPS = 1e-6


def run(state):
    if not own:
        return {"rope": _plain_rope, "norm": _plain_norm, "attend": _plain_attend}[state["op"]](state)
    import rope_block_sparse_b200 as h3a

    if state["op"] == "rope":
        plan = h3a.rope_plan(state["rotary"], _THETA, interleaved=state["interleaved"], scaling=state["scaling"],
                             factor=state["factor"], original_length=_TRAINED, low_turns=_SLOW, high_turns=_FAST)
        return h3a.rope(state["q"], state["k"], state["positions"], plan)
    if state["op"] == "norm":
        scales = None if state["scales"] == "none" else state["scales"]
        h, y, s = h3a.residual_rmsnorm(state["x"], state["f"], state["gamma"], _EPS, scales=scales)
        return _norm_outputs(h, y, s)
    return h3a.packed_attention(state["q"], state["k"], state["v"], state["starts_q"], state["starts_k"], state["max_q"],
                                state["max_k"], lengths_k=state["lengths_k"], return_lse=state["lse"])


def _norm_outputs(h, y, s):
    return {name: t for name, t in (("h", h), ("y", y), ("s", s)) if t is not None}


def _plain_frequencies(state):
    r = state["rotary"]
    theta = _THETA
    if state["scaling"] == "base" and r > 2:
        theta *= state["factor"] ** (r / (r - 2))
    f = theta ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)
    if state["scaling"] == "linear":
        f = f / state["factor"]
    if state["scaling"] == "parts":
        keep = ((_TRAINED * f / (2 * math.pi) - _SLOW) / (_FAST - _SLOW)).clamp(0, 1)
        f = f * (keep + (1 - keep) / state["factor"])
    return f


def _plain_rope(state):
    r = state["rotary"]
    angle = state["positions"].double()[:, None] * _plain_frequencies(state)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x):
        y = x.float()
        if state["interleaved"]:
            a, b = y[..., 0:r:2], y[..., 1:r:2]
            y[..., :r] = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        else:
            a, b = y[..., :r // 2], y[..., r // 2:r]
            y[..., :r] = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        return y.to(x.dtype)

    return turned(state["q"]), turned(state["k"])


def _plain_norm(state):
    x, f = state["x"], state["f"]
    h = x if f is None else (x.float() + f.float()).to(x.dtype)
    y = h.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + _EPS) * state["gamma"]
    new_h = None if f is None else h
    if state["scales"] == "none":
        return _norm_outputs(new_h, y.to(x.dtype), None)
    if state["scales"] == "row":
        s = y.abs().amax(-1, keepdim=True).clamp_min(_LEAST_AMAX) / _E4M3_MOST
        return _norm_outputs(new_h, (y / s).clamp(-_E4M3_MOST, _E4M3_MOST).to(_E4M3), s[:, 0])
    n, c = y.shape
    groups = -(-c // _GROUP)
    wide = torch.nn.functional.pad(y, (0, groups * _GROUP - c)).view(n, groups, _GROUP)
    s = wide.abs().amax(-1, keepdim=True).clamp_min(_LEAST_AMAX) / _E4M3_MOST
    y8 = (wide / s).clamp(-_E4M3_MOST, _E4M3_MOST).to(_E4M3).view(n, groups * _GROUP)[:, :c]
    return _norm_outputs(new_h, y8.contiguous(), s[..., 0])


def _plain_attend(state):
    q, k, v = state["q"], state["k"], state["v"]
    h, kv, d = (state[x] for x in ("heads", "kv_heads", "head_dim"))
    first_q, first_k = state["starts_q"][:-1].long(), state["starts_k"][:-1].long()
    lq = state["starts_q"].diff().long()
    lk = state["starts_k"].diff().long() if state["lengths_k"] is None else state["lengths_k"].long()
    i, j = torch.arange(state["max_q"], device="cuda"), torch.arange(state["max_k"], device="cuda")
    at_q = (first_q[:, None] + i).clamp_(max=len(q) - 1)
    at_k = (first_k[:, None] + j).clamp_(max=len(k) - 1)
    count, nq, nk = len(lq), len(i), len(j)
    qs = q[at_q].float().view(count, nq, kv, h // kv, d).permute(0, 2, 3, 1, 4).reshape(count, kv, -1, d)
    p = torch.matmul(qs * d ** -0.5, k[at_k].float().permute(0, 2, 3, 1)).view(count, h, nq, nk)
    # key j is seen by query i of its sequence where j <= i + (keys - queries)
    last = torch.minimum(lk[:, None] - 1, i + (lk - lq)[:, None])
    p.masked_fill_((j > last[:, :, None])[:, None], -math.inf)
    top = p.amax(-1, keepdim=True).nan_to_num_(neginf=0.0)
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(count, kv, -1, nk), v[at_k].float().transpose(1, 2)).view(count, h, nq, d)
    o = o / total.masked_fill(total == 0, 1.0)
    # back to packed rows
    row = torch.arange(len(q), device="cuda")
    seq = torch.searchsorted(state["starts_q"].long(), row, right=True) - 1
    o = o[seq, :, row - first_q[seq]].to(q.dtype)
    if not state["lse"]:
        return o
    return o, (top + total.log())[seq, :, row - first_q[seq], 0]


# ------------------------------------------------------------------------------------- what it costs

def _pairs(lq, lk):
    """(query, key) pairs under the causal rule aligned at the last key."""
    full = sum(max(0, min(n, m)) * m for n, m in zip(lq, lk))
    return full - sum(min(n, m) * (min(n, m) - 1) // 2 for n, m in zip(lq, lk))


def work(case):
    if case["op"] == "rope":
        values = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["head_dim"]
        turned = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["rotary"]
        return {"bytes": 4 * values + 4 * case["tokens"], "flops": 3 * turned}
    if case["op"] == "norm":
        n, c = case["rows"], case["width"]
        scales = {"none": 0, "row": n, "group": n * -(-c // _GROUP)}[case["scales"]]
        out = 2 if case["scales"] == "none" else 1
        return {"bytes": n * c * (2 + out + (4 if case["residual"] else 0)) + 4 * c + 4 * scales, "flops": 6 * n * c}
    lq, lk = _lengths(case)
    h, kv, d = (case[x] for x in ("heads", "kv_heads", "head_dim"))
    return {"bytes": 4 * sum(lq) * h * d + 4 * sum(lk) * kv * d + (4 * sum(lq) * h if case["lse"] else 0),
            "flops": 4 * d * h * _pairs(lq, lk)}


# ------------------------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(state)
    if case["op"] == "norm":
        return _exact_norm(state)
    return _exact_attend(state)


def _exact_rope(state):
    r, s = state["rotary"], state["factor"]
    turns = []
    for pair in range(r // 2):
        theta = _THETA * s ** (r / (r - 2)) if state["scaling"] == "base" and r > 2 else _THETA
        f = 1.0 / theta ** (2 * pair / r)
        if state["scaling"] == "linear":
            f /= s
        elif state["scaling"] == "parts":
            n = _TRAINED * f / (2 * math.pi)
            w = 0.0 if n < _SLOW else 1.0 if n > _FAST else (n - _SLOW) / (_FAST - _SLOW)
            f = (1 - w) * f / s + w * f
        turns.append(f)
    angle = state["positions"].double().unsqueeze(1) * torch.tensor(turns, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
    pairs = [(2 * p, 2 * p + 1) if state["interleaved"] else (p, p + r // 2) for p in range(r // 2)]
    re, im = (torch.tensor(x, device="cuda") for x in zip(*pairs))
    got = []
    for x in (state["q"], state["k"]):
        y = x.double()
        z = torch.complex(y[:, :, re], y[:, :, im]) * turn
        y[:, :, re], y[:, :, im] = z.real, z.imag
        got.append(y)
    return tuple(got)


def _exact_norm(state):
    x, c = state["x"], state["width"]
    got = {"h": [], "y": [], "s": []}
    for i in range(0, len(x), 8192):
        h = x[i:i + 8192].double()
        if state["f"] is not None:
            h = (h + state["f"][i:i + 8192].double()).to(x.dtype)  # the sum of two such values fits 64 bits
            got["h"].append(h)
            h = h.double()
        y = h / (h.pow(2).sum(1, keepdim=True) / c + _EPS).sqrt() * state["gamma"].double()
        if state["scales"] == "none":
            got["y"].append(y)
            continue
        step = c if state["scales"] == "row" else _GROUP
        scales = [y[:, a:a + step].abs().max(1, keepdim=True).values.clamp(min=_LEAST_AMAX) / _E4M3_MOST for a in range(0, c, step)]
        got["y"].append(torch.cat([y[:, a * step:(a + 1) * step] / s for a, s in enumerate(scales)], 1))
        got["s"].append(torch.cat(scales, 1))
    got = {name: torch.cat(parts) for name, parts in got.items() if parts}
    if state["scales"] == "row":
        got["s"] = got["s"][:, 0]
    return got


def _exact_attend(state):
    q, k, v = state["q"], state["k"], state["v"]
    group = state["heads"] // state["kv_heads"]
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    starts_q, starts_k = state["starts_q"].tolist(), state["starts_k"].tolist()
    ends_k = starts_k[1:] if state["lengths_k"] is None else [a + n for a, n in zip(starts_k, state["lengths_k"].tolist())]
    for a, b, c, e in zip(starts_q, starts_q[1:], starts_k, ends_k):
        for g in range(state["kv_heads"]):
            keys, values = k[c:e, g].double(), v[c:e, g].double()
            for at in range(a, b, 4096):
                end = min(b, at + 4096)
                seen = torch.ones(end - at, e - c, dtype=torch.bool, device="cuda").tril_((at - a) + (e - c) - (b - a))
                for h in range(g * group, (g + 1) * group):
                    s = q[at:end, h].double() @ keys.T / math.sqrt(state["head_dim"])
                    s = s.where(seen, -math.inf)
                    norm = torch.logsumexp(s, 1)
                    lse[at:end, h] = norm
                    o[at:end, h] = torch.exp(s - norm[:, None].nan_to_num(neginf=0.0)) @ values
    return (o, lse) if state["lse"] else o
