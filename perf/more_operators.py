"""The operators that hold long contexts in less memory and read less of them, as cases to measure: their inputs, their plain forms and the calls a
program makes.

An 8-bit cache keeps a code for every value and a whole exponent E for every (token, kv head), keys and values apart; a value is code * 2^E.
With a the largest magnitude of the D values: e4m3 codes take the smallest E with a <= 448 * 2^E (at most 119), int8 codes the smallest with
a <= 127 * 2^E (at most 121), at least -100 both; codes are rounded to nearest, ties to even.  A row at position p sees keys j <= p; with a
window it sees the last `window` of them, its own among them, and the first `sinks` of the sequence.  Five operators:

  append   norms of the query and key heads, rotation, keys and values into the 8-bit cache; then those slots read back
  convert  bf16 keys and values into the 8-bit cache, then read back
  decode   attention of one new row per sequence
  prefill  attention of the rows of a prompt's chunk; these two over a bf16 cache with a window, and over an 8-bit cache with and without
"""
import math

import torch

own = False

HEADS = {"8b": (32, 8, 128), "small": (4, 2, 64), "one kv head": (8, 1, 128), "no sharing": (2, 2, 64)}
TOP = {"e4m3": (0.875, 9, 119), "int8": (127 / 128, 7, 121)}  # the largest code as f * 2^x, and the largest exponent


def listed():
    return [
        # a decode step's rows of 16 requests; a prompt chunk's rows at the prefill workload's size
        {"name": "append 16x1 e4m3", "op": "append", "heads": "8b", "cache": "e4m3", "B": 16, "n": 1, "lo": 1, "hi": 4000},
        {"name": "append 1x4096 int8", "op": "append", "heads": "8b", "cache": "int8", "B": 1, "n": 4096, "lo": 0, "hi": 0},
        # a short prompt prefix, and the long contexts of a batch, moved into the smaller cache
        {"name": "convert 1x500 int8", "op": "convert", "heads": "8b", "cache": "int8", "B": 1, "n": 500, "lo": 3, "hi": 3},
        {"name": "convert 8x32768 e4m3", "op": "convert", "heads": "8b", "cache": "e4m3", "B": 8, "n": 32768, "lo": 0, "hi": 0},
        # one request right after a short prompt: the call's latency; a serving batch at the decode workload's lengths; a window over them
        {"name": "decode 1 ctx500 e4m3", "op": "decode", "heads": "8b", "cache": "e4m3", "B": 1, "lo": 500, "hi": 500, "window": 0, "sinks": 0},
        {"name": "decode 32 ctx32768 e4m3", "op": "decode", "heads": "8b", "cache": "e4m3", "B": 32, "lo": 1, "hi": 32768, "window": 0, "sinks": 0},
        {"name": "decode 64 w4096 int8", "op": "decode", "heads": "8b", "cache": "int8", "B": 64, "lo": 1, "hi": 16384, "window": 4096, "sinks": 4},
        {"name": "decode 16 w4096 bf16", "op": "decode", "heads": "8b", "cache": "bf16", "B": 16, "lo": 1, "hi": 32768, "window": 4096, "sinks": 4},
        # a chunk behind a long prompt; a windowed prompt in one chunk; ragged chunks of the small layer, some sequences without a row
        {"name": "prefill 1x512 ctx8192 e4m3", "op": "prefill", "heads": "8b", "cache": "e4m3", "B": 1, "n_lo": 512, "n_hi": 512, "lo": 7680, "hi": 7680, "window": 0, "sinks": 0},
        {"name": "prefill 1x4096 w1024 bf16", "op": "prefill", "heads": "8b", "cache": "bf16", "B": 1, "n_lo": 4096, "n_hi": 4096, "lo": 0, "hi": 0, "window": 1024, "sinks": 4},
        {"name": "prefill small 7x0-100 int8", "op": "prefill", "heads": "small", "cache": "int8", "B": 7, "n_lo": 0, "n_hi": 100, "lo": 0, "hi": 900, "window": 300, "sinks": 1},
        {"name": "decode small 7 w64 bf16", "op": "decode", "heads": "small", "cache": "bf16", "B": 7, "lo": 0, "hi": 1021, "window": 64, "sinks": 3},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "convert", "decode", "decode", "prefill", "prefill"])
    c = {"op": op, "heads": rng.choice(["8b", "8b", "small", "one kv head", "no sharing"])}
    if op in ("append", "convert"):
        c["cache"] = rng.choice(["e4m3", "int8"])
        c["B"] = _log_uniform(rng, 1, 64)
        c["n"] = _log_uniform(rng, 1, (4096 if op == "append" else 200000) // c["B"])
        c["hi"] = rng.randint(0, 2000)
        c["lo"] = rng.randint(0, c["hi"])
        return c
    c["cache"] = rng.choice(["e4m3", "int8", "bf16"])
    c["window"] = 0 if c["cache"] != "bf16" and rng.random() < 0.5 else _log_uniform(rng, 1, 8192)
    c["sinks"] = rng.choice([0, 1, 4, rng.randint(5, 600)]) if c["window"] else 0
    if op == "decode":
        c["B"] = _log_uniform(rng, 1, 64)
        c["hi"] = _log_uniform(rng, 1, min(32768, 400000 // c["B"]))
        c["lo"] = rng.choice([0, c["hi"] // 2, c["hi"]])
        return c
    c["B"] = _log_uniform(rng, 1, 8)
    c["n_hi"] = _log_uniform(rng, 1, 4096 // c["B"])
    c["n_lo"] = rng.randint(0, c["n_hi"])
    c["hi"] = rng.randint(0, min(8000, 5000000 // (c["B"] * c["n_hi"])))
    c["lo"] = rng.randint(0, c["hi"])
    return c


# ------------------------------------------------------------------ the inputs
def _spread(lo, hi, n):
    """n whole numbers that cover lo .. hi evenly (their sum does not depend on a seed)."""
    return [lo + (hi - lo) * (2 * i + 1) // (2 * n) if n > 1 else hi for i in range(n)]


def _slots(n):
    return max(64, (n + 63) // 64 * 64)


def _normal(shape, seed, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    out = torch.empty(shape, dtype=dtype, device="cuda")
    return out.normal_(0.0, std, generator=g)


def _uneven(shape, seed):
    """Keys or values as a layer gives them: a few loud channels, and tokens of different loudness."""
    x = _normal(shape, seed)
    d = shape[-1]
    x *= torch.where(_normal((d,), seed + 50, 1.0, torch.float32) > 2.0, 6.0, 1.0).to(torch.bfloat16)
    x *= torch.exp(_normal((*shape[:-1], 1), seed + 60, 0.5, torch.float32)).to(torch.bfloat16)
    return x


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _codes(shape, cache):
    return torch.zeros(shape, dtype=torch.float8_e4m3fn if cache == "e4m3" else torch.int8, device="cuda")


def prepare(case, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    hq, hkv, d = HEADS[case["heads"]]
    B, op = case["B"], case["op"]

    def shuffled(lo, hi):
        v = _spread(lo, hi, B)
        return [v[i] for i in torch.randperm(B, generator=g).tolist()]

    s = {"op": op, "cache": case["cache"], "hq": hq, "hkv": hkv, "d": d, "B": B}
    at = shuffled(case["lo"], case["hi"])
    if op in ("append", "convert"):
        n = case["n"]
        cap = _slots(case["hi"] + n)
        s["start"], s["len"], s["n"] = _i32(at), _i32([n] * B), n
        s["k8"], s["v8"] = _codes((B, cap, hkv, d), case["cache"]), _codes((B, cap, hkv, d), case["cache"])
        s["ke"], s["ve"] = (torch.zeros(B, hkv, cap, dtype=torch.int8, device="cuda") for _ in range(2))
        if op == "append":
            s["seq"] = torch.arange(B, dtype=torch.int32, device="cuda").repeat_interleave(n)
            s["pos"] = (s["start"][:, None] + torch.arange(n, dtype=torch.int32, device="cuda")).reshape(-1).contiguous()
            s["qkv"] = _uneven((B * n, hq + 2 * hkv, d), seed + 1).view(B * n, -1)
            s["q_norm"] = (1 + 0.1 * _normal((d,), seed + 4, 1.0, torch.float32)).to(torch.bfloat16)
            s["k_norm"] = (1 + 0.1 * _normal((d,), seed + 5, 1.0, torch.float32)).to(torch.bfloat16)
            s["base"], s["eps"] = 1e6, 1e-6
        else:
            s["k"], s["v"] = _uneven((B, n, hkv, d), seed + 1), _uneven((B, n, hkv, d), seed + 2)
        return s
    s["window"], s["sinks"] = case["window"], case["sinks"]
    if op == "decode":
        cap = _slots(case["hi"])
        s["len"] = _i32(at)
        s["q"] = _normal((B, hq, d), seed + 1)
    else:
        n = shuffled(case["n_lo"], case["n_hi"])
        n[0] = max(1, n[0])
        cap = _slots(max(a + m for a, m in zip(at, n)))
        s["start"], s["len"], s["off"] = _i32(at), _i32(n), _i32([sum(n[:b]) for b in range(B)])
        s["rows"], s["n_max"], s["kv_max"] = sum(n), max(n), max(a + m for a, m in zip(at, n))
        s["q"] = _normal((s["rows"], hq, d), seed + 1)
    k, v = _uneven((B, cap, hkv, d), seed + 2), _uneven((B, cap, hkv, d), seed + 3)
    if case["cache"] == "bf16":
        s["k"], s["v"] = k, v
    else:
        for x, c, e in ((k, "k8", "ke"), (v, "v8", "ve")):
            s[c], s[e] = _codes((B, cap, hkv, d), case["cache"]), torch.zeros(B, hkv, cap, dtype=torch.int8, device="cuda")
            for b in range(B):  # a sequence at a time: a long batch's cache is large in 32 bits
                codes, exps = _quantised(x[b], case["cache"])
                s[c].view(torch.uint8)[b] = codes.view(torch.uint8)
                s[e][b] = exps.T
    return s


# ------------------------------------------------------------ the plain forms
def _two_to(e):
    """2^e of whole numbers -126 .. 127, exactly, in fp32."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantised(x, cache):
    """bf16 [..., d] -> codes of the same shape, whole exponents [...] (int8)."""
    most, width, top = TOP[cache]
    m, e = torch.frexp(x.float().abs().amax(-1))
    e = torch.where(m <= most, e - width, e - width + 1).clamp(-100, top)
    y = x.float() * _two_to(-e)[..., None]
    if cache == "e4m3":
        codes = y.clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        codes = torch.round(y).clamp(-127, 127).to(torch.int8)
    return codes, e.to(torch.int8)


def _values(codes, exps):
    """codes [B][slots][Hkv][D], exponents [B][Hkv][slots] -> fp32 values."""
    return codes.float() * _two_to(exps.transpose(1, 2))[..., None]


def _cache(s):
    if s["cache"] == "bf16":
        return s["k"].float(), s["v"].float()
    return _values(s["k8"], s["ke"]), _values(s["v8"], s["ve"])


def _attend(s, q, k, v, sees):
    """q [B][N][Hq][D], sees [B][N][slots] -> fp32 [B][N][Hq][D]; rows that see nothing give zeros."""
    B, N, hq, d = q.shape
    cap, hkv = k.shape[1], k.shape[2]
    G = hq // hkv
    x = q.float().view(B, N, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, N * G, d)
    x = torch.matmul(x, k.permute(0, 2, 3, 1)).view(B, hkv, N, G, cap)
    x *= 1.0 / math.sqrt(d)
    x.masked_fill_(~sees[:, None, :, None, :], -math.inf)
    x -= x.amax(-1, keepdim=True).clamp_min(-3e38)
    x.exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, hkv, N * G, cap), v.permute(0, 2, 1, 3)).view(B, hkv, N, G, d) / total.clamp_min(1e-30)
    return o.permute(0, 2, 1, 3, 4).reshape(B, N, hq, d)


def _sees(s, pos, cap):
    """Whether the row at position pos [...] sees slot j: [..., cap]."""
    j = torch.arange(cap, device="cuda")
    p = pos.long()[..., None]
    sees = j <= p
    if s["window"]:
        sees = sees & ((j > p - s["window"]) | (j < s["sinks"]))
    return sees


def _plain_decode(s):
    k, v = _cache(s)
    o = _attend(s, s["q"][:, None], k, v, _sees(s, s["len"][:, None] - 1, k.shape[1]))
    return {"out": o[:, 0].to(torch.bfloat16)}


def _plain_prefill(s):
    k, v = _cache(s)
    i = torch.arange(s["n_max"], device="cuda")
    at = (s["off"].long()[:, None] + i).clamp(max=s["rows"] - 1)
    o = _attend(s, s["q"][at], k, v, _sees(s, s["start"].long()[:, None] + i, k.shape[1]))
    r = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted((s["off"] + s["len"]).long(), r, right=True)
    return {"out": o[b, r - s["off"].long()[b]].to(torch.bfloat16)}


def _store(s, x, c, e):
    """bf16 x [B][n][Hkv][D] into slots start .. start + n - 1 of codes s[c] and exponents s[e], and what they then hold."""
    b = torch.arange(s["B"], device="cuda")[:, None]
    slot = s["start"].long()[:, None] + torch.arange(s["n"], device="cuda")
    codes, exps = _quantised(x, s["cache"])
    s[c].view(torch.uint8)[b, slot] = codes.view(torch.uint8)
    s[e].transpose(1, 2)[b, slot] = exps
    held = s[c].view(torch.uint8)[b, slot].view(s[c].dtype).float()
    return (held * _two_to(s[e].transpose(1, 2)[b, slot])[..., None]).to(torch.bfloat16)


def _plain_append(s):
    hq, hkv, d, B, n = s["hq"], s["hkv"], s["d"], s["B"], s["n"]
    x = s["qkv"].float().view(B * n, hq + 2 * hkv, d)
    inv = torch.pow(torch.tensor(s["base"], dtype=torch.float64, device="cuda"), -2.0 * torch.arange(d // 2, dtype=torch.float64, device="cuda") / d)
    th = s["pos"].double()[:, None] * inv
    c, sn = torch.cos(th).float()[:, None], torch.sin(th).float()[:, None]

    def turn(h, gain):
        h = h / torch.sqrt((h * h).mean(-1, keepdim=True) + s["eps"]) * gain.float()
        lo, hi = h[..., : d // 2], h[..., d // 2:]
        return torch.cat([lo * c - hi * sn, hi * c + lo * sn], -1).to(torch.bfloat16)

    k = turn(x[:, hq: hq + hkv], s["k_norm"]).view(B, n, hkv, d)
    v = s["qkv"].view(B, n, hq + 2 * hkv, d)[:, :, hq + hkv:]
    return {"q": turn(x[:, :hq], s["q_norm"]), "k": _store(s, k, "k8", "ke"), "v": _store(s, v, "v8", "ve")}


def _plain_convert(s):
    return {"k": _store(s, s["k"], "k8", "ke"), "v": _store(s, s["v"], "v8", "ve")}


# ----------------------------------------------------------------- one pass
def run(state):
    s = state
    if not own:
        return {"append": _plain_append, "convert": _plain_convert, "decode": _plain_decode, "prefill": _plain_prefill}[s["op"]](s)
    from invariant_deterministic_gb300 import kinv

    if s["cache"] != "bf16" and "handle" not in s:  # a serving loop keeps its cache's handle, its outputs' memory and its workspace
        s["handle"] = kinv.Cache8(s["k8"], s["v8"], s["ke"], s["ve"])
    if s["op"] in ("append", "convert"):
        c = s["handle"]
        if s["op"] == "append":
            q = torch.empty(s["B"] * s["n"], s["hq"], s["d"], dtype=torch.bfloat16, device="cuda")
            kinv.rope_append8(s["qkv"], q, c, s["seq"], s["pos"], s["hq"], s["hkv"], s["d"], s["base"], s["q_norm"], s["k_norm"], s["eps"])
            k, v = kinv.cache8_read(c, s["start"], s["len"], s["n"])
            return {"q": q, "k": k, "v": v}
        kinv.cache8_write(c, s["k"], s["v"], s["start"], s["len"])
        k, v = kinv.cache8_read(c, s["start"], s["len"], s["n"])
        return {"k": k, "v": v}
    if s["op"] == "decode":
        if s["cache"] == "bf16":
            if "ws" not in s:
                s["ws"] = torch.empty(max(16, kinv.attn_decode_workspace(s["B"], s["hq"], s["d"], s["k"].shape[1], window=s["window"], sinks=s["sinks"])), dtype=torch.uint8, device="cuda")
            return {"out": kinv.attn_decode(s["q"], s["k"], s["v"], s["len"], workspace=s["ws"], window=s["window"], sinks=s["sinks"])}
        if "ws" not in s:
            s["ws"] = torch.empty(max(16, kinv.attn_decode8_workspace(s["B"], s["hq"], s["d"], s["handle"].slots, s["window"], s["sinks"])), dtype=torch.uint8, device="cuda")
        return {"out": kinv.attn_decode8(s["q"], s["handle"], s["len"], workspace=s["ws"], window=s["window"], sinks=s["sinks"])}
    if s["cache"] == "bf16":
        return {"out": kinv.attn_prefill(s["q"], s["k"], s["v"], s["start"], s["len"], s["off"], s["n_max"], s["kv_max"], window=s["window"], sinks=s["sinks"])}
    if "ws" not in s:
        s["ws"] = torch.empty(max(16, kinv.attn_prefill8_workspace(s["B"], s["rows"], s["hq"], s["hkv"], s["d"], s["kv_max"])), dtype=torch.uint8, device="cuda")
    return {"out": kinv.attn_prefill8(s["q"], s["handle"], s["start"], s["len"], s["off"], s["n_max"], s["kv_max"], workspace=s["ws"], window=s["window"], sinks=s["sinks"])}


# ------------------------------------------------------------- what it costs
def _visible(length, window, sinks):
    """Keys that the last of `length` positions sees."""
    return length if not window else min(length, window) + min(sinks, max(0, length - window))


def work(case):
    hq, hkv, d = HEADS[case["heads"]]
    B = case["B"]
    if case["op"] in ("append", "convert"):
        n = B * case["n"]
        rows = hq + 2 * hkv if case["op"] == "append" else 2 * hkv
        return {"bytes": n * (rows * d * 2 + (hq * d * 2 if case["op"] == "append" else 0) + 2 * hkv * (2 * (d + 1) + 2 * d)), "flops": n * rows * d * 10}
    key = 2 * hkv * (2 * d if case["cache"] == "bf16" else d + 1)
    at = _spread(case["lo"], case["hi"], B)
    if case["op"] == "decode":
        seen = sum(_visible(m, case["window"], case["sinks"]) for m in at)
        return {"bytes": seen * key + B * hq * d * 4, "flops": 4 * d * hq * seen}
    n = _spread(case["n_lo"], case["n_hi"], B)
    n[0] = max(1, n[0])
    pairs = sum(_visible(a + i + 1, case["window"], case["sinks"]) for a, m in zip(at, n) for i in range(m))
    keys = sum(_visible(a + m, case["window"] and case["window"] + m - 1, case["sinks"]) for a, m in zip(at, n) if m)
    return {"bytes": keys * key + sum(n) * hq * d * 4, "flops": 4 * d * hq * pairs}


# ---------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "convert": _exact_convert, "decode": _exact_decode, "prefill": _exact_prefill}[case["op"]](s)


def _exact_held(x, cache):
    """The values that the 8-bit cache holds for bf16 x [..., d], in 64 bits: x rounded to the codes' grid."""
    two_to = lambda e: ((e.long() + 1023) << 52).view(torch.float64)  # noqa: E731
    x = x.double()
    limit, most = (448.0, 119) if cache == "e4m3" else (127.0, 121)
    loud = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(loud.clamp_min(1e-300) / limit))
    e = torch.where(loud > limit * two_to(e), e + 1, e)
    e = torch.where(loud <= limit * two_to(e - 1), e - 1, e).clamp(-100, most)
    y = x * two_to(-e)
    step = torch.ones_like(y) if cache == "int8" else two_to(torch.frexp(y.abs().clamp_min(2.0 ** -6)).exponent - 4)
    return (torch.round(y / step) * step).clamp(-limit, limit) * two_to(e)


def _exact_convert(s):
    return {name: torch.cat([_exact_held(x[b: b + 1], s["cache"]) for b in range(s["B"])]) for name, x in (("k", s["k"]), ("v", s["v"]))}


def _exact_append(s):
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    heads = s["qkv"].double().reshape(s["B"] * s["n"], -1, d)
    i = torch.arange(d // 2, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["pos"].double()[:, None] * torch.exp(-2.0 * i / d * math.log(s["base"])))[:, None]

    def rotated(x, gain):
        x = x * torch.rsqrt(x.square().sum(-1, keepdim=True) / d + s["eps"]) * gain.double()
        z = torch.complex(x[..., : d // 2], x[..., d // 2:]) * turn
        return torch.cat([z.real, z.imag], -1)

    k = rotated(heads[:, hq: hq + hkv], s["k_norm"]).to(torch.bfloat16)  # the cache takes the bf16 keys
    shape = (s["B"], s["n"], hkv, d)
    return {"q": rotated(heads[:, :hq], s["q_norm"]), "k": _exact_held(k, s["cache"]).view(shape),
            "v": _exact_held(heads[:, hq + hkv:], s["cache"]).view(shape)}


def _exact_keys(s, b, g, used):
    if s["cache"] == "bf16":
        return s["k"][b, :used, g].double(), s["v"][b, :used, g].double()
    return tuple(s[c][b, :used, g].to(torch.float32).double() * torch.exp2(s[e][b, g, :used].double())[:, None] for c, e in (("k8", "ke"), ("v8", "ve")))


def _exact_rows(s, q, b, first):
    """Rows q [n][Hq][D] of sequence b at positions first .. first + n - 1."""
    n, hq, d = q.shape
    out = torch.zeros(n, hq, d, dtype=torch.float64, device="cuda")
    used = first + n
    if used <= 0 or n == 0:
        return out
    p = torch.arange(first, used, device="cuda")[:, None]
    j = torch.arange(used, device="cuda")[None]
    hidden = j > p
    if s["window"]:
        hidden = hidden | ((p - j >= s["window"]) & (j >= s["sinks"]))
    G = hq // s["hkv"]
    for g in range(s["hkv"]):
        k, v = _exact_keys(s, b, g, used)
        for h in range(g * G, g * G + G):
            w = (q[:, h].double() @ k.T) / math.sqrt(d)
            out[:, h] = torch.softmax(w.masked_fill(hidden, -math.inf), 1) @ v
    return out


def _exact_decode(s):
    n = s["len"].tolist()
    return {"out": torch.stack([_exact_rows(s, s["q"][b: b + 1], b, n[b] - 1)[0] for b in range(s["B"])])}


def _exact_prefill(s):
    start, n, off = (s[k].tolist() for k in ("start", "len", "off"))
    return {"out": torch.cat([_exact_rows(s, s["q"][off[b]: off[b] + n[b]], b, start[b]) for b in range(s["B"])])}
