"""The operators that verify and score drafted tokens, as cases to measure: their inputs, their plain forms and the calls a program makes.

A drafted tree: sequence b has ctx_len[b] keys in its cache and n_nodes[b] drafted nodes after them, rows row_offset[b] + i of the row tensors.
parent[row] is the node's parent (an index below its own within the sequence, or -1: the node follows the context itself).  A node of depth t (its
number of ancestors) is the token at position ctx_len + t; its keys and values sit in cache slot ctx_len + i, and it sees the context, its
ancestors and itself.  Four operators:

  rope   norms of the query and key heads, rotation to the node's position, keys and values into the node's slot
  attn   attention of the nodes over the context and their own ancestors
  accept the path of nodes that the model's own tokens agree with, and the move of that path's keys and values to their positions
  score  log probabilities of given tokens, entropy and the most likely alternatives of rows of logits
"""
import math

import torch

own = False

HEADS = {"8b": (32, 8, 128), "small": (4, 2, 64), "one kv head": (8, 1, 128), "no sharing": (2, 2, 64)}
VOCAB = 151936


def listed():
    return [
        # one request, a small tree right after a short prompt: the call's latency
        {"name": "attn 1x8 ctx500", "op": "attn", "heads": "8b", "B": 1, "n_lo": 8, "n_hi": 8, "ctx_lo": 500, "ctx_hi": 500, "shape": "tree"},
        # one request deep into a long document with a full tree: the keys split over the whole GPU
        {"name": "attn 1x64 ctx32000", "op": "attn", "heads": "8b", "B": 1, "n_lo": 64, "n_hi": 64, "ctx_lo": 32000, "ctx_hi": 32000, "shape": "tree"},
        # a serving batch at the decode workload's lengths
        {"name": "attn 16x32 ctx32736", "op": "attn", "heads": "8b", "B": 16, "n_lo": 32, "n_hi": 32, "ctx_lo": 1, "ctx_hi": 32736, "shape": "tree"},
        # a larger batch at the full model's prompt lengths, ragged trees
        {"name": "attn 64x1-16 ctx4096", "op": "attn", "heads": "8b", "B": 64, "n_lo": 1, "n_hi": 16, "ctx_lo": 16, "ctx_hi": 4096, "shape": "tree"},
        # the small layer, a draft without branches (odd lengths, some contexts empty)
        {"name": "attn small 7x5-13", "op": "attn", "heads": "small", "B": 7, "n_lo": 5, "n_hi": 13, "ctx_lo": 0, "ctx_hi": 1021, "shape": "chain"},
        # the same trees' rows before attention: one request, and a large ragged batch
        {"name": "rope 1x8", "op": "rope", "heads": "8b", "B": 1, "n_lo": 8, "n_hi": 8, "ctx_lo": 500, "ctx_hi": 500, "shape": "tree"},
        {"name": "rope 64x1-64", "op": "rope", "heads": "8b", "B": 64, "n_lo": 1, "n_hi": 64, "ctx_lo": 1, "ctx_hi": 200, "shape": "tree"},
        # after the model's own tokens are known, all 36 layers' cache
        {"name": "accept 1x8", "op": "accept", "heads": "8b", "layers": 36, "B": 1, "n_lo": 8, "n_hi": 8, "ctx_lo": 60, "ctx_hi": 60, "shape": "tree"},
        {"name": "accept 32x64", "op": "accept", "heads": "8b", "layers": 36, "B": 32, "n_lo": 64, "n_hi": 64, "ctx_lo": 1, "ctx_hi": 190, "shape": "tree"},
        # a served token's alternatives; the rows of a decode batch; the scored rows of a prompt, bf16 logits
        {"name": "score 1 f32 top5", "op": "score", "rows": 1, "V": VOCAB, "dtype": "f32", "ids": 1, "top": 5},
        {"name": "score 256 f32 top20", "op": "score", "rows": 256, "V": VOCAB, "dtype": "f32", "ids": 2, "top": 20},
        {"name": "score 4096 bf16 top1", "op": "score", "rows": 4096, "V": VOCAB, "dtype": "bf16", "ids": 1, "top": 1},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "rope", "accept", "score"])
    if op == "score":
        dtype = rng.choice(["f32", "bf16"])
        V = _log_uniform(rng, 500, VOCAB)
        rows = _log_uniform(rng, 1, min(8192, 4096 * VOCAB * 2 // (V * (4 if dtype == "f32" else 2))))
        return {"op": op, "rows": rows, "V": V, "dtype": dtype, "ids": rng.randint(0, 4), "top": rng.choice([0, 1, 3, 8, 20, 32])}
    c = {"op": op, "heads": rng.choice(["8b", "8b", "small", "one kv head", "no sharing"]), "shape": rng.choice(["tree", "tree", "chain"])}
    n = _log_uniform(rng, 1, 64)
    c["n_hi"], c["n_lo"] = n, rng.randint(1, n)
    if op == "attn":
        c["B"] = _log_uniform(rng, 1, 64)
        c["ctx_hi"] = _log_uniform(rng, 1, min(32704, 16 * 32736 * 32 // (c["B"] * max(32, n))))  # at most the largest listed case's keys and work
        c["ctx_lo"] = rng.choice([0, c["ctx_hi"] // 2, c["ctx_hi"]])
    else:
        c["B"] = _log_uniform(rng, 1, 64 if op == "rope" else 32)
        c["ctx_hi"] = rng.randint(0, 190)
        c["ctx_lo"] = rng.randint(0, c["ctx_hi"])
        if op == "accept":
            c["layers"] = _log_uniform(rng, 1, 36)
    return c


# ------------------------------------------------------------------ the inputs
def _spread(lo, hi, n):
    """n whole numbers that cover lo .. hi evenly (their sum does not depend on a seed)."""
    return [lo + (hi - lo) * (2 * i + 1) // (2 * n) if n > 1 else hi for i in range(n)]


def _capacity(case):
    return (case["ctx_hi"] + case["n_hi"] + 63) // 64 * 64


def _mean_depth(shape, n):
    """Nodes on the longest path of the trees below, for a tree of n nodes."""
    if shape == "chain":
        return n
    d, i = 1, n - 1
    while i > 0:
        i, d = max(0, i // 3), d + 1
    return d


def _normal(shape, seed, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    out = torch.empty(shape, dtype=dtype, device="cuda")
    return out.normal_(0.0, std, generator=g)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator()
    g.manual_seed(seed)

    def below(n):
        return int(torch.randint(0, max(1, n), (1,), generator=g))

    if case["op"] == "score":
        rows, V = case["rows"], case["V"]
        x = _normal((rows, V), seed + 1, 2.0, torch.float32)
        likely = torch.randint(0, V, (rows, 8), generator=g).cuda()  # each row has a few tokens that the model prefers
        x.scatter_add_(1, likely, torch.rand(rows, 8, generator=g).cuda() * 12)
        if case["dtype"] == "bf16":
            x = x.to(torch.bfloat16)
        ids = torch.randint(0, V, (rows, case["ids"]), generator=g).cuda()
        ids = torch.where(torch.rand(rows, case["ids"], generator=g).cuda() < 0.7, likely[:, :1].expand_as(ids), ids).to(torch.int32)
        return {"op": "score", "logits": x, "ids": ids.contiguous() if case["ids"] else None, "top": case["top"]}

    hq, hkv, d = HEADS[case["heads"]]
    B = case["B"]
    order = torch.randperm(B, generator=g).tolist()
    ctx = [_spread(case["ctx_lo"], case["ctx_hi"], B)[i] for i in order]
    order = torch.randperm(B, generator=g).tolist()
    n = [_spread(case["n_lo"], case["n_hi"], B)[i] for i in order]
    off, parent = [], []
    for b in range(B):
        off.append(len(parent))
        for i in range(n[b]):
            if case["shape"] == "chain" or i < 2:
                parent.append(i - 1)
            else:
                parent.append(i // 4 + below(i // 2 - i // 4 + 1))
    rows, cap = len(parent), _capacity(case)
    s = {"op": case["op"], "rows": rows, "max_nodes": case["n_hi"], "cap": cap, "hq": hq, "hkv": hkv, "d": d,
         "ctx": _i32(ctx), "n": _i32(n), "off": _i32(off), "parent": _i32(parent)}
    if case["op"] == "attn":
        s["q"] = _normal((rows, hq, d), seed + 1)
        s["k"] = _normal((B, cap, hkv, d), seed + 2)
        s["v"] = _normal((B, cap, hkv, d), seed + 3)
    elif case["op"] == "rope":
        s["qkv"] = _normal((rows, (hq + 2 * hkv) * d), seed + 1)
        s["k"] = _normal((B, cap, hkv, d), seed + 2)
        s["v"] = _normal((B, cap, hkv, d), seed + 3)
        s["q_norm"] = (1 + 0.1 * _normal((d,), seed + 4, 1.0, torch.float32)).to(torch.bfloat16)
        s["k_norm"] = (1 + 0.1 * _normal((d,), seed + 5, 1.0, torch.float32)).to(torch.bfloat16)
        s["base"], s["eps"] = 1e6, 1e-6
    else:
        tokens = torch.randint(0, VOCAB, (rows,), generator=g)
        nxt = torch.randint(0, VOCAB, (rows,), generator=g)
        agree = (torch.rand(rows, generator=g) < 0.8).tolist()
        for b in range(B):
            for i in range(1, n[b]):  # the model's token after a node is one of its children's for most nodes
                p = off[b] + parent[off[b] + i]
                if agree[p] and below(2) or i == n[b] - 1:
                    nxt[p] = tokens[off[b] + i]
        s["tokens"], s["next"] = tokens.to(torch.int32).cuda(), nxt.to(torch.int32).cuda()
        s["kv"] = _normal((case["layers"], 2, B, cap, hkv, d), seed + 1)
    return s


# ------------------------------------------------------------ the plain forms
def _rows_of(s):
    """(sequence, node) of every row."""
    r = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(s["off"].long(), r, right=True) - 1
    return b, r - s["off"].long()[b]


def _padded(s, x, fill=0):
    """Row tensor [rows, ...] -> [B, max_nodes, ...]."""
    i = torch.arange(s["max_nodes"], device="cuda")
    at = (s["off"].long()[:, None] + i).clamp(max=s["rows"] - 1)
    live = i < s["n"].long()[:, None]
    return torch.where(live.view(*live.shape, *([1] * (x.dim() - 1))), x[at], torch.full((), fill, dtype=x.dtype, device="cuda"))


def _ancestors(s):
    """[B, N, N]: whether node j is node i itself or one of its ancestors."""
    par = _padded(s, s["parent"], -1).long()
    N = s["max_nodes"]
    j = torch.arange(N, device="cuda")
    up = (par[:, :, None] == j).float() + torch.eye(N, device="cuda")
    for _ in range(6):  # 2^6 = 64 generations
        up = (torch.matmul(up, up) > 0).float()
    return up > 0


def _plain_attn(s):
    B, cap, hkv, d = s["k"].shape
    N, G = s["max_nodes"], s["hq"] // hkv
    anc = _ancestors(s)
    q = _padded(s, s["q"]).float().view(B, N, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, N * G, d)
    k = s["k"].permute(0, 2, 1, 3).float()
    v = s["v"].permute(0, 2, 1, 3).float()
    rel = torch.arange(cap, device="cuda")[None, :] - s["ctx"].long()[:, None]  # slot - ctx_len
    in_tree = torch.gather(anc, 2, rel.clamp(0, N - 1)[:, None, :].expand(B, N, cap)) & (rel >= 0)[:, None] & (rel < N)[:, None]
    sees = (rel < 0)[:, None] | in_tree
    x = torch.matmul(q, k.transpose(2, 3)).view(B, hkv, N, G, cap) / math.sqrt(d)
    x = x.masked_fill(~sees[:, None, :, None, :], -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(e.view(B, hkv, N * G, cap), v).view(B, hkv, N, G, d) / e.sum(-1, keepdim=True)
    b, i = _rows_of(s)
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(B, N, s["hq"], d)[b, i].to(torch.bfloat16)}


def _plain_rope(s):
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    b, i = _rows_of(s)
    depth = _ancestors(s).sum(-1)[b, i] - 1
    ctx = s["ctx"].long()[b]
    x = s["qkv"].float().view(s["rows"], hq + 2 * hkv, d)
    inv = torch.pow(torch.tensor(s["base"], dtype=torch.float64, device="cuda"), -2.0 * torch.arange(d // 2, dtype=torch.float64, device="cuda") / d)
    th = (ctx + depth).double()[:, None] * inv
    c, sn = torch.cos(th).float()[:, None], torch.sin(th).float()[:, None]

    def turn(h, gain):
        h = h / torch.sqrt((h * h).mean(-1, keepdim=True) + s["eps"]) * gain.float()
        lo, hi = h[..., : d // 2], h[..., d // 2:]
        return torch.cat([lo * c - hi * sn, hi * c + lo * sn], -1).to(torch.bfloat16)

    s["k"][b, ctx + i] = turn(x[:, hq: hq + hkv], s["k_norm"])
    s["v"][b, ctx + i] = x[:, hq + hkv:].to(torch.bfloat16)
    return {"q": turn(x[:, :hq], s["q_norm"]), "k": s["k"], "v": s["v"]}


def _plain_accept(s):
    B, N = s["n"].shape[0], s["max_nodes"]
    j = torch.arange(N, device="cuda")
    par, tok, nxt = (_padded(s, s[k], -1).long() for k in ("parent", "tokens", "next"))
    live = j < s["n"].long()[:, None]
    wanted = torch.gather(nxt, 1, par.clamp(min=0)) == tok
    twin = (par[:, :, None] == par[:, None, :]) & (tok[:, :, None] == tok[:, None, :]) & (j[None, :] < j[:, None])  # an elder with the same token
    good = live & ((j == 0) | ((par >= 0) & wanted & ~twin.any(-1)))
    anc = _ancestors(s)
    taken = good & ~(anc & ~good[:, None, :]).any(-1) & anc[:, :, 0]
    count = taken.sum(-1)
    depth = anc.sum(-1) - 1
    path = torch.full((B, N + 1), -1, dtype=torch.int64, device="cuda")
    path.scatter_(1, torch.where(taken, depth, N), j.expand(B, N))
    path = path[:, :N]
    on = j < count[:, None]
    path = torch.where(on, path, -1)
    out = torch.where(on, torch.gather(nxt, 1, path.clamp(min=0)), -1)
    b = torch.arange(B, device="cuda")[:, None].expand(B, N)
    dst = s["ctx"].long()[:, None] + j
    src = s["ctx"].long()[:, None] + torch.where(on, path, j)
    s["kv"][:, :, b, dst] = s["kv"][:, :, b, src]
    return {"count": count.to(torch.int32), "path": path.to(torch.int32), "tokens": out.to(torch.int32), "kv": s["kv"]}


def _plain_score(s):
    x = s["logits"].float()
    V = x.shape[1]
    a = x - x.amax(1, keepdim=True)
    e = torch.exp(a)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    got = {"entropy": (log_total - (e * a).sum(1, keepdim=True) / total)[:, 0]}
    if s["ids"] is not None:
        got["logprobs"] = torch.gather(a, 1, s["ids"].long()) - log_total
    if s["top"]:
        bits = (x + 0.0).view(torch.int32)
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 32) + (V - 1 - torch.arange(V, device="cuda"))  # larger logits first, then lower ids
        ids = V - 1 - (torch.topk(key, s["top"], dim=1).values & 0xFFFFFFFF)
        got["top_ids"] = ids.to(torch.int32)
        got["top_logprobs"] = torch.gather(a, 1, ids) - log_total
    return got


# ----------------------------------------------------------------- one pass
def run(state):
    s = state
    if not own:
        return {"attn": _plain_attn, "rope": _plain_rope, "accept": _plain_accept, "score": _plain_score}[s["op"]](s)
    from invariant_deterministic_gb300 import kinv

    if s["op"] == "score":
        lp, entropy, top_ids, top_lp = kinv.logprobs(s["logits"], s["ids"], top_k=s["top"])
        got = {"entropy": entropy}
        if s["ids"] is not None:
            got["logprobs"] = lp
        if s["top"]:
            got["top_ids"], got["top_logprobs"] = top_ids, top_lp
        return got
    if "tree" not in s:  # a serving loop keeps its tree's buffers and its workspace
        s["tree"] = kinv.Tree(s["ctx"], s["n"], s["off"], s["parent"], s["max_nodes"], s["cap"])
        if s["op"] == "attn":
            s["ws"] = torch.empty(max(16, kinv.attn_tree_workspace(s["tree"], s["hq"], s["hkv"], s["d"])), dtype=torch.uint8, device="cuda")
    if s["op"] == "attn":
        return {"out": kinv.attn_tree(s["q"], s["k"], s["v"], s["tree"], workspace=s["ws"])}
    if s["op"] == "rope":
        q = torch.empty(s["rows"], s["hq"], s["d"], dtype=torch.bfloat16, device="cuda")
        kinv.rope_append_tree(s["qkv"], q, s["k"], s["v"], s["tree"], s["hq"], s["hkv"], s["d"], s["base"], s["q_norm"], s["k_norm"], s["eps"])
        return {"q": q, "k": s["k"], "v": s["v"]}
    count, path, tokens = kinv.tree_accept(s["tree"], s["tokens"], s["next"], s["kv"])
    return {"count": count, "path": path, "tokens": tokens, "kv": s["kv"]}


# ------------------------------------------------------------- what it costs
def work(case):
    if case["op"] == "score":
        e = case["rows"] * case["V"]
        return {"bytes": e * (4 if case["dtype"] == "f32" else 2) + case["rows"] * 4 * (1 + 2 * case["ids"] + 2 * case["top"]), "flops": 6 * e}
    hq, hkv, d = HEADS[case["heads"]]
    ctx, n = _spread(case["ctx_lo"], case["ctx_hi"], case["B"]), _spread(case["n_lo"], case["n_hi"], case["B"])
    nodes = sum(n)
    if case["op"] == "attn":
        # a mean over the pairing of lengths and trees, which the seed shuffles
        pairs = sum(ctx) * nodes / case["B"] + nodes * (1 + _mean_depth(case["shape"], case["n_hi"])) / 2
        return {"bytes": (sum(ctx) + nodes) * hkv * d * 4 + nodes * hq * d * 4, "flops": 4 * d * hq * pairs}
    if case["op"] == "rope":
        return {"bytes": nodes * (hq + 2 * hkv) * d * 4, "flops": nodes * (hq + hkv) * d * 8}
    moved = sum(max(0, _mean_depth(case["shape"], v) // 2) for v in n) if case["shape"] == "tree" else 0
    return {"bytes": moved * case["layers"] * hkv * d * 8 + nodes * 12 + case["B"] * case["n_hi"] * 8, "flops": 0}


# ---------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "score":
        return _exact_score(s)
    n, off, ctx, parent = (s[k].tolist() for k in ("n", "off", "ctx", "parent"))
    paths = []
    for b in range(len(n)):
        mine = []
        for i in range(n[b]):
            p = parent[off[b] + i]
            mine.append((mine[p] if p >= 0 else []) + [i])
        paths.append(mine)
    return {"attn": _exact_attn, "rope": _exact_rope, "accept": _exact_accept}[case["op"]](s, n, off, ctx, paths)


def _exact_attn(s, n, off, ctx, paths):
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    out = torch.zeros(s["rows"], hq, d, dtype=torch.float64, device="cuda")
    for b in range(len(n)):
        used = ctx[b] + n[b]
        k, v = s["k"][b, :used].double(), s["v"][b, :used].double()
        hidden = torch.ones(n[b], used, dtype=torch.bool)
        hidden[:, : ctx[b]] = False
        for i, path in enumerate(paths[b]):
            hidden[i, torch.tensor([ctx[b] + j for j in path])] = False
        hidden = hidden.cuda()
        for h in range(hq):
            g = h // (hq // hkv)
            w = s["q"][off[b]: off[b] + n[b], h].double() @ k[:, g].T * (1.0 / math.sqrt(d))
            w = torch.softmax(w.masked_fill(hidden, -math.inf), 1)
            out[off[b]: off[b] + n[b], h] = w @ v[:, g]
    return {"out": out}


def _exact_rope(s, n, off, ctx, paths):
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    seqs = [b for b in range(len(n)) for _ in range(n[b])]
    slots = torch.tensor([ctx[b] + i for b in range(len(n)) for i in range(n[b])], device="cuda")
    place = torch.tensor([ctx[b] + len(path) - 1 for b in range(len(n)) for path in paths[b]], dtype=torch.float64, device="cuda")
    heads = s["qkv"].double().reshape(s["rows"], -1, d)
    i = torch.arange(d // 2, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), place[:, None] * torch.exp(-2.0 * i / d * math.log(s["base"])))[:, None]

    def rotated(x, gain):
        x = x * torch.rsqrt(x.square().sum(-1, keepdim=True) / d + s["eps"]) * gain.double()
        z = torch.complex(x[..., : d // 2], x[..., d // 2:]) * turn
        return torch.cat([z.real, z.imag], -1)

    k, v = s["k"].double(), s["v"].double()
    k[seqs, slots] = rotated(heads[:, hq: hq + hkv], s["k_norm"])
    v[seqs, slots] = heads[:, hq + hkv:]
    return {"q": rotated(heads[:, :hq], s["q_norm"]), "k": k, "v": v}


def _exact_accept(s, n, off, ctx, paths):
    tokens, nxt, parent = (s[k].tolist() for k in ("tokens", "next", "parent"))
    kv = s["kv"]
    for b in range(len(n)):
        at, path = 0, [0]
        while True:
            step = [j for j in range(n[b]) if parent[off[b] + j] == at and tokens[off[b] + j] == nxt[off[b] + at]]
            if not step:
                break
            at = step[0]
            path.append(at)
        for t, j in enumerate(path):
            kv[:, :, b, ctx[b] + t] = kv[:, :, b, ctx[b] + j].clone()
    return {"count": None, "path": None, "tokens": None, "kv": kv}


def _exact_score(s):
    rows, V = s["logits"].shape
    entropy = torch.empty(rows, dtype=torch.float64, device="cuda")
    given = torch.empty(rows, 0 if s["ids"] is None else s["ids"].shape[1], dtype=torch.float64, device="cuda")
    best = torch.empty(rows, s["top"], dtype=torch.float64, device="cuda")
    for r in range(0, rows, 256):
        x = torch.log_softmax(s["logits"][r: r + 256].double(), 1)
        entropy[r: r + 256] = -(torch.exp(x) * x).sum(1)
        if s["ids"] is not None:
            given[r: r + 256] = x.gather(1, s["ids"][r: r + 256].long())
        if s["top"]:
            best[r: r + 256] = torch.topk(x, s["top"], dim=1).values
    got = {"entropy": entropy}
    if s["ids"] is not None:
        got["logprobs"] = given
    if s["top"]:
        got["top_ids"], got["top_logprobs"] = None, best
    return got
