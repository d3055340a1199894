"""What the speculative-decoding operators compute, and what they cost.

Four operators that belong together: a key/value cache that is quantised as it
is written and can be read back, the attention of a tree of drafted tokens
over such a cache, the verification of the drafted tokens against the target
model's logits from given random numbers, and the cache's commit of the
accepted path.  For each there are cases (listed() and draw()), their inputs
(prepare()), one pass (run(): the plain form in torch, or, with `own`, the
calls into transformer_decode_token_gb300.binding), the bytes and operations a
pass cannot do without (work()), and the result in 64 bits (exact()).

Layouts.  Caches are [slots][heads][positions][dim]; an int8 or e4m3 cache has
one fp32 scale per (slot, head, position) for the keys and one for the values.
The drafted nodes of all sequences are packed: rows first[b] .. first[b+1]-1
are sequence b's nodes in topological order, node 0 the last chosen token.
Node j's key and value are at cache row cached[b] + j.  A node sees the cached
prefix and the nodes named by the bits of its mask.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "int8": torch.int8,
         "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "int8": 1, "e4m3": 1}
SCALED = ("int8", "e4m3")
TINY = 2.0 ** -126
VOCAB = 50257


# ---- the cases ---------------------------------------------------------------------

def listed():
    return [
        # the k, v of one batched decode step, read out of the fused QKV rows
        # (64 sequences, 12 heads of 64)
        _kv("kv decode step int8", 64, 12, 64, 1024, 64, "f32", "int8", "f32", True),
        # the k, v of 64 packed prompts of 32 to 512 tokens, one layer
        _kv("kv prompts int8", 17408, 12, 64, 1024, 64, "f32", "int8", "f32", True),
        # bf16 rows of 128 into an e4m3 cache, an odd number of rows
        _kv("kv prompts e4m3", 8191, 8, 128, 2048, 8, "bf16", "e4m3", "bf16", False),
        # one sequence, a tree of 8 drafted tokens: latency of one layer
        _attn("tree one sequence", 1, 8, 12, 12, 64, 1024, 1000, 1000, "f32", "f32"),
        # the batched decode step's attention (single tokens) over ragged bf16 caches
        _attn("single tokens bf16", 64, 1, 12, 12, 64, 1024, 32, 575, "f32", "bf16"),
        # 16 sequences with trees of up to 16 drafted tokens over an int8 cache
        _attn("trees int8", 16, 16, 12, 12, 64, 1024, 100, 1000, "bf16", "int8"),
        # grouped heads, long contexts
        _attn("grouped heads long", 8, 8, 32, 8, 128, 16384, 4000, 16000, "bf16", "bf16"),
        # the largest trees over full caches
        _attn("large trees f16", 32, 64, 12, 12, 64, 4096, 2000, 4000, "f16", "f16"),
        # one sequence, a chain of 5 drafted tokens with the draft's distributions
        _verify("verify one chain", 1, 6, 1, VOCAB, 1.0, True),
        # 8 sequences, trees of 8 given tokens (no draft distribution)
        _verify("verify given trees", 8, 8, 3, VOCAB, 0.8, False),
        # 64 sequences, chains of 7 drafted tokens
        _verify("verify 64 chains", 64, 8, 1, VOCAB, 1.0, True),
        # 12 layers' caches after one tree step of 8 sequences
        _commit("commit bf16", 12, 8, 12, 64, 1024, 8, "bf16"),
    ]


def _kv(name, rows, heads, dim, positions, slots, src, cache, back, fused):
    return {"name": name, "op": "kv", "rows": rows, "heads": heads, "dim": dim, "positions": positions,
            "slots": slots, "src": src, "cache": cache, "back": back, "fused": fused}


def _attn(name, seqs, nodes, heads, kv_heads, dim, positions, lo, hi, q, cache):
    return {"name": name, "op": "attn", "seqs": seqs, "nodes": nodes, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "positions": positions, "lo": lo, "hi": hi, "q": q, "cache": cache}


def _verify(name, seqs, nodes, width, vocab, temperature, dense):
    return {"name": name, "op": "verify", "seqs": seqs, "nodes": nodes, "width": width, "vocab": vocab,
            "temperature": temperature, "dense": dense}


def _commit(name, layers, seqs, heads, dim, positions, nodes, cache):
    return {"name": name, "op": "commit", "layers": layers, "seqs": seqs, "heads": heads, "dim": dim,
            "positions": positions, "nodes": nodes, "cache": cache}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["kv", "attn", "attn", "verify", "commit"])
    dim = rng.choice([32, 64, 128])
    if op == "kv":
        heads = rng.randint(1, 12)
        rows = _log(rng, 1, min(20000, 12_000_000 // (heads * dim)))
        slots = rng.randint(1, 64)
        c = _kv("", rows, heads, dim, max(16, -(-rows // slots) + rng.randint(0, 99)), slots,
                rng.choice(["f32", "f16", "bf16"]), rng.choice(["int8", "int8", "e4m3", "bf16", "f16"]),
                rng.choice(["f32", "f16", "bf16"]), rng.random() < 0.5)
    elif op == "attn":
        kv_heads = rng.randint(1, 12)
        group = rng.choice([1, 1, 1, 2, 4, 8])
        seqs = _log(rng, 1, 64)
        nodes = rng.choice([1, _log(rng, 1, 64), _log(rng, 1, 16)])
        q, cache = rng.choice([("f32", "f32"), ("f32", "bf16"), ("f32", "f16"), ("f32", "int8"), ("bf16", "bf16"),
                               ("f16", "f16"), ("bf16", "int8"), ("f16", "e4m3"), ("f32", "e4m3")])
        # (keys x rows x heads x dim stays below the largest listed case's)
        top = min(8000, 4_000_000_000 // (seqs * nodes * kv_heads * group * dim),
                  400_000_000 // (seqs * kv_heads * dim))
        hi = _log(rng, 1, max(1, top))
        lo = rng.randint(0, hi)
        c = _attn("", seqs, nodes, kv_heads * group, kv_heads, dim, hi + nodes + rng.randint(0, 40), lo, hi, q, cache)
    elif op == "verify":
        seqs, nodes = _log(rng, 1, 64), _log(rng, 1, 16)
        vocab = _log(rng, 300, VOCAB)
        while seqs * nodes > 512:
            nodes = (nodes + 1) // 2
        c = _verify("", seqs, nodes, rng.choice([1, 1, 2, 4]), vocab, rng.choice([0.0, 0.6, 1.0, 1.0, 1.4]),
                    rng.random() < 0.6)
    else:
        seqs, nodes = _log(rng, 1, 32), rng.randint(1, 32)
        c = _commit("", rng.randint(1, 12), seqs, rng.randint(1, 12), dim, nodes + rng.randint(8, 500), nodes,
                    rng.choice(["f32", "f16", "bf16"]))
    del c["name"]
    return c


# ---- inputs ------------------------------------------------------------------------

def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 16 + salt)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _order(g, n):
    return torch.randperm(n, generator=g, device=DEV).to(torch.int32)


def _spread(lo, hi, n):
    """n lengths from lo to hi, the same for every seed."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _shuffled(values, seed):
    import random
    values = list(values)
    random.Random(seed).shuffle(values)
    return values


def _parents(seed, counts, width):
    """Random trees: node i's parent is one of the `width` nodes before it
    (width 1: a chain), as a packed list of indices within the sequence."""
    import random
    r = random.Random(seed + 77)
    return [[-1] + [r.randint(max(0, i - width), i - 1) for i in range(1, n)] for n in counts]


def _masks(parents):
    out = []
    for p in parents:
        m = []
        for i, q in enumerate(p):
            m.append((1 << i) | (m[q] if q >= 0 else 0))
        out += m
    return torch.tensor([v - (1 << 64) if v >> 63 else v for v in out], dtype=torch.int64, device=DEV)


def _first(counts):
    f = [0]
    for n in counts:
        f.append(f[-1] + n)
    return f


def _uniform(g, *shape):
    """Uniform numbers strictly inside (0, 1), as the sampler's: 23 bits and a half."""
    return (torch.randint(0, 1 << 23, shape, generator=g, device=DEV).to(torch.float32) + 0.5) * 2.0 ** -23


def _cache(g, kind, *shape):
    """A filled cache and its scales (None, or [slots][heads][positions])."""
    if kind == "int8":
        return (torch.randint(-127, 128, shape, generator=g, device=DEV).to(torch.int8),
                0.004 + 0.02 * torch.rand(shape[:-1], generator=g, device=DEV))
    if kind == "e4m3":
        e = torch.randint(-9, -6, shape[:-1], generator=g, device=DEV)
        return (_normal(g, *shape) * 100).clamp(-448, 448).to(TYPES[kind]), torch.exp2(e.to(torch.float32))
    return _normal(g, *shape).to(TYPES[kind]), None


def prepare(case, seed):
    s = dict(case)
    g = _gen(seed, 1)
    op = case["op"]
    if op == "kv":
        n, H, D, S, P = case["rows"], case["heads"], case["dim"], case["slots"], case["positions"]
        E = H * D
        rows = _normal(g, n, (3 if case["fused"] else 2) * E)
        rows *= torch.exp(0.5 * _normal(g, 1, rows.shape[1]))   # some dimensions are larger than others
        rows = rows.to(TYPES[case["src"]])
        s["k"], s["v"] = rows[:, -2 * E:-E].view(n, H, D), rows[:, -E:].view(n, H, D)
        per = -(-n // S)
        start = int(torch.randint(0, P - per + 1, (1,), generator=g, device=DEV))
        i = torch.arange(n, device=DEV, dtype=torch.int32)
        s["slot"] = _order(g, S)[(i // per).long()]
        s["pos"] = start + i % per
        for part in "kv":
            s[part + "_cache"] = torch.zeros((S, H, P, D), device=DEV).to(TYPES[case["cache"]])
            s[part + "_scale"] = torch.ones((S, H, P), device=DEV) if case["cache"] in SCALED else None
    elif op == "attn":
        B, H, K, D, P = case["seqs"], case["heads"], case["kv_heads"], case["dim"], case["positions"]
        lens = _shuffled(_spread(case["lo"], case["hi"], B), seed)
        # every sequence but the first may have drafted fewer tokens
        counts = [case["nodes"]] + [max(1, case["nodes"] - i % 4) for i in range(1, B)]
        s["first"], s["cached"] = _i32(_first(counts)), _i32(lens)
        s["mask"] = _masks(_parents(seed, counts, 4))
        s["slot"] = _order(g, B)
        s["k_cache"], s["k_scale"] = _cache(g, case["cache"], B, K, P, D)
        s["v_cache"], s["v_scale"] = _cache(g, case["cache"], B, K, P, D)
        s["q"] = (1.5 * _normal(g, sum(counts), H, D)).to(TYPES[case["q"]])
        s["keys"] = min(P, case["hi"] + case["nodes"])
    elif op == "verify":
        B, T, V = case["seqs"], case["nodes"], case["vocab"]
        counts = [T] + [max(1, T - i % 3) for i in range(1, B)]
        par = _parents(seed, counts, case["width"])
        f = _first(counts)
        n = f[-1]
        s["first"], s["parents"] = _i32(f), _i32([q for p in par for q in p])
        s["logits"] = 3.0 * _normal(g, n, V)
        drafted = s["logits"] + 1.2 * _normal(g, n, V)
        # node i's token is drawn from the draft's distribution at its parent
        up = torch.tensor([f[b] + max(q, 0) for b, p in enumerate(par) for q in p], device=DEV)
        s["tokens"] = (drafted[up] - torch.log(-torch.log(_uniform(g, n, V)))).argmax(1).to(torch.int32)
        s["draft"] = torch.softmax(drafted, 1) if case["dense"] and case["temperature"] > 0 else None
        s["u_accept"] = _uniform(g, n) if case["temperature"] > 0 else None
        s["u_draw"] = _uniform(g, B, V) if case["temperature"] > 0 else None
    else:
        L, B, H, D, P, T = (case[k] for k in ("layers", "seqs", "heads", "dim", "positions", "nodes"))
        s["cached"] = _i32(_shuffled(_spread(0, P - T, B), seed))
        s["slot"] = _order(g, B)
        s["k_cache"], _ = _cache(g, case["cache"], L, B, H, P, D)
        s["v_cache"], _ = _cache(g, case["cache"], L, B, H, P, D)
        # accepted paths: the root, then some of the later nodes in increasing order
        keep = torch.rand((B, T), generator=g, device=DEV) < 0.5
        keep[:, 0] = True
        at = torch.arange(T, device=DEV).expand(B, T)
        s["n_path"] = keep.sum(1).to(torch.int32)
        path = torch.where(keep, at, at + T).sort(1).values
        s["path"] = torch.where(path < T, path, -1).to(torch.int32)
    return s


# ---- one pass ----------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"kv": _plain_kv, "attn": _plain_attn, "verify": _plain_verify, "commit": _plain_commit}[s["op"]](s)


def _run_own(s):
    from transformer_decode_token_gb300 import binding as b
    op = s["op"]
    if op == "kv":
        b.op_kv_store(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slot"], s["pos"], s["k_scale"], s["v_scale"])
        return b.op_kv_load(s["k_cache"], s["v_cache"], s["slot"], s["pos"], s["k_scale"], s["v_scale"],
                            dtype=TYPES[s["back"]])
    if op == "attn":
        return b.op_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["slot"], s["cached"], s["first"], s["mask"],
                                   s["nodes"], s["k_scale"], s["v_scale"])
    if op == "verify":
        return b.op_verify_tree(s["logits"], s["tokens"], s["parents"], s["first"], s["nodes"], s["temperature"],
                                s["draft"], s["u_accept"], s["u_draw"])
    b.op_kv_commit(s["k_cache"], s["v_cache"], s["slot"], s["cached"], s["path"], s["n_path"])
    return s["k_cache"], s["v_cache"]


def _quantise(x, kind):
    """Codes and scales of rows of `dim` values; a row that holds an infinity
    or a NaN gets the scale NaN and codes of zero."""
    x = x.float()
    top = x.abs().amax(-1)
    fine = torch.isfinite(x).all(-1)
    if kind == "int8":      # nearest of x / scale, ties to even
        scale = torch.clamp(top / 127, min=TINY)
        code = torch.round(x.double() / scale.double().unsqueeze(-1)).clamp(-127, 127)
    else:                   # the smallest power of two that brings the row into e4m3's range
        m, e = torch.frexp(top.double() / 448)
        scale = torch.exp2(torch.where(m == 0.5, e - 1, e).clamp(min=-126).double()).float()
        code = x.double() / scale.double().unsqueeze(-1)
    code = torch.where(fine.unsqueeze(-1), code, 0.0).float()
    return code.to(TYPES[kind]), torch.where(fine, scale, torch.nan)


def _plain_kv(s):
    at = (s["slot"].long(), slice(None), s["pos"].long())
    back = []
    for part in "kv":
        cache, scale = s[part + "_cache"], s[part + "_scale"]
        if scale is None:
            cache[at] = s[part].to(cache.dtype)
            back.append(cache[at].to(TYPES[s["back"]]))
        else:
            code, sc = _quantise(s[part], s["cache"])
            cache.view(torch.uint8)[at] = code.view(torch.uint8)
            scale[at] = sc
            back.append((cache.view(torch.uint8)[at].view(cache.dtype).float() * scale[at].unsqueeze(-1))
                        .to(TYPES[s["back"]]))
    return tuple(back)


def _widened(cache, scale, slot, keys):
    """Rows 0..keys-1 of the named slots in fp32."""
    if cache.dtype == torch.float8_e4m3fn:
        x = cache.view(torch.uint8)[slot, :, :keys].view(cache.dtype).float()
    else:
        x = cache[slot, :, :keys].float()
    return x if scale is None else x * scale[slot, :, :keys].unsqueeze(-1)


def _plain_attn(s):
    q, T, L = s["q"], s["nodes"], s["keys"]
    n, H, D = q.shape
    slot, cached, first = s["slot"].long(), s["cached"].long(), s["first"].long()
    B, K = slot.numel(), s["k_cache"].shape[1]
    G = H // K
    row = torch.arange(n, device=DEV)
    b = torch.searchsorted(first, row, right=True) - 1
    t = row - first[b]
    qp = torch.zeros((B, T, H, D), device=DEV)
    qp[b, t] = q.float()
    bits = torch.zeros((B, T), dtype=torch.int64, device=DEV)
    bits[b, t] = s["mask"]
    key = torch.arange(L, device=DEV)
    j = key - cached.unsqueeze(1)                                    # [B][L]: the node at a cache row
    count = (first[1:] - first[:-1]).unsqueeze(1)
    node = (j >= 0) & (j < count)
    seen = (bits.unsqueeze(2) >> j.clamp(0, 63).unsqueeze(1)) & 1
    see = (j < 0).unsqueeze(1) | (node.unsqueeze(1) & (seen != 0))   # [B][T][L]
    k = _widened(s["k_cache"], s["k_scale"], slot, L)
    v = _widened(s["v_cache"], s["v_scale"], slot, L)
    v = torch.where(((j < 0) | node)[:, None, :, None], v, 0.0)
    qg = qp.view(B, T, K, G, D).permute(0, 2, 3, 1, 4).reshape(B, K, G * T, D)
    a = torch.matmul(qg, k.transpose(2, 3)).view(B, K, G, T, L) * (1.0 / math.sqrt(D))
    a = torch.where(see[:, None, None], a, -torch.inf)
    top = a.amax(-1, keepdim=True)
    p = torch.exp(a - torch.where(top == -torch.inf, 0.0, top))
    p = torch.where(see[:, None, None], p, 0.0)
    z = p.sum(-1).view(B, K, G * T, 1)
    o = torch.matmul(p.view(B, K, G * T, L), v)
    o = torch.where(z > 0, o / z, 0.0)
    o = o.view(B, K, G, T, D).permute(0, 3, 1, 2, 4).reshape(B, T, H, D)
    return o[b, t].to(q.dtype)


def _packed(first, B, T, n):
    """The packed row of each (sequence, node), and which nodes there are."""
    at = first[:-1].unsqueeze(1) + torch.arange(T, device=DEV)
    there = at < first[1:].unsqueeze(1)
    return torch.where(there, at, 0).clamp(max=n - 1), there


def _plain_verify(s):
    n, V = s["logits"].shape
    first, T, B = s["first"].long(), s["nodes"], s["first"].numel() - 1
    at, there = _packed(first, B, T, n)
    parent = torch.where(there, s["parents"].long()[at], -2)
    token = s["tokens"].long()[at]
    seq = torch.arange(B, device=DEV)
    cur = torch.zeros(B, dtype=torch.long, device=DEV)
    path = torch.full((B, T), -1, dtype=torch.long, device=DEV)
    path[:, 0] = torch.where(there[:, 0], 0, -1)
    length = there[:, 0].long()
    greedy = s["temperature"] == 0
    # (probabilities in 64 bits: an acceptance is a comparison)
    p = s["logits"] if greedy else torch.softmax(s["logits"].double() / s["temperature"], 1)
    best = p.argmax(1) if greedy else None
    left = None if greedy else p[at[:, 0]].clone()
    for i in range(1, T):
        tried = parent[:, i] == cur
        x, row = token[:, i], at[seq, cur]
        if greedy:
            yes = tried & (best[row] == x)
        else:
            q = torch.nn.functional.one_hot(x, V).double() if s["draft"] is None else s["draft"][row].double()
            yes = tried & (s["u_accept"][at[:, i]].double() * q[seq, x] < left[seq, x])
            less = (left - q).clamp(min=0)
            mass = less.sum(1, keepdim=True)
            less = torch.where(mass > 0, less / mass, 0.0)
            left = torch.where((tried & ~yes).unsqueeze(1), less, left)
            left = torch.where(yes.unsqueeze(1), p[at[:, i]], left)
        path[seq, length.clamp(max=T - 1)] = torch.where(yes, i, path[seq, length.clamp(max=T - 1)])
        length = length + yes.long()
        cur = torch.where(yes, i, cur)
    last = at[seq, cur]
    if greedy:
        token = best[last]
    else:
        left = torch.where(left.sum(1, keepdim=True) > 0, left, p[last])
        token = (left / -torch.log(s["u_draw"].double())).argmax(1)
    return path.to(torch.int32), length.to(torch.int32), torch.where(there[:, 0], token, -1).to(torch.int32)


def _plain_commit(s):
    slot, cached, path = s["slot"].long().unsqueeze(1), s["cached"].long().unsqueeze(1), s["path"].long()
    to = cached + torch.arange(path.shape[1], device=DEV)
    src = torch.where(path >= 0, cached + path, to)
    for c in (s["k_cache"], s["v_cache"]):
        c[:, slot, :, to] = c[:, slot, :, src]
    return s["k_cache"], s["v_cache"]


# ---- what a pass cannot do without ---------------------------------------------------

def work(case):
    op = case["op"]
    if op == "kv":
        values = 2 * case["rows"] * case["heads"] * case["dim"]
        scales = 2 * case["rows"] * case["heads"] * 4 if case["cache"] in SCALED else 0
        return {"bytes": values * (SIZE[case["src"]] + 2 * SIZE[case["cache"]] + SIZE[case["back"]]) + 2 * scales,
                "flops": 4 * values}
    if op == "attn":
        B, T, D = case["seqs"], case["nodes"], case["dim"]
        counts = [T] + [max(1, T - i % 4) for i in range(1, B)]
        lens = _spread(case["lo"], case["hi"], B)
        per_key = case["kv_heads"] * 2 * (D * SIZE[case["cache"]] + (4 if case["cache"] in SCALED else 0))
        keys = sum(lens) + sum(counts)
        pairs = sum(counts) * (sum(lens) / B) + sum(c * c for c in counts) / 2
        return {"bytes": keys * per_key + 2 * sum(counts) * case["heads"] * D * SIZE[case["q"]],
                "flops": 4 * pairs * case["heads"] * D}
    if op == "verify":
        B, T, V = case["seqs"], case["nodes"], case["vocab"]
        n = T + sum(max(1, T - i % 3) for i in range(1, B))
        drawn = case["temperature"] > 0
        # every logit once; per sequence the uniform numbers of the final draw
        # and the draft's distribution at the node where the path ends
        rows = n + (B if drawn else 0) + (B if drawn and case["dense"] else 0)
        return {"bytes": rows * V * 4, "flops": n * V * 4}
    # half of the nodes are accepted, and nearly all of those move
    moved = case["layers"] * case["seqs"] * max(1, (case["nodes"] - 1) // 2) * case["heads"] * case["dim"]
    return {"bytes": 2 * 2 * moved * SIZE[case["cache"]], "flops": 0}


# ---- the operators in 64 bits --------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "kv":
        return _exact_kv(s)
    if case["op"] == "attn":
        return _exact_attn(s)
    if case["op"] == "commit":
        return _exact_commit(s)
    return None     # whole numbers


def _exact_kv(s):
    out = []
    for part in "kv":
        x = s[part].double()
        if s["cache"] == "int8":
            step = (x.abs().max(-1, keepdim=True).values.float() / 127).double()
            y = torch.round(x / step) * step
        elif s["cache"] == "e4m3":
            step = torch.exp2(torch.ceil(torch.log2(x.abs().max(-1, keepdim=True).values / 448)))
            z = x / step
            # e4m3: three fraction bits, exponents down to -6
            ulp = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
            y = torch.round(z / ulp) * ulp * step
        else:
            y = x.to(TYPES[s["cache"]]).double()
        out.append(y)
    return tuple(out)


def _exact_attn(s):
    q, first, cached, slot = s["q"].double(), s["first"].tolist(), s["cached"].tolist(), s["slot"].tolist()
    n, H, D = q.shape
    K = s["k_cache"].shape[1]
    out = torch.zeros_like(q)
    for b in range(len(slot)):
        lo, hi, c = first[b], first[b + 1], cached[b]
        T = hi - lo
        kv = []
        for part in "kv":
            x = s[part + "_cache"][slot[b], :, :c + T].double()
            if s[part + "_scale"] is not None:
                x = x * s[part + "_scale"][slot[b], :, :c + T, None].double()
            kv.append(x.repeat_interleave(H // K, 0))
        a = torch.einsum("thd,hld->htl", q[lo:hi], kv[0]) / math.sqrt(D)
        see = torch.ones((T, c + T), dtype=torch.bool, device=DEV)
        see[:, c:] = (s["mask"][lo:hi, None] >> torch.arange(T, device=DEV)) & 1 == 1
        w = torch.softmax(a.masked_fill(~see, -math.inf), -1)
        out[lo:hi] = torch.einsum("htl,hld->thd", torch.nan_to_num(w), kv[1])
    return out


def _exact_commit(s):
    slot, cached, path = s["slot"].tolist(), s["cached"].tolist(), s["path"].tolist()
    out = []
    for part in "kv":
        x = s[part + "_cache"].clone()
        for b, c in enumerate(cached):
            for i, node in enumerate(path[b]):
                if node > i:
                    x[:, slot[b], :, c + i] = s[part + "_cache"][:, slot[b], :, c + node]
        out.append(x.double())
    return tuple(out)
