"""What the operators of a served step over a paged cache compute, and what they cost.

Three operators that follow one another in a step: the block tables and the
slot map of the step's tokens, built on the GPU from the requests' lengths;
the attention of each new token over its request's pages; and the choice of
the next tokens by temperature, top-k, top-p and min-p from given random
numbers.  For each there are cases (listed() and draw()), their inputs
(prepare()), one pass (run(): the plain form in torch, or, with `own`, the
calls into transformer_decode_token_gb300.binding), the bytes and operations a
pass cannot do without (work()), and the result in 64 bits (exact()).

Layouts.  A paged cache is [blocks][heads][block size][dim]; an int8 or e4m3
cache has one fp32 scale per (block, head, offset) for the keys and one for the
values.  Sequence b's position p lies in block table[b][p // block size], at
offset p % block size.  The free blocks are a ring [blocks] with (next, count);
blocks are taken at its front and given back at its end.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "int8": torch.int8,
         "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "int8": 1, "e4m3": 1}
SCALED = ("int8", "e4m3")
VOCAB = 50257


# ---- the cases ---------------------------------------------------------------------

def listed():
    return [
        # one decode step of 64 requests, a token each: latency
        _map("pages decode step", 64, 16, 64, 32, 1000, "decode", 64, False),
        # a step that decodes most requests, begins some prompts and lets some requests go
        _map("pages mixed step", 256, 16, 64, 32, 900, "mixed", 16384, False),
        # 64 long prompts at once, with too few free blocks for all of them
        _map("pages prompts, few free", 64, 64, 128, 256, 1500, "prompts", 65536, True),
        # one request, GPT-2's heads, fp32: latency of one layer
        _attn("one request f32", 1, 1, 12, 12, 64, 16, 1000, 1000, "f32", "f32"),
        # the batched decode step's attention (64 requests) over bf16 pages of 16
        _attn("decode step bf16", 64, 1, 12, 12, 64, 16, 32, 575, "f32", "bf16"),
        # long contexts over int8 pages of 32
        _attn("long contexts int8", 32, 1, 12, 12, 64, 32, 3000, 8000, "f32", "int8"),
        # grouped heads, few requests with long contexts of very different lengths
        _attn("grouped heads long bf16", 8, 1, 32, 8, 128, 64, 1000, 16000, "bf16", "bf16"),
        # eight query heads on a cache head, many requests, int8 pages
        _attn("grouped heads int8", 128, 1, 16, 2, 128, 16, 100, 3000, "bf16", "int8"),
        # one request's next token, top-p over GPT-2's vocabulary: latency
        _sample("sample one row top-p", 1, VOCAB, "f32", 0.8, 0, 0.95, 0.0, False, 0),
        # a batched step's 64 rows, top-k and top-p
        _sample("sample 64 rows top-k top-p", 64, VOCAB, "f32", 0.8, 50, 0.9, 0.0, False, 0),
        # the whole distribution, nothing cut
        _sample("sample 64 rows all", 64, VOCAB, "f32", 1.0, 0, 1.0, 0.0, False, 0),
        # requests with settings of their own (greedy ones among them), bf16 rows with padding behind them
        _sample("sample 256 rows mixed bf16", 256, VOCAB, "bf16", 0.9, 40, 0.95, 0.05, True, 47),
    ]


def _map(name, seqs, block, max_blocks, lo, hi, kind, rows, tight):
    return {"name": name, "op": "map", "seqs": seqs, "block": block, "max_blocks": max_blocks, "lo": lo, "hi": hi,
            "kind": kind, "rows": rows, "tight": tight}


def _attn(name, seqs, new, heads, kv_heads, dim, block, lo, hi, q, cache):
    return {"name": name, "op": "attn", "seqs": seqs, "new": new, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "block": block, "lo": lo, "hi": hi, "q": q, "cache": cache}


def _sample(name, rows, vocab, dtype, temperature, top_k, top_p, min_p, mixed, pad):
    return {"name": name, "op": "sample", "rows": rows, "vocab": vocab, "dtype": dtype, "temperature": temperature,
            "top_k": top_k, "top_p": top_p, "min_p": min_p, "mixed": mixed, "pad": pad}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["map", "attn", "attn", "attn", "sample", "sample"])
    if op == "map":
        block = rng.choice([8, 16, 16, 32, 64, 24])
        seqs, max_blocks = _log(rng, 1, 1000), rng.randint(8, 128)
        hi = rng.randint(1, block * max_blocks - 1)
        kind = rng.choice(["decode", "decode", "mixed", "prompts"])
        rows = seqs if kind == "decode" else min(65536, max(64, seqs * (hi if kind == "prompts" else 64)))
        c = _map("", seqs, block, max_blocks, rng.randint(0, hi), hi, kind, rows, rng.random() < 0.3)
    elif op == "attn":
        dim = rng.choice([32, 64, 64, 128])
        kv_heads = rng.randint(1, 12)
        group = rng.choice([1, 1, 1, 2, 4, 8, 12])
        seqs = _log(rng, 1, 200)
        new = rng.choice([1, 1, 1, 1, rng.randint(2, 6)])
        q, cache = rng.choice([("f32", "f32"), ("f32", "bf16"), ("f32", "f16"), ("f32", "int8"), ("bf16", "bf16"),
                               ("f16", "f16"), ("bf16", "int8"), ("f16", "e4m3"), ("f32", "e4m3"), ("f16", "int8")])
        # (rows x keys x heads x dim stays below the largest listed case's)
        top = min(16000, 120_000_000 // (seqs * kv_heads * dim), 500_000_000 // (seqs * new * kv_heads * group * dim))
        hi = _log(rng, 1, max(1, top))
        c = _attn("", seqs, new, kv_heads * group, kv_heads, dim, rng.choice([8, 16, 16, 32, 64, 128, 24]),
                  rng.randint(0, hi), hi, q, cache)
    else:
        rows, vocab = _log(rng, 1, 256), _log(rng, 300, 130000)
        while rows * vocab > 256 * VOCAB:
            rows = (rows + 1) // 2
        c = _sample("", rows, vocab, rng.choice(["f32", "f32", "bf16", "f16"]), rng.choice([0.5, 0.7, 1.0, 1.3]),
                    rng.choice([0, 0, 1, 20, 50, 200, 1000]), rng.choice([1.0, 0.5, 0.9, 0.99]),
                    rng.choice([0.0, 0.0, 0.02, 0.1]), rng.random() < 0.3, rng.choice([0, 0, 3, 64]))
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
    values = list(values)
    random.Random(seed).shuffle(values)
    return values


def _uniform(g, *shape):
    """Uniform numbers strictly inside (0, 1), as the sampler's: 23 bits and a half."""
    return (torch.randint(0, 1 << 23, shape, generator=g, device=DEV).to(torch.float32) + 0.5) * 2.0 ** -23


def _cache(g, kind, *shape):
    """A filled cache and its scales (None, or one per row)."""
    if kind == "int8":
        return (torch.randint(-127, 128, shape, generator=g, device=DEV).to(torch.int8),
                0.004 + 0.02 * torch.rand(shape[:-1], generator=g, device=DEV))
    if kind == "e4m3":
        e = torch.randint(-9, -6, shape[:-1], generator=g, device=DEV)
        return (_normal(g, *shape) * 100).clamp(-448, 448).to(TYPES[kind]), torch.exp2(e.to(torch.float32))
    return _normal(g, *shape).to(TYPES[kind]), None


def _requests(case):
    """(cached, grow) of the step's requests, the same for every seed."""
    out = []
    for i, n in enumerate(_spread(case["lo"], case["hi"], case["seqs"])):
        if case["kind"] == "prompts" or (case["kind"] == "mixed" and i % 8 == 0):
            out.append((0, min(n, 512) if case["kind"] == "mixed" else n))
        elif case["kind"] == "mixed" and i % 16 == 5:
            out.append((n, -1))
        else:
            out.append((n, 1))
    return out


def _blocks(n, block):
    return -(-n // block)


def prepare(case, seed):
    s = dict(case)
    g = _gen(seed, 3)
    op = case["op"]
    if op == "map":
        bs, width = case["block"], case["max_blocks"]
        asked = _shuffled(_requests(case), seed)
        have = [_blocks(c, bs) for c, _ in asked]
        need = sum(_blocks(c + n, bs) - _blocks(c, bs) for c, n in asked if n > 0)
        held = sum(have)
        free = need * 2 // 3 if case["tight"] else need + 100
        order = _order(g, held + free)
        s["table"] = torch.full((len(asked), width), -1, dtype=torch.int32, device=DEV)
        at = torch.arange(width, device=DEV) < torch.tensor(have, device=DEV).unsqueeze(1)
        s["table"][at] = order[:held]
        n = held + free
        head = int(torch.randint(0, n, (1,), generator=g, device=DEV)) if n else 0
        s["free"] = torch.full((max(n, 1),), -1, dtype=torch.int32, device=DEV)
        s["free"][(head + torch.arange(free, device=DEV)) % max(n, 1)] = order[held:]
        s["state"] = _i32([head, free])
        s["cached"], s["grow"] = _i32([c for c, _ in asked]), _i32([n for _, n in asked])
    elif op == "attn":
        B, T, H, K, D, bs = (case[k] for k in ("seqs", "new", "heads", "kv_heads", "dim", "block"))
        lens = _shuffled(_spread(case["lo"], case["hi"], B), seed)
        have = [_blocks(n + T, bs) for n in lens]
        n = sum(have) + 3
        width = max(have)
        s["table"] = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        at = torch.arange(width, device=DEV) < torch.tensor(have, device=DEV).unsqueeze(1)
        s["table"][at] = _order(g, n)[:sum(have)]
        s["k_cache"], s["k_scale"] = _cache(g, case["cache"], n, K, bs, D)
        s["v_cache"], s["v_scale"] = _cache(g, case["cache"], n, K, bs, D)
        s["position"] = _i32([n + t for n in lens for t in range(T)])
        s["seq"] = None if T == 1 else _i32([b for b in range(B) for _ in range(T)])
        s["q"] = (1.5 * _normal(g, B * T, H, D)).to(TYPES[case["q"]])
    else:
        n, V = case["rows"], case["vocab"]
        x = _normal(g, n, V + case["pad"])
        # some ids stand out, in some rows more than in others
        x = (2.0 * x + 6.0 * (x - 2.0).clamp(min=0)) * torch.exp(0.3 * _normal(g, n, 1))
        s["logits"] = x.to(TYPES[case["dtype"]])[:, :V]
        s["u"] = _uniform(g, n, V)
        i = torch.arange(n, device=DEV)
        t, k, p, m = (torch.full((n,), float(case[x]), device=DEV) for x in ("temperature", "top_k", "top_p", "min_p"))
        if case["mixed"]:       # greedy, plain, top-k and top-p, min-p in turn
            t[i % 4 == 0] = 0.0
            k[i % 4 != 2], p[i % 4 != 2], m[i % 4 != 3] = 0.0, 1.0, 0.0
        s["temperature_"], s["top_k_"], s["top_p_"], s["min_p_"] = t, k.to(torch.int32), p, m
    return s


# ---- one pass ----------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"map": _plain_map, "attn": _plain_attn, "sample": _plain_sample}[s["op"]](s)


def _run_own(s):
    from transformer_decode_token_gb300 import binding as b
    if s["op"] == "map":
        return b.op_page_map(s["cached"], s["grow"], s["table"], s["free"], s["state"], s["block"],
                             s["rows"]) + (s["table"], s["free"])
    if s["op"] == "attn":
        return b.op_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["position"], s["seq"],
                                    s["k_scale"], s["v_scale"])
    return b.op_sample(s["logits"], s["temperature_"], s["u"], s["top_k_"], s["top_p_"], s["min_p_"])


def _plain_map(s):
    bs, n_rows, table, ring = s["block"], s["rows"], s["table"].long(), s["free"].clone()
    B, width = table.shape
    n, (head, count) = ring.numel(), s["state"].long()
    cached, grow = s["cached"].long(), s["grow"].long()
    more, leaves = grow.clamp(min=0), grow < 0
    end = torch.cumsum(more, 0)
    have, want = (cached + bs - 1) // bs, (cached + more + bs - 1) // bs
    fits = ~leaves & (end <= n_rows) & (want <= width)
    need = torch.where(fits, want - have, 0)
    total = torch.cumsum(need, 0)
    served = fits & ((need == 0) | (total <= count))
    # blocks for the served, from the front of the ring; blocks of those that leave, to its end
    at = torch.arange(width, device=DEV)
    taken = served.unsqueeze(1) & (at >= have.unsqueeze(1)) & (at < want.unsqueeze(1))
    rank = (total - need).unsqueeze(1) + at - have.unsqueeze(1)
    given = torch.where(leaves, have, 0)
    back = leaves.unsqueeze(1) & (at < have.unsqueeze(1))
    after = (torch.cumsum(given, 0) - given).unsqueeze(1) + at
    table = torch.where(taken, ring[(head + rank) % n].long(), table)
    ring[((head + count + after) % n)[back]] = table[back].to(torch.int32)
    out = torch.where(leaves, 0, cached + torch.where(served, more, 0))
    used = torch.where(served, need, 0).sum()
    state = torch.stack([(head + used) % n, count - used + given.sum()])
    # the tokens, one after another
    first = torch.cat([end.new_zeros(1), end]).clamp(max=n_rows)
    i = torch.arange(n_rows, device=DEV)
    b = torch.searchsorted(end, i, right=True)
    there = b < B
    b = b.clamp(max=B - 1)
    p = cached[b] + i - (end - more)[b]
    yes = there & served[b]
    slot = torch.where(yes, table[b, (p // bs).clamp(0, width - 1)], -1)
    return tuple(x.to(torch.int32) for x in (
        out, state, first, torch.where(there, b, -1), slot, torch.where(yes, p % bs, -1), torch.where(yes, p, -1), table,
        ring))


def _paged(s, part):
    """Every request's keys or values, [requests][heads][keys][dim], in fp32."""
    cache, scale, table = s[part + "_cache"], s[part + "_scale"], s["table"].long().clamp(min=0)
    if cache.dtype == torch.float8_e4m3fn:
        x = cache.view(torch.uint8)[table].view(cache.dtype).float()
    else:
        x = cache[table].float()
    if scale is not None:
        x = x * scale[table].unsqueeze(-1)
    B, nb, K, bs, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, K, nb * bs, D)


def _plain_attn(s):
    q, B, T, K = s["q"], s["seqs"], s["new"], s["kv_heads"]
    n, H, D = q.shape
    G = H // K
    k = _paged(s, "k")
    L = k.shape[2]
    qg = q.float().view(B, T, K, G, D).permute(0, 2, 1, 3, 4).reshape(B, K, T * G, D)
    a = torch.matmul(qg, k.transpose(2, 3)).view(B, K, T, G, L) * (1.0 / math.sqrt(D))
    del k
    see = torch.arange(L, device=DEV) <= s["position"].view(B, 1, T, 1, 1)
    a = torch.where(see, a, -torch.inf)
    p = torch.where(see, torch.exp(a - a.amax(-1, keepdim=True)), 0.0)
    z = p.sum(-1, keepdim=True)
    v = _paged(s, "v")
    o = torch.matmul(p.view(B, K, T * G, L), v).view(B, K, T, G, D) / z
    return o.permute(0, 2, 1, 3, 4).reshape(n, H, D).to(q.dtype)


def _plain_sample(s):
    n, V = s["logits"].shape
    t = s["temperature_"].double().unsqueeze(1)
    # highest first, ties to the lowest id (weights in 64 bits: a cut is a comparison)
    top, order = s["logits"].float().sort(dim=1, descending=True, stable=True)
    w = torch.exp((top.double() - top[:, :1].double()) / torch.where(t > 0, t, 1.0))
    at = torch.arange(V, device=DEV)
    k = s["top_k_"].long().unsqueeze(1)
    w = torch.where((k > 0) & (at >= k), 0.0, w)
    total = torch.cumsum(w, 1)
    keep = (total - w < s["top_p_"].double().unsqueeze(1) * total[:, -1:]) | (at == 0)
    w = torch.where(keep & (w >= s["min_p_"].double().unsqueeze(1)), w, 0.0)
    race = w / -torch.log(s["u"].double().gather(1, order))
    won = torch.where(t > 0, race.argmax(1, keepdim=True), 0)
    prob = torch.where(t > 0, w.gather(1, won) / w.sum(1, keepdim=True), 1.0)
    return order.gather(1, won).squeeze(1).to(torch.int32), prob.squeeze(1).float()


# ---- what a pass cannot do without ---------------------------------------------------

def work(case):
    op = case["op"]
    if op == "map":
        asked = _requests(case)
        bs = case["block"]
        new = sum(_blocks(c + n, bs) - _blocks(c, bs) for c, n in asked if n > 0)
        gone = sum(_blocks(c, bs) for c, n in asked if n < 0)
        old = sum(1 for c, n in asked if n > 0 and c % bs)       # half-filled blocks that tokens go to
        # lengths in and out, four numbers a row, table entries read and written, the ring
        return {"bytes": 4 * (4 * len(asked) + 4 * case["rows"] + old + 2 * (new + gone)), "flops": 0}
    if op == "attn":
        B, T, D, bs = case["seqs"], case["new"], case["dim"], case["block"]
        lens = _spread(case["lo"], case["hi"], B)
        per_key = case["kv_heads"] * 2 * (D * SIZE[case["cache"]] + (4 if case["cache"] in SCALED else 0))
        keys = sum(n + T for n in lens)
        pairs = sum((n + t + 1) for n in lens for t in range(T))
        return {"bytes": keys * per_key + 4 * sum(_blocks(n + T, bs) for n in lens) +
                2 * B * T * case["heads"] * D * SIZE[case["q"]], "flops": 4 * pairs * case["heads"] * D}
    n, V = case["rows"], case["vocab"]
    # every logit; the random numbers of the ids that are left: of all of them where nothing is cut
    plain = 0.25 if case["mixed"] else 1.0 if case["top_k"] == 0 and case["top_p"] == 1 and case["min_p"] == 0 else 0.0
    return {"bytes": n * V * (SIZE[case["dtype"]] + 4 * plain), "flops": n * V * 4}


# ---- the operators in 64 bits --------------------------------------------------------

def exact(case, seed):
    if case["op"] == "map":
        return None     # whole numbers
    s = prepare(case, seed)
    return _exact_attn(s) if case["op"] == "attn" else _exact_sample(s)


def _exact_attn(s):
    q, K, bs = s["q"].double(), s["kv_heads"], s["block"]
    n, H, D = q.shape
    out = torch.zeros_like(q)
    for i, last in enumerate(s["position"].tolist()):
        b = i // s["new"]
        j = torch.arange(last + 1, device=DEV)
        block, offset = s["table"][b].long()[j // bs], j % bs
        kv = []
        for part in "kv":
            c = s[part + "_cache"]
            x = c.view(torch.uint8)[block, :, offset].view(c.dtype).double() if c.dtype == torch.float8_e4m3fn else \
                c[block, :, offset].double()
            if s[part + "_scale"] is not None:
                x = x * s[part + "_scale"][block, :, offset].double().unsqueeze(-1)
            kv.append(x)
        a = torch.einsum("kgd,lkd->kgl", q[i].view(K, H // K, D), kv[0]) / math.sqrt(D)
        out[i] = torch.einsum("kgl,lkd->kgd", torch.softmax(a, -1), kv[1]).reshape(H, D)
    return out


def _exact_sample(s):
    prob = torch.ones(s["rows"], dtype=torch.float64, device=DEV)
    settings = zip(*(s[x].tolist() for x in ("temperature_", "top_k_")))
    for i, (t, k) in enumerate(settings):
        if t == 0:
            continue
        # (the settings are fp32 numbers)
        p, m = s["top_p_"][i].double(), s["min_p_"][i].double()
        l = s["logits"][i].double() / s["temperature_"][i].double()
        ids = torch.argsort(l, descending=True, stable=True)
        ids = ids[:k] if k > 0 else ids
        r = torch.softmax(l[ids], 0)
        n = ids.numel() if p >= 1 else 1 + int((torch.cumsum(r, 0)[:-1] < p).sum())
        n = min(n, max(1, int((r >= m * r[0]).sum())))
        r = r[:n] / r[:n].sum()
        prob[i] = r[(torch.log(r) - torch.log(-torch.log(s["u"][i, ids[:n]].double()))).argmax()]
    return None, prob
