"""A served step in one piece: requests of a small GPT-2 whose layers keep their
keys and values in shared pages (page_map, kv_store, paged_attention, sample),
against the CPU oracle; and sampling on the batched model."""
import math

import numpy as np
import pytest

from oracle import oracle as orc
from transformer_decode_token_gb300 import binding, synth

from gpu_util import max_abs, top2_margin
from test_gpu_sample import sample64
from test_gpu_spec import dt, i32, uniform

pytestmark = pytest.mark.gpu

ATOL = 2e-3                    # as for the batched model's logits (test_gpu_batch.py)


class Server:
    """GPT-2 over paged caches, its products by torch in fp32."""

    def __init__(self, cfg, w, blocks, block, requests, width, kind):
        import torch
        self.cfg, self.kind = cfg, kind
        self.w = binding.upload_weights(w)
        H, D = cfg.n_head, cfg.n_embd // cfg.n_head
        shape = (blocks, H, block, D)
        self.block = block
        self.cache = [[torch.full(shape, 1.0, device="cuda").to(dt(kind)) for _ in "kv"] for _ in range(cfg.n_layer)]
        scaled = kind in ("int8", "e4m3")
        self.scale = [[torch.ones(shape[:3], device="cuda") if scaled else None for _ in "kv"]
                      for _ in range(cfg.n_layer)]
        self.cached = i32(np.zeros(requests))
        self.table = i32(np.full((requests, width), -1))
        self.free, self.state = i32(np.random.default_rng(0).permutation(blocks)), i32([0, blocks])

    def step(self, tokens, grow, rows):
        """tokens: the new rows' ids, packed; returns the rows' logits."""
        import torch
        c = self.cfg
        H, D, E = c.n_head, c.n_embd // c.n_head, c.n_embd
        _, _, first, seq, slot, offset, position = binding.op_page_map(
            self.cached, i32(grow), self.table, self.free, self.state, self.block, rows, self.cached, self.state)
        at = position.long().clamp(min=0)
        x = self.w["wte"][i32(tokens).long()] + self.w["wpe"][at]
        for L, (kc, vc), (ks, vs) in zip(self.w["layers"], self.cache, self.scale):
            h = binding.op_layernorm(x, L["ln1_w"], L["ln1_b"], c.ln_eps)
            qkv = torch.addmm(L["attn_b"], h, L["attn_w"])
            q, k, v = (qkv[:, i * E:(i + 1) * E].unflatten(1, (H, D)) for i in range(3))
            binding.op_kv_store(k, v, kc, vc, slot, offset, ks, vs)
            a = binding.op_paged_attention(q, kc, vc, self.table, position, seq, ks, vs)
            x = x + torch.addmm(L["proj_b"], a.flatten(1), L["proj_w"])
            h = binding.op_layernorm(x, L["ln2_w"], L["ln2_b"], c.ln_eps)
            f = torch.nn.functional.gelu(torch.addmm(L["fc_b"], h, L["fc_w"]), approximate="tanh")
            x = x + torch.addmm(L["mlp_proj_b"], f, L["mlp_proj_w"])
        h = binding.op_layernorm(x, self.w["ln_f_w"], self.w["ln_f_b"], c.ln_eps)
        return h @ self.w["wte"].t(), first


@pytest.mark.parametrize("kind,block", [("f32", 4), ("f32", 7), ("bf16", 8)])
def test_requests_come_and_go(kind, block):
    """Requests begin with prompts, decode greedily, leave and make room for others,
    all in one batch; the logits of every request's tokens are the oracle's."""
    cfg = synth.TINY
    w = synth.make_weights(cfg, 0)
    rng = np.random.default_rng(block)
    requests, width = 5, -(-40 // block)
    s = Server(cfg, w, requests * width // 2 + 3, block, requests, width, kind)
    prompts = [[int(t) for t in rng.integers(0, cfg.vocab_size, n)] for n in (9, 1, 17, 5, 12, 3, 8)]
    kv = "bf16" if kind == "bf16" else "f32"
    ref = [orc.greedy(cfg, w, p, 8, omp=True, kv=kv) for p in prompts]
    waiting, active, done = list(range(len(prompts))), {}, 0
    rows = 32
    for step in range(40):
        grow, tokens, parts = np.zeros(requests, np.int64), [], []
        for b in range(requests):
            if b in active:
                r, ids = active[b]
                if len(ids) == len(prompts[r]) + 8:
                    grow[b] = -1
                    del active[b]
                    done += 1
                    continue
                new = ids[-1:]
            elif waiting and len(tokens) + len(prompts[waiting[0]]) <= rows:
                r = waiting.pop(0)
                ids = list(prompts[r])
                active[b] = (r, ids)
                new = ids
            else:
                continue
            grow[b] = len(new)
            tokens += new
            parts.append((b, len(new)))
        before = s.cached.cpu().numpy()
        logits, first = s.step(tokens + [0] * (rows - len(tokens)), grow, rows)
        after = s.cached.cpu().numpy()
        first = first.cpu().numpy()
        for b, n in parts:
            if after[b] != before[b] + n:                    # not served: waits for blocks
                assert after[b] == before[b]
                if before[b] == 0:
                    waiting.insert(0, active.pop(b)[0])
                continue
            r, ids = active[b]
            got = logits[first[b] + n - 1].cpu().numpy()
            i, row = after[b] - len(prompts[r]), ref[r][1][after[b] - 1]     # the oracle's choice and pass
            assert max_abs(got, row) <= ATOL, (step, r, i)
            choice = int(got.argmax())
            if top2_margin(row) > 2 * ATOL:
                assert choice == ref[r][0][i]
            ids.append(int(ref[r][0][i]))
        if done == len(prompts):
            break
    assert done == len(prompts)
    assert s.state.tolist()[1] == s.free.numel()             # every block came back


@pytest.mark.parametrize("kind,block", [("int8", 8), ("e4m3", 16)])
def test_quantised_pages_are_the_slabs(kind, block):
    """The same rows in pages and in slabs: attention over pages gives what tree
    attention gives over a slot of its own, in one step of several tokens each."""
    import torch
    rng = np.random.default_rng(3)
    H, D, B = 3, 64, 4
    lens, new = [50, 3, 0, 31], [1, 4, 2, 1]
    width = -(-60 // block)
    kc, vc = (torch.zeros((B * width, H, block, D), device="cuda").to(dt(kind)) for _ in "kv")
    ks, vs = (torch.ones((B * width, H, block), device="cuda") for _ in "kv")
    ks2, vs2 = (torch.ones((B, H, 60), device="cuda") for _ in "kv")
    kc2, vc2 = (torch.zeros((B, H, 60, D), device="cuda").to(dt(kind)) for _ in "kv")
    table, ring, state, cached = i32(np.full((B, width), -1)), i32(rng.permutation(B * width)), i32([0, B * width]), i32([0] * B)
    for grow in (lens, new):
        n = sum(grow)
        before = cached.clone()
        _, _, first, seq, slot, offset, position = binding.op_page_map(cached, i32(grow), table, ring, state, block, n,
                                                                       cached, state)
        k, v, q = (torch.from_numpy(rng.standard_normal((n, H, D)).astype(np.float32)).cuda() for _ in range(3))
        binding.op_kv_store(k, v, kc, vc, slot, offset, ks, vs)
        binding.op_kv_store(k, v, kc2, vc2, seq, position, ks2, vs2)
    got = binding.op_paged_attention(q, kc, vc, table, position, seq, ks, vs)
    masks = np.concatenate([binding.tree_masks(list(range(-1, m - 1))) for m in new])
    want = binding.op_tree_attention(q, kc2, vc2, i32(range(B)), before, first, torch.from_numpy(masks).cuda(), 4, ks2, vs2)
    # (both are fp32 sums of the same values, in another order)
    assert (got - want).abs().max().item() <= 1e-5


def test_a_captured_step():
    """page_map in place, kv_store, attention and sampling captured once and
    replayed for many tokens: every replay goes on where the last one ended."""
    import torch
    rng = np.random.default_rng(5)
    B, H, D, block, width, V = 6, 2, 64, 8, 10, 300
    kc, vc = (torch.zeros((B * width, H, block, D), device="cuda") for _ in "kv")
    table, ring, state, cached = i32(np.full((B, width), -1)), i32(rng.permutation(B * width)), i32([0, B * width]), i32([0] * B)
    grow = i32([1] * B)
    k, v, q = (torch.zeros((B, H, D), device="cuda") for _ in range(3))
    head = torch.from_numpy(rng.standard_normal((H * D, V)).astype(np.float32)).cuda()
    t, p, u = torch.full((B,), 0.8, device="cuda"), torch.full((B,), 0.9, device="cuda"), torch.full((B, V), 0.5, device="cuda")

    def step():
        _, _, _, _, slot, offset, position = binding.op_page_map(cached, grow, table, ring, state, block, B, cached, state)
        binding.op_kv_store(k, v, kc, vc, slot, offset)
        o = binding.op_paged_attention(q, kc, vc, table, position)
        logits = o.flatten(1) @ head
        return o, position, logits, binding.op_sample(logits, t, u, top_p=p)

    kept = [x.clone() for x in (table, ring, state, cached)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip((table, ring, state, cached), kept):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, position, logits, (token, prob) = step()
    ks, vs = [], []
    for n in range(30):
        for x in (k, v, q):
            x.copy_(torch.from_numpy(rng.standard_normal((B, H, D)).astype(np.float32)))
        uu = uniform(rng, B, V).astype(np.float32)
        u.copy_(torch.from_numpy(uu))
        ks.append(k.double().cpu().numpy())
        vs.append(v.double().cpu().numpy())
        graph.replay()
        torch.cuda.synchronize()
        assert position.tolist() == [n] * B
        a = np.einsum("bhd,nbhd->bhn", q.double().cpu().numpy(), np.stack(ks)) / math.sqrt(D)
        w = np.exp(a - a.max(-1, keepdims=True))
        want = np.einsum("bhn,nbhd->bhd", w / w.sum(-1, keepdims=True), np.stack(vs))
        assert max_abs(o.cpu().numpy(), want) <= 1e-5
        rows = logits.cpu().numpy().astype(np.float64)
        for b in range(B):
            may, _, near = sample64(rows[b], uu[b], float(np.float32(0.8)), 0, float(np.float32(0.9)), 0.0)
            assert near or token.tolist()[b] in may


@pytest.mark.parametrize("kv", ["f32", "int8"])
def test_model_sampling(kv):
    """BatchModel.sample after a prompt and after steps: tokens as the operation
    draws them from the model's logits; they are its choices and its recorded ids;
    sequences that sat out keep theirs; greedy steps go on from them."""
    import torch
    cfg = synth.TINY
    w = synth.make_weights(cfg, 0)
    prompts = synth.make_batch_prompts(cfg, 5, 3, 9, seed=3)
    V, B = cfg.vocab_size, 5
    rng = np.random.default_rng(4)
    m = binding.BatchModel(cfg, binding.upload_weights(w), 6, kv=kv)
    try:
        with pytest.raises(binding.GPT2Error) as e:
            m.sample(1)
        assert e.value.name == "NOT_READY"
        m.prefill(prompts)
        greedy = m.argmax(B)
        assert m.sample(B) == greedy                         # no temperature: greedy
        t = torch.tensor([0.7, 1.0, 0.0, 1.3, 0.9], device="cuda")
        k = torch.tensor([0, 5, 0, 40, 0], dtype=torch.int32, device="cuda")
        p = torch.tensor([0.9, 1.0, 1.0, 0.95, 1.0], device="cuda")
        q = torch.tensor([0.0, 0.0, 0.0, 0.0, 0.05], device="cuda")
        pos = [len(x) for x in prompts]
        for step in range(4):
            u = uniform(rng, B, V).astype(np.float32)
            logits = m.logits(B)
            ids = m.sample(B, t, torch.from_numpy(u).cuda(), k, p, q)
            want, _ = binding.op_sample(torch.from_numpy(logits).cuda(), t, torch.from_numpy(u).cuda(), k, p, q)
            assert ids == want.tolist() == m.argmax(B)
            for b in range(B):
                assert m.ids(pos[b] - 1, 1)[0, b] == ids[b]
            if step == 2:                                    # sequence 1 sits a step out
                m.decode([ids[0], 0] + ids[2:], [pos[0], -1] + pos[2:])
                pos = [x + (b != 1) for b, x in enumerate(pos)]
                u = torch.from_numpy(uniform(rng, B, V).astype(np.float32)).cuda()
                now = m.sample(B, t, u, k, p, q)
                assert now[1] == -1 and m.argmax(B)[1] == ids[1]
                ids = [ids[1] if b == 1 else x for b, x in enumerate(now)]
            m.decode(ids, pos)
            pos = [x + 1 for x in pos]
        ids = m.sample(B, t, torch.from_numpy(uniform(rng, B, V).astype(np.float32)).cuda(), k, p, q)
        m.decode_greedy(1)
        got = m.logits(B)
        m.decode(ids, pos)                                   # the same step again, fed by hand
        assert np.array_equal(got, m.logits(B))
        # a tree step's logits are its nodes': nothing to draw from
        m.decode_tree([([ids[0], 1], [-1, 0])] + [None] * 4)
        with pytest.raises(binding.GPT2Error) as e:
            m.sample(B)
        assert e.value.name == "NOT_READY"
        with pytest.raises(ValueError):
            m.sample(B, t[:2], torch.zeros((B, V), device="cuda"))
        with pytest.raises(binding.GPT2Error):
            m.sample(7)
        with pytest.raises(binding.GPT2Error):
            m.sample(0)
    finally:
        m.close()
