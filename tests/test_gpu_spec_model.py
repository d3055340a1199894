"""Speculative decoding on the batched model: tree steps and their acceptance
against the CPU oracle, through the C ABI.

As in test_gpu_batch.py the oracle runs each sequence on its own with the
weights as the model stores them, and logits agree within 2e-3 abs.
"""
import ctypes

import numpy as np
import pytest

from oracle import oracle as orc
from transformer_decode_token_gb300 import binding, synth

from gpu_util import max_abs, top2_margin

ATOL = 2e-3


def oracle_ids(cfg, w, prompt, steps, kv):
    sw = orc.stored_weights(w, "bf16", head="bf16")
    return orc.greedy(cfg, sw, prompt, steps, omp=True, kv=kv)


def test_tree_calls_are_refused_on_the_host():
    L = binding.lib()
    one = (ctypes.c_int32 * 1)(1)
    assert L.gpt2_decode_tree_batch(None, one, one, one, 1, None) == -1
    assert L.gpt2_accept_tree_batch(None, 0.0, None, None, None, one, one) == -1


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["f32", "bf16"])
@pytest.mark.parametrize("deep", [False, True])
def test_greedy_trees_give_the_greedy_tokens(kv, deep):
    """Ragged sequences, each step a tree that holds the oracle's own
    continuation for a few tokens, wrong siblings before and after it, and a
    wrong child at its end: exactly the right branch is accepted, its logits
    are the oracle's, and the tokens are those of plain greedy decoding.  deep:
    one sequence with trees of up to 30 nodes."""
    cfg = synth.TINY
    w = synth.make_weights(cfg, 0)
    prompts = synth.make_batch_prompts(cfg, 1 if deep else 5, 4, 20, seed=4)
    B, V = len(prompts), cfg.vocab_size
    ref = [oracle_ids(cfg, w, p, 40, kv) for p in prompts]
    rng = np.random.default_rng(1)
    m = binding.BatchModel(cfg, binding.upload_weights(w), 40, kv=kv)
    try:
        m.prefill(prompts)
        gained = [[t] for t in m.argmax(B)]              # ids after the prompt, the first by the prefill
        for step in range(5):
            trees, right = [], []
            for b in range(B):
                ids = ref[b][0]
                at = len(gained[b]) - 1                  # the last gained id is consumed next
                if step == 2 and b == 1:
                    trees.append(None)
                    right.append([])
                    continue
                take = int(rng.integers(0, 6 if deep else 3))
                tok, par, path = [gained[b][-1]], [-1], [0]
                for k in range(take):
                    for wrong in range(int(rng.integers(0, 3))):   # siblings tried before the right one
                        tok.append((ids[at + 1 + k] + 1 + wrong) % V)
                        par.append(path[-1])
                    tok.append(ids[at + 1 + k])
                    par.append(path[-1])
                    path.append(len(tok) - 1)
                tok.append((ids[at + 1 + take] + 7) % V)
                par.append(path[-1])
                while deep and len(tok) < 30 and step % 2:
                    tok.append(int(rng.integers(0, V)))
                    par.append(0)
                trees.append((tok, par))
                right.append(path)
            addr = m.decode_tree(trees)
            rows = sum(len(t[0]) for t in trees if t)
            assert addr
            lg = m.logits(rows)
            r0 = 0
            for b in range(B):
                if trees[b] is None:
                    continue
                for depth, node in enumerate(right[b]):
                    row = ref[b][1][len(prompts[b]) + len(gained[b]) - 1 + depth]
                    d = max_abs(lg[r0 + node], row)
                    assert d <= ATOL, f"sequence {b} node {node}: {d:.3g}"
                r0 += len(trees[b][0])
            new = m.accept_tree()
            for b in range(B):
                if trees[b] is None:
                    assert new[b] == []
                    continue
                at = len(gained[b]) - 1
                want = ref[b][0][at + 1:at + 1 + len(right[b])]
                rows_ = ref[b][1][len(prompts[b]) + at:len(prompts[b]) + at + len(right[b])]
                assert min(top2_margin(x) for x in rows_) > 1e-3, "the seed gives near ties"
                assert new[b] == want, f"sequence {b} step {step}"
                gained[b] += new[b]
        # the cache holds what plain decoding leaves: the next plain steps agree
        lens = [len(p) + len(g) - 1 for p, g in zip(prompts, gained)]
        m.decode([g[-1] for g in gained], lens)
        lg = m.logits(B)
        for b in range(B):
            assert max_abs(lg[b], ref[b][1][lens[b]]) <= ATOL
        m.decode_greedy(2)
        m.sync()
    finally:
        m.close()


@pytest.mark.gpu
def test_next_tokens_feed_the_greedy_steps():
    """After an acceptance gpt2_decode_batch_greedy goes on from the next token."""
    cfg = synth.TINY
    w = synth.make_weights(cfg, 0)
    prompts = synth.make_batch_prompts(cfg, 3, 5, 9, seed=6)
    ref = [oracle_ids(cfg, w, p, 12, "f32")[0] for p in prompts]
    m = binding.BatchModel(cfg, binding.upload_weights(w), 16)
    try:
        m.prefill(prompts)
        m.decode_tree([([r[0], r[1], r[2]], [-1, 0, 1]) for r in ref])
        assert m.accept_tree() == [r[1:4] for r in ref]
        m.decode_greedy(3)
        assert m.argmax(3) == [r[6] for r in ref]
        with pytest.raises(binding.GPT2Error) as e:      # the nodes are gone
            m.accept_tree()
        assert e.value.name == "NOT_READY"
    finally:
        m.close()


@pytest.mark.gpu
def test_sampled_acceptance_is_the_operation():
    """temperature > 0: path, tokens and cache are those of gpt2_op_verify_tree
    on the step's logits; a chain whose u_accept are 0 is accepted whole, with
    u_accept just below 1 and improbable drafts none of it."""
    import torch
    cfg = synth.TINY
    w = synth.make_weights(cfg, 0)
    prompts = synth.make_batch_prompts(cfg, 2, 5, 9, seed=6)
    m = binding.BatchModel(cfg, binding.upload_weights(w), 16)
    rng = np.random.default_rng(2)
    try:
        m.prefill(prompts)
        first = m.argmax(2)
        trees = [([first[0], 5, 9], [-1, 0, 1]), ([first[1], 7, 8, 7], [-1, 0, 0, 2])]
        m.decode_tree(trees)
        lg = torch.from_numpy(m.logits(7)).cuda()
        ud = torch.from_numpy(((rng.integers(0, 1 << 23, (2, cfg.vocab_size)) + 0.5) * 2.0 ** -23).astype(np.float32)).cuda()
        for ua, lens in ((1e-9, [3, 2]), (1 - 2.0 ** -24, [1, 1])):
            u = torch.full((7,), ua, device="cuda")
            i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
            path, n_path, nxt = binding.op_verify_tree(lg, i32([first[0], 5, 9, first[1], 7, 8, 7]),
                                                       i32([-1, 0, 1, -1, 0, 0, 2]), i32([0, 3, 7]), 64, 0.9, None, u, ud)
            assert n_path.tolist() == lens
            if ua > 0.5:
                got = m.accept_tree(0.9, None, u, ud)
                assert got == [[nxt[0].item()], [nxt[1].item()]]
    finally:
        m.close()


@pytest.mark.gpu
def test_tree_steps_refuse():
    cfg = synth.TINY                                     # 64 positions
    w = synth.make_weights(cfg, 0)
    m = binding.BatchModel(cfg, binding.upload_weights(w), 8)
    try:
        def status(*trees):
            with pytest.raises(binding.GPT2Error) as e:
                m.decode_tree(list(trees))
            return e.value.name
        m.prefill([[1, 2, 3], list(range(60))])
        assert status(None, None) == "INVALID_ARG"
        assert status(([1] * 9, list(range(-1, 8)))) == "INVALID_ARG"            # more than max_batch rows
        assert status(([1, 2], [-1, 1])) == "INVALID_ARG"
        assert status(([1, 2], [-1, -1])) == "INVALID_ARG"
        assert status(([cfg.vocab_size], [-1])) == "TOKEN_RANGE"
        assert status(([-1], [-1])) == "TOKEN_RANGE"
        assert status(None, ([1] * 5, list(range(-1, 4)))) == "POSITION_RANGE"
        with pytest.raises(binding.GPT2Error) as e:
            m.accept_tree()
        assert e.value.name == "NOT_READY"
        m.decode_tree([None, ([1] * 4, list(range(-1, 3)))])                      # to the last position
        assert len(m.accept_tree()[1]) >= 1
        m.decode_tree([([1, 2], [-1, 0])])
        with pytest.raises(binding.GPT2Error):
            m.accept_tree(-1.0)
        with pytest.raises(binding.GPT2Error):
            m.accept_tree(1.0)
        assert len(m.accept_tree()[0]) >= 1
    finally:
        m.close()


@pytest.mark.gpu
def test_logits_without_a_choice():
    """A token whose embedding is NaN ruins its own sequence's logits only: the
    error carries what every sequence gained."""
    cfg = synth.TINY
    w = dict(synth.make_weights(cfg, 0))
    clean = binding.BatchModel(cfg, binding.upload_weights(w), 8)
    w["wpe"] = np.array(w["wpe"])
    w["wpe"][9] = np.nan
    m = binding.BatchModel(cfg, binding.upload_weights(w), 8)
    try:
        prompts = [[1, 2, 3], [4, 5, 6, 7, 8, 9, 10, 11, 12]]     # the second's next position is 9
        for x in (clean, m):
            x.prefill(prompts)
        first = clean.argmax(2)
        trees = [([first[0], 5], [-1, 0]), ([first[1], 6], [-1, 0])]
        clean.decode_tree(trees)
        want = clean.accept_tree()
        m.decode_tree(trees)
        with pytest.raises(binding.GPT2Error) as e:
            m.accept_tree()
        assert e.value.name == "DEVICE_STATE" and e.value.tokens == [want[0], []]
        m.decode_tree([([want[0][-1]], [-1])])                    # the first goes on
        clean.decode_tree([([want[0][-1]], [-1])])
        assert m.accept_tree() == clean.accept_tree()
    finally:
        m.close()
        clean.close()


# ---- the int8 cache -----------------------------------------------------------------

def quantise(x):
    """Rows [..][D] as an int8 cache holds them, by the definition in gpt2.h, and
    the steps (scales)."""
    s = np.maximum(np.abs(x).max(-1, keepdims=True).astype(np.float32) * (np.float32(1) / np.float32(127)),
                   np.float32(2.0 ** -126))
    return np.rint(x / s.astype(np.float64)) * s.astype(np.float64), s.astype(np.float64)


def forward64(cfg, w, tokens, kv=quantise):
    """Float64 GPT-2 forward (logits of every position) whose keys and values
    pass through the int8 cache's rounding, per head and row."""
    d = lambda a: np.asarray(a, np.float64)
    E, H, D, n = cfg.n_embd, cfg.n_head, cfg.head_dim, len(tokens)

    def norm(x, g, b):
        x = x - x.mean(-1, keepdims=True)
        return x / np.sqrt((x * x).mean(-1, keepdims=True) + cfg.ln_eps) * d(g) + d(b)

    x = d(w["wte"])[tokens] + d(w["wpe"])[:n]
    rows = []
    for L in w["layers"]:
        q, k, v = np.split(norm(x, L["ln1_w"], L["ln1_b"]) @ d(L["attn_w"]) + d(L["attn_b"]), 3, -1)
        q, k, v = (a.reshape(n, H, D).transpose(1, 0, 2) for a in (q, k, v))
        k, v = (kv(a)[0] for a in (k, v))
        rows.append((k, v))
        s = q @ k.transpose(0, 2, 1) / np.sqrt(D)
        s[:, np.triu(np.ones((n, n), bool), 1)] = -np.inf
        p = np.exp(s - s.max(-1, keepdims=True))
        a = (p / p.sum(-1, keepdims=True)) @ v
        x = x + a.transpose(1, 0, 2).reshape(n, E) @ d(L["proj_w"]) + d(L["proj_b"])
        h = norm(x, L["ln2_w"], L["ln2_b"]) @ d(L["fc_w"]) + d(L["fc_b"])
        h = h / (1 + np.exp(-2 * np.sqrt(2 / np.pi) * (h + 0.044715 * h ** 3)))
        x = x + h @ d(L["mlp_proj_w"]) + d(L["mlp_proj_b"])
    return norm(x, w["ln_f_w"], w["ln_f_b"]) @ d(w.get("head", w["wte"])).T, rows


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [7, 1])
def test_int8_cache_model(batch):
    """Ragged prompts (packed prompt steps; one sequence: a step per position)
    and decode steps against the float64 forward with the same rounding of the
    keys and values.  The model's own k and v are off from exact ones by about
    2^-17 (bf16 hi + lo products), so a code differs where a value lies that
    near to a rounding border, for about one in a thousand, by one step (1/127
    of its row's largest): far below the tolerance of 2e-3 in the logits.
    Layer 0's exported rows are within half a step, and that error, of the
    exact rows."""
    cfg = synth.TINY
    w = synth.make_weights(cfg, 0)
    sw = orc.stored_weights(w, "bf16", head="bf16")
    prompts = synth.make_batch_prompts(cfg, batch, 3, 30, seed=8)
    m = binding.BatchModel(cfg, binding.upload_weights(w), batch, kv="int8")
    rng = np.random.default_rng(3)
    try:
        m.prefill(prompts)
        lg = m.logits(batch)
        seqs = [list(p) for p in prompts]
        for step in range(4):
            for b in range(batch):
                want, _ = forward64(cfg, sw, np.array(seqs[b]))
                d = max_abs(lg[b], want[-1])
                assert d <= ATOL, f"sequence {b} step {step}: {d:.3g}"
            if step == 3:
                break
            nxt = [int(x) for x in rng.integers(0, cfg.vocab_size, batch)]
            m.decode(nxt, [len(q) for q in seqs])
            for q, t in zip(seqs, nxt):
                q.append(t)
            lg = m.logits(batch)
        b = batch - 1
        k, v = m.export_kv(0, b, len(seqs[b]))
        for got, exact in zip((k, v), forward64(cfg, sw, np.array(seqs[b]), kv=lambda a: (a, None))[1][0]):
            _, step_size = quantise(exact)
            assert np.all(np.abs(got - exact) <= 0.5 * step_size + 2.0 ** -15 * (1 + np.abs(exact)))
        m.decode_greedy(2)
        m.sync()
    finally:
        m.close()


@pytest.mark.gpu
def test_int8_cache_tree_steps():
    """A tree step over the int8 cache: every node's logits are those of its own
    path run through the float64 forward, and after the acceptance plain steps go
    on from the kept path."""
    cfg = synth.TINY
    w = synth.make_weights(cfg, 0)
    sw = orc.stored_weights(w, "bf16", head="bf16")
    prompts = synth.make_batch_prompts(cfg, 3, 5, 20, seed=9)
    m = binding.BatchModel(cfg, binding.upload_weights(w), 24, kv="int8")
    try:
        m.prefill(prompts)
        first = m.argmax(3)
        follow = []
        for p, t in zip(prompts, first):                 # two exact greedy tokens after the first
            ids = list(p) + [t]
            for _ in range(2):
                ids.append(int(np.argmax(forward64(cfg, sw, np.array(ids))[0][-1])))
            follow.append(ids[-2:])
        trees = [([t, 3, f[0], 9, f[1], 8], [-1, 0, 0, 1, 2, 4]) for t, f in zip(first, follow)]
        m.decode_tree(trees)
        lg = m.logits(18)
        margins = []
        for b, (tok, par) in enumerate(trees):
            for i in range(6):
                path, j = [], i
                while j >= 0:
                    path.append(tok[j])
                    j = par[j]
                want = forward64(cfg, sw, np.array(list(prompts[b]) + path[::-1]))[0][-1]
                assert max_abs(lg[6 * b + i], want) <= ATOL, (b, i)
                if i in (0, 2, 4):
                    margins.append(top2_margin(want))
        assert min(margins) > 4e-3, "the seed gives near ties"
        got = m.accept_tree()
        for b in range(3):
            assert got[b][:2] == follow[b] and len(got[b]) == (4 if got[b][2] == 8 else 3)
        m.decode([g[-1] for g in got], [len(p) + len(g) for p, g in zip(prompts, got)])
        lg = m.logits(3)
        for b in range(3):
            ids = list(prompts[b]) + [first[b]] + got[b]
            assert max_abs(lg[b], forward64(cfg, sw, np.array(ids))[0][-1]) <= ATOL
    finally:
        m.close()
