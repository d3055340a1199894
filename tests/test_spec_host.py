"""Refusals of the speculative-decoding operations that need no GPU: the C
entry points validate their arguments before any device work."""
import ctypes

import numpy as np
import pytest

from transformer_decode_token_gb300 import binding

P = 4096                                   # a 16-byte aligned address that is never read


def kv(**change):
    f = dict(k=P, v=P, k_scale=None, v_scale=None, dtype=binding.GPT2_F32, n_slots=2, n_head=3, n_positions=10,
             head_dim=64)
    f.update(change)
    return binding.KV(*f.values())


BAD_KV = [dict(k=None), dict(v=None), dict(k=P + 8), dict(v=P + 4), dict(dtype=binding.GPT2_INT4), dict(dtype=6),
          dict(dtype=-1), dict(dtype=binding.GPT2_INT8), dict(dtype=binding.GPT2_E4M3, k_scale=P), dict(n_slots=0),
          dict(n_head=0), dict(n_positions=0), dict(head_dim=48), dict(head_dim=256),
          dict(n_head=1 << 16, n_positions=1 << 15)]


def store(c, k=P, v=P, dtype=0, stride=192, slot=P, pos=P, n=1):
    return binding.lib().gpt2_op_kv_store(ctypes.byref(c) if c else None, k, v, dtype, stride, slot, pos, n, None)


def load(c, slot=P, pos=P, n=1, k=P, v=P, dtype=0, stride=192):
    return binding.lib().gpt2_op_kv_load(ctypes.byref(c) if c else None, slot, pos, n, k, v, dtype, stride, None)


def commit(c, layers=1, slot=P, cached=P, path=P, n_path=P, seqs=1, nodes=4):
    return binding.lib().gpt2_op_kv_commit(ctypes.byref(c) if c else None, layers, slot, cached, path, n_path, seqs,
                                           nodes, None)


def attend(c, q=P, dtype=0, q_stride=192, heads=3, slot=P, cached=P, first=P, mask=P, seqs=1, rows=1, nodes=1,
           scale=0.125, out=P, out_stride=192, ws=None, size=0):
    return binding.lib().gpt2_op_tree_attention(ctypes.byref(c) if c else None, q, dtype, q_stride, heads, slot,
                                                cached, first, mask, seqs, rows, nodes, scale, out, out_stride, ws, size,
                                                None)


def verify(logits=P, vocab=100, tokens=P, parents=P, first=P, seqs=1, rows=4, nodes=4, temperature=1.0, draft=None,
           ua=P, ud=P, path=P, n_path=P, token=P, ws=P, size=1 << 20):
    return binding.lib().gpt2_op_verify_tree(logits, vocab, tokens, parents, first, seqs, rows, nodes, temperature,
                                             draft, ua, ud, path, n_path, token, ws, size, None)


@pytest.mark.parametrize("call", [store, load, commit, attend])
def test_bad_caches_are_refused(call):
    for change in BAD_KV:
        assert call(kv(**change)) == -1, change
    assert call(None) == -1


@pytest.mark.parametrize("call", [store, load])
def test_bad_rows_are_refused(call):
    for bad in (dict(k=None), dict(v=None), dict(slot=None), dict(pos=None), dict(n=-1), dict(stride=191),
                dict(stride=-192), dict(dtype=binding.GPT2_INT8), dict(dtype=binding.GPT2_INT4), dict(dtype=7),
                dict(k=P + 2), dict(v=P + 1), dict(n=(1 << 31) - 1, stride=1 << 40)):
        c = kv(n_head=1 << 14) if bad.get("n", 0) > 1 else kv()
        assert call(c, **bad) == -1, bad


def test_bad_commits_are_refused():
    for bad in (dict(layers=0), dict(slot=None), dict(cached=None), dict(path=None), dict(n_path=None),
                dict(seqs=-1), dict(nodes=0), dict(nodes=65)):
        assert commit(kv(), **bad) == -1, bad


def test_bad_attentions_are_refused():
    for bad in (dict(q=None), dict(slot=None), dict(cached=None), dict(first=None), dict(mask=None), dict(out=None),
                dict(dtype=binding.GPT2_INT8), dict(dtype=9), dict(q_stride=184), dict(q_stride=196),
                dict(out_stride=100), dict(out_stride=194), dict(heads=4), dict(heads=0), dict(heads=-3),
                dict(seqs=-1), dict(rows=-1), dict(nodes=0), dict(nodes=65), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(q=P + 8), dict(out=P + 4), dict(mask=P + 4)):
        assert attend(kv(), **bad) == -1, bad
    # 16-bit rows only over a cache of their type (or an 8-bit one)
    for row, cache in ((1, 0), (3, 0), (1, 3), (3, 1)):
        assert attend(kv(dtype=cache), dtype=row) == -1


def test_bad_verifications_are_refused():
    for bad in (dict(logits=None), dict(tokens=None), dict(parents=None), dict(first=None), dict(path=None),
                dict(n_path=None), dict(token=None), dict(ws=None), dict(vocab=0), dict(seqs=-1), dict(rows=-1),
                dict(nodes=0), dict(nodes=65), dict(temperature=-1.0), dict(temperature=float("nan")),
                dict(temperature=float("inf")), dict(temperature=1e-39), dict(ua=None), dict(ud=None),
                dict(ws=P + 8), dict(size=8), dict(logits=P + 2)):
        assert verify(**bad) == -1, bad
    L = binding.lib()
    assert L.gpt2_op_verify_tree_workspace(4, 50257) == 4 * 7 * 16
    assert L.gpt2_op_verify_tree_workspace(0, 50257) == 16


def test_nothing_to_do_is_not_an_error():
    assert store(kv(), n=0) == 0
    assert load(kv(), n=0) == 0
    assert commit(kv(), seqs=0) == 0
    assert attend(kv(), seqs=0) == 0
    assert attend(kv(), rows=0) == 0
    assert verify(seqs=0) == 0


def test_tree_masks():
    m = binding.tree_masks([-1, 0, 0, 1, 3, 2])
    assert m.dtype == np.int64
    assert [int(x) for x in m] == [1, 0b11, 0b101, 0b1011, 0b11011, 0b100101]
    assert int(binding.tree_masks(list(range(-1, 63)))[63]) == -1        # a chain of 64: every bit
    for bad in ([-1, 1], [-1, 0, 2], [-1, -1], [], list(range(-1, 64))):
        with pytest.raises(ValueError):
            binding.tree_masks(bad)
