"""Refusals of the paged-cache and sampling operations that need no GPU: the C
entry points validate their arguments before any device work."""
import ctypes

import pytest

from transformer_decode_token_gb300 import binding

from test_spec_host import BAD_KV, P, kv

MAP_ARRAYS = ("cached", "grow", "table", "ring", "state", "cached_out", "state_out", "first", "seq", "slot", "offset",
              "position")
SAMPLE_ARRAYS = ("temperature", "top_k", "top_p", "min_p", "u", "token", "prob", "dist")


def page_map(cached=P, grow=P, seqs=2, block=16, table=P, width=8, ring=P, blocks=32, state=P, cached_out=P,
             state_out=P, first=P, seq=P, slot=P, offset=P, position=P, rows=4):
    return binding.lib().gpt2_op_page_map(cached, grow, seqs, block, table, width, ring, blocks, state, cached_out,
                                          state_out, first, seq, slot, offset, position, rows, None)


def attend(c, q=P, dtype=0, q_stride=192, heads=3, table=P, seqs=2, width=4, seq=None, position=P, rows=2, scale=0.125,
           out=P, out_stride=192, ws=P, size=1 << 30):
    return binding.lib().gpt2_op_paged_attention(ctypes.byref(c) if c else None, q, dtype, q_stride, heads, table, seqs,
                                                 width, seq, position, rows, scale, out, out_stride, ws, size, None)


def sample(logits=P, dtype=0, stride=100, rows=2, vocab=100, temperature=P, top_k=P, top_p=P, min_p=P, u=P, token=P,
           prob=P, dist=None):
    return binding.lib().gpt2_op_sample(logits, dtype, stride, rows, vocab, temperature, top_k, top_p, min_p, u, token,
                                        prob, dist, None)


def test_bad_page_maps_are_refused():
    for name in MAP_ARRAYS:
        assert page_map(**{name: None}) == -1, name
        for off in (1, 2, 3):
            assert page_map(**{name: P + off}) == -1, (name, off)
    for bad in (dict(seqs=-1), dict(seqs=8193), dict(rows=-1), dict(block=0), dict(block=-16), dict(width=0),
                dict(blocks=0), dict(block=1 << 15, width=1 << 15)):
        assert page_map(**bad) == -1, bad


def test_bad_paged_attentions_are_refused():
    for change in BAD_KV:
        assert attend(kv(**change)) == -1, change
    assert attend(None) == -1
    for bad in (dict(q=None), dict(table=None), dict(position=None), dict(out=None), dict(dtype=binding.GPT2_INT8),
                dict(dtype=9), dict(q_stride=184), dict(q_stride=196), dict(out_stride=100), dict(out_stride=194),
                dict(heads=4), dict(heads=0), dict(heads=-3), dict(seqs=-1), dict(rows=-1), dict(rows=3), dict(width=0),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(q=P + 8), dict(out=P + 4),
                dict(width=1 << 28), dict(seq=P + 2)):
        assert attend(kv(), **bad) == -1, bad
    for name in ("table", "position"):
        for off in (1, 2, 3):
            assert attend(kv(), **{name: P + off}) == -1, (name, off)
    # 16-bit rows only over a cache of their type (or an 8-bit one)
    for row, cache in ((1, 0), (3, 0), (1, 3), (3, 1)):
        assert attend(kv(dtype=cache), dtype=row) == -1
    # cache rows are counted in 32 bits, the tiles of all rows too
    assert attend(kv(n_slots=1 << 30, n_head=1, n_positions=16), heads=1) == -1
    assert attend(kv(n_head=1, n_positions=16), heads=1, rows=1 << 20, seqs=1 << 20, width=1 << 20) == -1
    assert attend(kv(n_head=1, n_positions=16), heads=1, rows=1 << 30, seqs=1 << 30, width=1) == -1


def test_bad_samplings_are_refused():
    for bad in (dict(logits=None), dict(token=None), dict(u=None), dict(dtype=binding.GPT2_INT8), dict(dtype=2),
                dict(rows=-1), dict(vocab=0), dict(stride=99), dict(vocab=524289, stride=524289), dict(logits=P + 2),
                dict(dtype=1, logits=P + 1), dict(rows=1 << 28)):
        assert sample(**bad) == -1, bad
    for name in SAMPLE_ARRAYS:
        for off in (1, 2, 3):
            assert sample(**{name: P + off}) == -1, (name, off)


def test_nothing_to_do_is_not_an_error():
    assert attend(kv(), rows=0) == 0
    assert sample(rows=0) == 0
    assert sample(rows=0, temperature=None, u=None) == 0


def test_workspace_of_a_refused_shape_is_none():
    L = binding.lib()
    assert L.gpt2_op_paged_attention_workspace(ctypes.byref(kv(head_dim=48)), 0, 3) == 0
    assert L.gpt2_op_paged_attention_workspace(None, 0, 3) == 0


def test_constants_are_the_header_s():
    import os
    import re
    header = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gpt2.h")).read()
    assert int(re.search(r"GPT2_MAX_PAGED_SEQS (\d+)", header).group(1)) == binding.MAX_PAGED_SEQS
    assert int(re.search(r"GPT2_SAMPLE_MAX_VOCAB (\d+)", header).group(1)) == binding.SAMPLE_MAX_VOCAB


def test_sampling_of_a_model_is_refused_on_the_host():
    L = binding.lib()
    one = (ctypes.c_int32 * 1)(1)
    assert L.gpt2_sample_batch(None, 1, None, None, None, None, None, one) == -1
