"""Sampling on the batched model where there is nothing to draw from."""
import ctypes

import numpy as np
import pytest

from transformer_decode_token_gb300 import binding, synth

pytestmark = pytest.mark.gpu


def call(m, n, temperature=None):
    """gpt2_sample_batch itself, on ids that hold something."""
    out = (ctypes.c_int32 * 8)(*[7] * 8)
    status = binding.lib().gpt2_sample_batch(m._h, n, temperature, None, None, None, None, out)
    return binding.STATUS[status], list(out)


def test_ids_of_a_call_that_draws_nothing():
    """Its ids are -1, as those of a sequence that has none, and the choices stay."""
    import torch
    cfg = synth.TINY
    m = binding.BatchModel(cfg, binding.upload_weights(synth.make_weights(cfg, 0)), 4)
    try:
        assert call(m, 3) == ("NOT_READY", [-1] * 3 + [7] * 5)
        m.prefill([[1, 2, 3], [4, 5]])
        first = m.argmax(2)
        t = torch.ones(4, device="cuda")
        # a temperature without random numbers
        assert call(m, 2, t.data_ptr()) == ("INVALID_ARG", [-1] * 2 + [7] * 6)
        assert call(m, 5)[0] == "INVALID_ARG"
        assert m.argmax(2) == first
        assert call(m, 4) == ("OK", first + [-1, -1] + [7] * 4)
        m.decode_greedy(1)
        m.sync()
    finally:
        m.close()


def test_logits_without_a_choice():
    """A sequence whose logits are NaN gets -1 and has no choice; the others go on."""
    import torch
    cfg = synth.TINY
    w = dict(synth.make_weights(cfg, 0))
    w["wpe"] = np.array(w["wpe"])
    w["wpe"][4] = np.nan
    m = binding.BatchModel(cfg, binding.upload_weights(w), 4)
    try:
        m.prefill([[1, 2, 3], [4, 5, 6, 7, 8]])       # the second's last position is 4
        t, u = torch.ones(2, device="cuda"), torch.full((2, cfg.vocab_size), 0.5, device="cuda")
        with pytest.raises(binding.GPT2Error) as e:
            m.sample(2, t, u)
        assert e.value.name == "DEVICE_STATE"
        one, none = e.value.tokens
        assert 0 <= one < cfg.vocab_size and none == -1 and m.argmax(2) == [one, -1]
        with pytest.raises(binding.GPT2Error) as e:
            m.decode_greedy(1)
        assert e.value.name == "NOT_READY"
        m.decode([one], [3])
        assert np.isfinite(m.logits(1)).all()
    finally:
        m.close()
