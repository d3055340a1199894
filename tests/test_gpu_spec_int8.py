"""An int8 model's prompts through full steps of 64 rows."""
import numpy as np
import pytest

from oracle import oracle as orc
from transformer_decode_token_gb300 import binding, synth

from gpu_util import max_abs
from test_gpu_spec_model import ATOL, forward64

pytestmark = pytest.mark.gpu


def test_prompts_of_whole_steps():
    """Prompts up to the cache's end, packed 64 rows to a step: a chain of 63
    rows, one that a step cuts in two, single tokens; each sequence's logits as in
    test_gpu_spec_model.test_int8_cache_model."""
    cfg = synth.TINY                                     # 64 positions
    w = synth.make_weights(cfg, 0)
    sw = orc.stored_weights(w, "bf16", head="bf16")
    rng = np.random.default_rng(12)
    lens = [64, 1, 50, 64, 2, 33]
    prompts = [[int(x) for x in rng.integers(0, cfg.vocab_size, n)] for n in lens]
    m = binding.BatchModel(cfg, binding.upload_weights(w), 64, kv="int8")
    try:
        m.prefill(prompts)
        lg = m.logits(len(lens))
        for b, p in enumerate(prompts):
            d = max_abs(lg[b], forward64(cfg, sw, np.array(p))[0][-1])
            assert d <= ATOL, f"sequence {b}: {d:.3g}"
        # and a tree step that fills the second sequence's cache to the last row
        t = [int(x) for x in rng.integers(0, cfg.vocab_size, 63)]
        m.decode_tree([None, (t, list(range(-1, 62)))])
        want = forward64(cfg, sw, np.array(prompts[1] + t))[0]
        lg = m.logits(63)
        for i in (0, 1, 30, 62):
            assert max_abs(lg[i], want[1 + i]) <= ATOL, i
        assert len(m.accept_tree()[1]) >= 1
    finally:
        m.close()
