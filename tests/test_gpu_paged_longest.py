"""Attention over the longest line of a block table: counts of its rows, rounded up to
whole tiles, pass 2^31."""
import numpy as np
import pytest

from transformer_decode_token_gb300 import binding

from test_gpu_spec import dt, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("qt,ct,G", [("f32", "int8", 1), ("f32", "bf16", 2), ("bf16", "bf16", 4)])
@pytest.mark.parametrize("short", [0, 1, 33])
def test_the_longest_sequence(qt, ct, G, short):
    """2^31 - 1 blocks of a row each (less `short` of them seen), five blocks in turn.  All scores are 0,
    so a warp's sums of weights and of values, whole numbers up to 8 times 1.2 million keys, are
    exact, and the result is off by the parts' joining: at most 2,432 of them in 76 steps of some
    ten roundings, and eight additions in each, relative to the largest value."""
    import torch
    n, D = 2 ** 31 - 1, 32
    rng = np.random.default_rng(1)
    table = torch.arange(n, dtype=torch.int32, device="cuda").remainder_(5).view(1, n)
    v = rng.integers(-8, 9, (5, D))
    kc = torch.from_numpy(rng.integers(-8, 9, (5, 1, 1, D))).to(dt(ct)).cuda()
    vc = torch.from_numpy(v.reshape(5, 1, 1, D)).to(dt(ct)).cuda()
    ones = torch.ones((5, 1, 1), device="cuda") if ct == "int8" else None
    q = torch.zeros((1, G, D), dtype=dt(qt), device="cuda")
    seen = n - short
    got = binding.op_paged_attention(q, kc, vc, table, i32([seen - 1]), None, ones, ones)
    count = np.array([(seen - b + 4) // 5 for b in range(5)], np.float64)
    assert count.sum() == seen
    want = count @ v / seen
    err = np.abs(got.double().cpu().numpy() - want)
    step = torch.finfo(got.dtype).eps / 2
    assert np.all(err <= 76 * 18 * 2.0 ** -24 * 8 + np.abs(want) * step)
