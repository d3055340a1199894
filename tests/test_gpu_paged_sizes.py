"""The paged-cache and sampling operations at sizes where there is nothing, or where
offsets pass 32 bits."""
import numpy as np
import pytest

from transformer_decode_token_gb300 import binding

from test_gpu_spec import i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(0, 4), (2, 0), (0, 0)])
@pytest.mark.parametrize("given", [False, True])
def test_a_table_of_nothing(shape, given):
    """No sequences, or none with a block: every row sees nothing."""
    import torch
    c = torch.ones((3, 2, 8, 64), device="cuda")
    q = torch.ones((5, 2, 64), device="cuda")
    wide = torch.full((5, 200), 7.0, device="cuda")
    out = wide[:, :128].unflatten(1, (2, 64)) if given else None
    got = binding.op_paged_attention(q, c, c, i32(np.zeros(shape)), i32([3, 0, -1, 7, 100]), i32([0, 1, -1, 5, 0]), out=out)
    assert got.shape == (5, 2, 64) and (got == 0).all()
    assert (wide[:, 128:] == 7).all()


def test_rows_of_logits_past_32_bits():
    """Logits, random numbers and a distribution of more than 2^31 values: the last rows are
    what they are on their own."""
    import torch
    n, V, dev = 17000, 131072, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    x = torch.empty((n, V), dtype=torch.bfloat16, device=dev).normal_(0, 3, generator=g)
    u = torch.empty((n, V), device=dev).uniform_(1e-6, 1 - 1e-6, generator=g)
    dist = torch.empty((n, V), device=dev)
    i = torch.arange(n, device=dev)
    t = torch.where(i % 4 == 0, 0.0, 0.8)
    k, p = torch.where(i % 4 == 2, 50, 0).to(torch.int32), torch.where(i % 4 == 3, 0.9, 1.0)
    token, prob = binding.op_sample(x, t, u, k, p, dist=dist)
    for rows in (slice(0, 8), slice(16380, 16400), slice(n - 9, n)):
        few = torch.empty((len(i[rows]), V), device=dev)
        one, its = binding.op_sample(x[rows], t[rows], u[rows], k[rows], p[rows], dist=few)
        # (few rows are split over more CTAs: the tokens and what is kept are the same, the
        # probabilities' sums may round another way: the last places of fp32)
        assert torch.equal(one, token[rows])
        assert torch.equal(few > 0, dist[rows] > 0)
        assert torch.allclose(its, prob[rows], rtol=4e-6, atol=0) and torch.allclose(few, dist[rows], rtol=4e-6, atol=1e-37)
    assert ((token >= 0) & (token < V)).all()
