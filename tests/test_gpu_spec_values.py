"""Infinities, NaN and extreme values in what the speculative-decoding
operations read, against plain implementations in 64 bits."""
import math

import numpy as np
import pytest

from transformer_decode_token_gb300 import binding

from test_gpu_spec import COMBOS, attend64, check_attention, dt, i32, make_cache, random_tree

pytestmark = pytest.mark.gpu

# (query rows over one sequence: on the CUDA cores, on the matrix instructions, on the tensor cores)
SHAPES = [("few", 1, 60, 150, 2), ("few", 2, 61, 150, 2), ("mma", 9, 60, 150, 2), ("mma", 23, 61, 150, 2),
          ("mma", 9, 1000, 1100, 2)]
TC_SHAPES = [("tc", 24, 60, 1600, 200), ("tc", 24, 1500, 40000, 8), ("tc", 40, 1021, 70000, 4)]


def attention_cases():
    for qt, ct in COMBOS:
        for shape in SHAPES:
            yield (qt, ct, 64, *shape)
    for t in ("bf16", "f16"):
        for D in (64, 128):
            for shape in TC_SHAPES:
                yield (t, t, D, *shape)


def poison_setup(qt, ct, D, n, c, P, K):
    import torch
    rng = np.random.default_rng(n + c + D)
    kc, ks = make_cache(rng, ct, 1, K, P, D)
    vc, vs = make_cache(rng, ct, 1, K, P, D)
    mask = binding.tree_masks(random_tree(rng, n, 6))
    q = torch.from_numpy(rng.standard_normal((n, K, D)).astype(np.float32)).to(dt(qt)).cuda()
    args = (i32([0]), i32([c]), i32([0, n]), torch.from_numpy(mask).cuda(), n)
    return q, kc, vc, ks, vs, mask, args


@pytest.mark.parametrize("qt,ct,D,kernel,n,c,P,K", list(attention_cases()))
def test_bad_values_of_the_prefix_reach_every_node(qt, ct, D, kernel, n, c, P, K):
    """A NaN or an infinity in a value of the cached prefix, at any distance
    before the nodes, makes that dimension of every node's result not finite."""
    import torch
    q, kc, vc, ks, vs, mask, args = poison_setup(qt, ct, D, n, c, P, K)
    h = K - 1
    for row in (0, c // 2, c - 31, c - 17, c - 5, c - 2, c - 1):
        if ct == "int8":
            spots = [(vs, (0, h, row), math.nan)]
        else:
            spots = [(vc, (0, h, row, 17), x) for x in ([math.nan] if ct == "e4m3" else [math.nan, math.inf, -math.inf])]
        for t, at, x in spots:
            old = t[at].clone()
            t[at] = torch.tensor(x).to(t.dtype)
            got = binding.op_tree_attention(q, kc, vc, *args, ks, vs).float()
            t[at] = old
            hit = got[:, h] if t is vs else got[:, h, 17]
            assert not torch.isfinite(hit).any(), (row, x)
            if t is vc:
                rest = [d for d in range(D) if d != 17]
                assert torch.isfinite(got[:, h][:, rest]).all() and torch.isfinite(got[:, :h]).all()


@pytest.mark.parametrize("qt,ct", [c for c in COMBOS if c[1] in ("int8", "e4m3")])
@pytest.mark.parametrize("n", [1, 9, 23])
def test_scales_of_either_sign(qt, ct, n):
    """A value is code * scale whatever the scale's sign: negative scales give
    what the negated codes with positive ones give."""
    import torch
    c = 170
    q, kc, vc, ks, vs, mask, args = poison_setup(qt, ct, 64, n, c, 200, 2)
    sign = torch.where(torch.arange(200, device="cuda") % 3 == 0, -1.0, 1.0)
    for flip in (torch.full_like(sign, -1.0), sign):
        turn = lambda t: (t.float() * flip[:, None]).to(t.dtype)
        want, tol = attend64(q, turn(kc), turn(vc), ks, vs, [0], [c], [0, n], mask, 1 / 8)
        check_attention(binding.op_tree_attention(q, kc, vc, *args, ks * flip, vs * flip), want, tol)
