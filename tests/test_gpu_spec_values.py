"""Infinities, NaN and extreme values in what the speculative-decoding
operations read, against plain implementations in 64 bits."""
import math

import numpy as np
import pytest

from transformer_decode_token_gb300 import binding

from test_gpu_spec import (COMBOS, attend64, check_attention, dt, i32, make_cache, random_tree, run_verify, uniform,
                           verify64, verify_inputs)

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


def by_definition64(q, kc, vc, ks, vs, c, mask, scale):
    """Results of one head's nodes q [n][D] over rows kc, vc [P][D] in float64,
    infinities and NaN included, and the tolerance of what is finite: as
    test_gpu_spec.attend64's, over the keys of finite scores."""
    host = lambda t: t.float().cpu().numpy().astype(np.float64)
    q, k, v = host(q), host(kc), host(vc)
    n = len(mask)
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    coarse = kc.dtype.itemsize < 4 and "bfloat" not in str(kc.dtype)
    with np.errstate(all="ignore"):
        if ks is not None:
            k, v = k * host(ks)[:, None], v * host(vs)[:, None]
        for i in range(n):
            see = list(range(c)) + [c + j for j in range(n) if int(mask[i]) >> j & 1]
            kk, vv = k[see], v[see]
            a = kk @ q[i] * scale
            w = np.exp(a - a.max())
            w /= w.sum()
            out[i] = w @ vv
            sane = np.isfinite(kk).all(1)
            size = (np.abs(kk[sane]) @ np.abs(q[i])).max() * abs(scale)
            flat = np.where(np.isfinite(vv), np.abs(vv), 0)
            tol[i] = (2 * size * 2.0 ** -18 + 2.0 ** -16) * (w @ flat)
            if coarse:
                tol[i] += len(see) * 2.0 ** -38 * (1 if vs is None else 2) * flat.max()
    return out, tol


def check_with_bad(got, want, tol):
    """NaN for NaN, infinities of the same sign, and what is finite within tol
    and half a step of the result's type."""
    import torch
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(want))
    assert np.array_equal(np.isinf(g), np.isinf(want)) and np.array_equal(np.sign(g[np.isinf(g)]),
                                                                         np.sign(want[np.isinf(want)]))
    fine = np.isfinite(want)
    lim = tol + np.abs(want) * torch.finfo(got.dtype).eps / 2 + 2.0 ** -25
    assert np.all(np.abs(g[fine] - want[fine]) <= lim[fine])


@pytest.mark.parametrize("qt,ct,D,kernel,n,c,P,K", list(attention_cases()))
def test_seen_infinities_are_as_defined(qt, ct, D, kernel, n, c, P, K):
    """Infinite and NaN values, keys and scales in rows that all nodes see and
    in a node's row: infinity times a weight above zero is infinite, of both signs
    NaN; a key of score -infinity has weight zero and one of +infinity leaves
    NaN; whichever kernel runs."""
    import torch
    q, kc, vc, ks, vs, mask, args = poison_setup(qt, ct, D, n, c, P, K)
    h, inf, nan = K - 1, math.inf, math.nan
    spots = []                                       # {(tensor, row, dimension or None): value}
    bad = [nan] if ct == "e4m3" else [nan, inf, -inf] if ct != "int8" else []
    at = [0, c // 2, c - 1, c + n // 2]
    spots += [{(vc, row, 17): x} for row in at for x in bad]
    spots += [{(kc, row, 5): x} for row in at for x in bad]
    if len(bad) == 3:
        spots += [{(vc, 3, 9): inf, (vc, c - 2, 9): -inf}, {(vc, 3, 9): inf, (vc, c - 2, 9): inf, (vc, 4, 11): -inf},
                  {(kc, 7, 5): -inf, (kc, c - 1, 5): -inf, (vc, 9, 1): inf}]
    if ks is not None:
        spots += [{(vs, row, None): x} for row in at for x in (nan, inf)] + [{(ks, c - 1, None): nan}]
    # a NaN among the last node's queries: all of its scores, whatever the values
    spots += [{(q, n - 1, 7): nan}, {(q, n - 1, 7): nan, (vs if ct == "int8" else vc, c - 1, None): inf if ct != "e4m3" else nan}]
    for spot in spots:
        old = {}
        for (t, row, d), x in spot.items():
            where = (row, h, d) if t is q else (0, h, row) if d is None else (0, h, row, d)
            old[t, where] = t[where].clone()
            t[where] = torch.tensor(x).to(t.dtype)
        got = binding.op_tree_attention(q, kc, vc, *args, ks, vs)
        s = lambda t: None if t is None else t[0, h]
        want, tol = by_definition64(q[:, h], kc[0, h], vc[0, h], s(ks), s(vs), c, mask, 1 / math.sqrt(D))
        check_with_bad(got[:, h], want, tol)
        assert torch.isfinite(got[:, :h].float()).all()
        for (t, where), x in old.items():
            t[where] = x


@pytest.mark.parametrize("n", [1, 3, 9, 30])
def test_values_next_to_the_largest(n):
    """fp32 values within a rounding of the largest number: the products' first
    parts round to infinity, the results are finite."""
    import torch
    top = float(np.finfo(np.float32).max)
    q, kc, vc, ks, vs, mask, args = poison_setup("f32", "f32", 64, n, 100, 150, 2)
    vc[0, 1, :, 3] = top
    vc[0, 1, 50, 7] = -top
    vc[0, 0, 99, 63] = top
    got = binding.op_tree_attention(q, kc, vc, *args)
    for h in range(2):
        want, tol = by_definition64(q[:, h], kc[0, h], vc[0, h], None, None, 100, mask, 1 / 8)
        g = got[:, h].double().cpu().numpy()
        # (a mean of the largest number may round past it by what tol allows)
        assert np.all((np.abs(g - want) <= tol + np.abs(want) * 2.0 ** -22 + 1e-30) | (np.isinf(g) & (want + tol > top)))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n", [24, 40])
def test_many_small_weights_count(dtype, D, n):
    """One key of weight 1 among 131,071 of weight 2^-26 each (a unit per CTA, so
    that they are summed against its maximum): together they are 2^-9 of the
    result, and all of it in the dimensions where the first value is zero.
    Scores are exact in 16 bits but for the scale; the weights' own error is
    that of an exponent of 26 in fp32, below 2^-17.  The tensor cores' fp32 sums
    are cut off, not rounded: each of the c / 16 additions of 16 products to
    either sum loses less than a unit in the last place, 2^-23 of the sum, per
    product, so the numerator and the denominator (1 + 2^-9) are each off by
    less than c 2^-23 = 2^-6 relatively.  (Dropping the small weights is off by
    the whole result.)"""
    import torch
    P, c = 131072 + 64, 131072
    K = 304 if D == 64 else 152
    kc = torch.zeros((1, K, P, D), dtype=dt(dtype), device="cuda")
    vc = torch.ones((1, K, P, D), dtype=dt(dtype), device="cuda")
    kc[:, :, 1:, 0] = -8.0
    vc[:, :, 0] = 0.0
    q = torch.zeros((n, K, D), dtype=dt(dtype), device="cuda")
    q[:, :, 0] = 1.0
    kc[:, :, c:, 0] = -8.0
    got = binding.op_tree_attention(q, kc, vc, i32([0]), i32([c]), i32([0, n]),
                                    torch.from_numpy(binding.tree_masks([-1] + [0] * (n - 1))).cuda(), n,
                                    scale=26 * math.log(2) / 8)
    for i in (0, 1, n - 1):
        tail = (c - 1 + (1 if i == 0 else 2)) * 2.0 ** -26
        want = tail / (1 + tail)
        worst = (got[i].double() - want).abs().max().item()
        assert worst <= want * (2 * 2.0 ** -6 + 2.0 ** -16 + torch.finfo(dt(dtype)).eps / 2), (i, worst / want)
    del kc, vc
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n", [1, 9, 24])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_far_below_zero(n, D):
    """Every score is about -10^35, the same for all keys: the mean of the values,
    from whichever kernel (bf16 q and k of 10^18)."""
    import torch
    K, P, c = 200, 1600, 1500
    rng = np.random.default_rng(n)
    vc, _ = make_cache(rng, "bf16", 1, K, P, D)
    kc = torch.zeros_like(vc)
    kc[..., 0] = -1e18
    q = torch.zeros((n, K, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1e18
    got = binding.op_tree_attention(q, kc, vc, i32([0]), i32([c]), i32([0, n]),
                                    torch.from_numpy(binding.tree_masks(list(range(-1, n - 1)))).cuda(), n)
    v = vc[0].double()
    for i in (0, n - 1):
        want = v[:, :c + i + 1].mean(1)
        lim = 2.0 ** -16 * v[:, :c + i + 1].abs().mean(1) + want.abs() * 2.0 ** -8
        assert ((got[i].double() - want).abs() <= lim).all()


@pytest.mark.parametrize("temperature", [0.0, 0.8])
@pytest.mark.parametrize("dense", [True, False])
@pytest.mark.parametrize("V", [65537, 70000, 140001])
def test_verify_large_vocabularies(V, dense, temperature):
    """Vocabularies of more than 65,536 ids (more than eight chunks): ordinary
    rows, rows of which only ids behind the first 65,536 are possible, and such
    rows with one NaN among the others, which end the walk at temperature > 0."""
    rng = np.random.default_rng(V)
    logits, draft, tokens, parents, first = verify_inputs(rng, [4] * 9, V, 2)
    for b in (1, 2, 4, 5, 7, 8):
        logits[4 * b:4 * b + 4, :65536 if b < 6 else V // 2] = -np.inf
        if b in (2, 5, 8):
            logits[4 * b + (0 if b != 5 else 1), 100 if b < 8 else V // 2 - 1] = np.nan
    # (drafts among the possible ids, the highest first)
    for b in (1, 2, 4, 5, 7, 8):
        for i in range(1, 4):
            tokens[4 * b + i] = np.nanargmax(logits[4 * b + parents[4 * b + i]])
    for again in range(20):
        ua, ud = uniform(rng, 36), uniform(rng, 9, V)
        ua[::2] *= 0.01
        d = draft if dense else None
        want, near = verify64(logits, tokens, parents, first, 4, temperature, d, ua, ud)
        if near > 1e-5:
            break
    else:
        raise AssertionError("no draw of the random numbers is clear of the borders")
    if temperature > 0:
        assert want[2] == ([0], -1) and want[8] == ([0], -1)
    assert run_verify(logits, tokens, parents, first, 4, temperature, d, ua, ud) == want
