"""Attention over pages of values so large that sums of them, weighed by a running
maximum that lies below the row's, pass the range of fp32: the result is the formula's,
which does not, for every kernel, for whole units and for cut ones."""
import numpy as np
import pytest

from transformer_decode_token_gb300 import binding

from test_gpu_paged import paged64, pages
from test_gpu_spec import dt, i32

pytestmark = pytest.mark.gpu

D, K = 64, 2
TYPES = [("f32", "f32"), ("f32", "bf16"), ("f32", "int8"), ("f32", "e4m3"), ("bf16", "bf16"), ("bf16", "int8"),
         ("f16", "f16")]


def rows_of(kind, rng):
    """(positions, sequences, lengths, repeats): rows of one tile; that are cut into many
    parts; or so many rows (each many times) that a warp has several whole ones."""
    if kind == "one tile":
        return [4, 0], [0, 1], [5, 1], 1
    if kind == "cut":
        return [2999, 1500], [0, 1], [3000, 1501], 1
    return rng.integers(30, 100, 40).tolist(), (np.arange(40) % 3).tolist(), [100, 100, 100], 90


def changed(cache, change):
    """change(the cache in fp32, in place), rounded to its type."""
    x = cache.float()
    change(x)
    cache.copy_(x.to(cache.dtype))


def check_large(q, kc, vc, ks, vs, table, position, seq, repeats):
    """As check_close of test_gpu_paged: and 2^-22 for the rounding of the quotient and of the
    sum of the formula's weights; a mean of the largest number may round past it by what is allowed."""
    import torch
    tile = lambda a: i32(np.tile(a, repeats))
    args = q.repeat(repeats, 1, 1), kc, vc, i32(table), tile(position), tile(seq), ks, vs
    got = binding.op_paged_attention(*args)
    want, tol = paged64(q, kc, vc, ks, vs, table, position, seq, 1 / 8)
    g = got.double().cpu().numpy().reshape(repeats, *want.shape)
    fi = torch.finfo(got.dtype)
    lim = tol + np.abs(want) * (fi.eps / 2 + 2.0 ** -22) + (2.0 ** -25 if got.dtype == torch.float16 else 1e-30)
    with np.errstate(invalid="ignore"):
        ok = (np.abs(g - want) <= lim) | (np.isinf(g) & (np.sign(g) == np.sign(want)) & (np.abs(want) + lim > float(fi.max)))
    assert ok.all(), (int((~ok).sum()), g[~ok][:4], np.broadcast_to(want, g.shape)[~ok][:4])
    assert torch.equal(binding.op_paged_attention(*args).isfinite(), got.isfinite())
    return want


@pytest.mark.parametrize("kind", ["one tile", "whole", "cut"])
@pytest.mark.parametrize("G", [1, 2, 4, 12])
@pytest.mark.parametrize("qt,ct", TYPES)
def test_values_next_to_the_largest(qt, ct, G, kind):
    """Values at, and some around, the cache type's largest (those of 8-bit caches next to
    fp32's, by their scales), in some dimensions of every row."""
    import torch
    rng = np.random.default_rng(G)
    position, seq, lens, repeats = rows_of(kind, rng)
    kc, vc, ks, vs, table = pages(rng, ct, lens, 16, K, D)
    top = float(torch.finfo(vc.dtype).max) if vs is None else 100.0

    def large(x):
        if vs is not None:
            x[:, 1].clamp_(-90, 90)
        x[:, 1, :, 3] = top
        x[:, 1, :, 4] = -top
        x[:, 1, ::2, 7] = top / 2
        x[:, 1, 1::2, 7] = -top / 4
    changed(vc, large)
    if vs is not None:
        vs[:, 1] = 3e36
    q = torch.from_numpy((1.5 * rng.standard_normal((len(position), K * G, D))).astype(np.float32)).to(dt(qt)).cuda()
    want = check_large(q, kc, vc, ks, vs, table, position, seq, repeats)
    # (of the inputs: e4m3 has 96 and 104 next to 100, and the even one, 96, times 3e36 is 2.88e38)
    assert np.abs(want).max() >= (6e4 if ct == "f16" else 2.87e38)


@pytest.mark.parametrize("kind", ["whole", "cut"])
@pytest.mark.parametrize("G", [1, 2, 4, 12])
@pytest.mark.parametrize("qt,ct", [x for x in TYPES if x[1] != "f16"])
def test_a_large_value_behind_a_low_maximum(qt, ct, G, kind):
    """All scores are 0 but that of one later key, 7.5 above in powers of two, which the
    running maximum does not follow: its value of 2e36 meets a weight of 181."""
    import torch
    rng = np.random.default_rng(G)
    position, seq, lens, repeats = rows_of(kind, rng)
    kc, vc, ks, vs, table = pages(rng, ct, lens, 16, K, D)
    up = 7.5 * np.log(2) * 8                 # (a score is times 1/8)
    at = [(int(table[b, 28 // 16]), slice(None), 28 % 16) for b in range(len(lens))]

    def keys(x):
        x[..., 0] = 0
        for i in at:
            x[i + (0,)] = up if ks is None else 52

    def values(x):
        x.clamp_(-4, 4)
        for i in at:
            x[i] = 1
            x[i + (9,)] = 2e36 if vs is None else 100
    changed(kc, keys)
    changed(vc, values)
    if ks is not None:
        ks.fill_(1.0)
        vs.fill_(1.0)
        for i in at:
            ks[i], vs[i] = up / 52, 2e34
    q = torch.zeros((len(position), K * G, D), dtype=dt(qt), device="cuda")
    q[..., 0] = 1.0
    want = check_large(q, kc, vc, ks, vs, table, position, seq, repeats)
    assert np.abs(want).max() > 1e35
