"""GPU parity of the sampling operation's cuts against a plain implementation in
64 bits, on every row: where a cut lies next to its border, between the smallest
and the largest set of ids that the border leaves open."""
import math

import numpy as np
import pytest

from transformer_decode_token_gb300 import binding

from test_gpu_sample import NEAR, OFF, peaked
from test_gpu_spec import dt, i32, uniform

pytestmark = pytest.mark.gpu

# How far a probability is off relatively, where its sum is that of a whole row or of a long
# list (of at most 2^15.62 = 50257 weights, the largest of them 1):
#   7e-7     the sum's exponents, rounded as a whole: t = d * hi is off by 2^-24 t (the product) and
#            2^-25 t (hi), so a weight of 2^-t by ln 2 times that; such weights are at most the share
#            s = V 2^-t / (1 + V 2^-t) of the sum, and 1.5 * 2^-24 ln 2 t s is at most 7e-7 (t = 13)
#   2^-22    ex2
#   7 2^-24  a thread's weights, eight at a time in fp32
#   2^-22 + 2^-25 + 6 2^-24   CTAs' sums: the factor of each, its conversion and product, additions
#   2^-22 + 2^-25 + 3 2^-24   the id's own weight; conversion, product, quotient
# (a list of up to 512 ids is settled more exactly: OFF)
WHOLE = 7e-7 + 3 * 2.0 ** -22 + 2 * 2.0 ** -25 + 16 * 2.0 ** -24


class Cut:
    """A row by the definition in gpt2.h (temperature above 0, finite logits): its ids in
    order, their weights, and how many of the first ones are kept: lo to hi."""

    def __init__(self, row, t, k, p, m):
        V = len(row)
        w = np.exp((row - row.max()) / t)
        self.ids = np.argsort(-row, kind="stable")
        self.r = r = w[self.ids]
        n = min(k, V) if k > 0 else V
        lo = hi = n
        if p < 1:
            total = r[:n].sum()
            before = (np.cumsum(r[:n]) - r[:n])[1:]
            lo = min(lo, 1 + int((before < (max(p, 0) - NEAR) * total).sum()))
            hi = min(hi, 1 + int((before < (max(p, 0) + NEAR) * total).sum()))
        if m > 0:
            m = min(m, 1.0)
            lo = min(lo, max(1, int((r >= m + (NEAR if m < 1 else 0)).sum())))
            hi = min(hi, max(1, int((r >= m - NEAR).sum())))
        self.lo, self.hi = lo, hi
        self.sums = np.cumsum(r)

    def check(self, u, token, prob, dist):
        lo, hi, ids, r = self.lo, self.hi, self.ids, self.r
        most, least = r / self.sums[lo - 1], r / self.sums[hi - 1]
        at = int(np.flatnonzero(ids == token)[0]) if token >= 0 else -1
        assert 0 <= at < hi, (token, at, lo, hi)
        # it wins among the first n for some n from lo to hi
        n = max(lo, at + 1)
        with np.errstate(divide="ignore"):
            score = r[:n] / -np.log(u[ids[:n]].astype(np.float64))
        assert score[at] >= score.max() * (1 - NEAR), (token, at, int(score.argmax()))
        assert least[at] * (1 - WHOLE) <= prob <= most[at] * (1 + WHOLE) + 1e-30, (prob, least[at], most[at])
        if dist is None:
            return
        d = dist[ids].astype(np.float64)
        assert np.all(d[hi:] == 0)
        assert np.all(d[:hi] <= most[:hi] * (1 + WHOLE) + 1e-34)
        assert np.all(d[:lo] >= least[:lo] * (1 - WHOLE) - 1e-34)
        open_ = d[lo:hi]
        assert np.all((open_ == 0) | (open_ >= least[lo:hi] * (1 - WHOLE) - 1e-34))
        # the draw and the distribution are of the same ids: the probability is the one
        # that the distribution has (each off by OFF)
        assert abs(d[at] - prob) <= 2 * OFF * prob + 1e-34, (d[at], prob)


def check(logits, t, u, k=None, p=None, m=None, dtype="f32", dist=True):
    """Every row; returns the tokens, and how many rows' borders left one set."""
    import torch
    n, V = logits.shape
    f32 = lambda a, off: np.asarray(np.full(n, off) if a is None else np.broadcast_to(a, n), np.float32)
    t, p, m = f32(t, 1.0), f32(p, 1.0), f32(m, 0.0)
    k = np.zeros(n, np.int64) if k is None else np.broadcast_to(k, n)
    x = torch.from_numpy(logits.astype(np.float32)).to(dt(dtype)).cuda()
    held = x.float().cpu().numpy().astype(np.float64)
    u = u.astype(np.float32)
    whole = torch.full((n, V), 7.0, device="cuda") if dist else None
    c = lambda a: torch.from_numpy(a.copy()).cuda()
    token, prob = binding.op_sample(x, c(t), c(u), i32(k), c(p), c(m), dist=whole)
    token, prob = token.tolist(), prob.cpu().numpy().astype(np.float64)
    whole = whole.cpu().numpy() if dist else [None] * n
    one = 0
    for i in range(n):
        cut = Cut(held[i], float(t[i]), int(k[i]), float(p[i]), float(m[i]))
        try:
            cut.check(u[i], token[i], prob[i], whole[i])
        except AssertionError as e:
            raise AssertionError(f"row {i}, kept {cut.lo} to {cut.hi}: {e}") from e
        one += cut.lo == cut.hi
    return token, one


def far_rows(rng, n, V, top, step, levels):
    """Rows of a few neighbouring fp32 values next to a large one."""
    return np.float32(top) - np.float32(step) * rng.integers(0, levels, (n, V)).astype(np.float32)


@pytest.mark.parametrize("V", [1500, 5003, 50257])
@pytest.mark.parametrize("top,step,levels,t", [
    (1e6, 0.0625, 100, 1.0), (1.5e6, 0.125, 2, 0.7), (1.5e7, 1.0, 5, 1.0), (2.0 ** 24, 1.0, 5, 3.0),
    (-1e6, 0.0625, 5, 0.1), (1e9, 64.0, 5, 100.0), (1e9, 64.0, 5, 1.0)])
def test_logits_far_from_zero(top, step, levels, t, V):
    """fp32 logits whose spacing is of the size of the cuts' bounds (scores with a large
    common part): lists of more than 512 ids, bounded by a logit that is rounded by
    more than the ids differ."""
    rng = np.random.default_rng(V)
    n = 6
    x = far_rows(rng, n, V, top, step, levels)
    u = uniform(rng, n, V)
    ps = [0.3, 0.6, 0.9, 0.9759, 0.99, 0.999]
    check(x, t, u, p=ps)
    check(x, t, u, p=0.9999, m=[0.95, 0.9, 0.714, 0.5, 0.2, 0.02])
    check(x, t, u, m=[0.95, 0.9, 0.714, 0.5, 0.2, 0.02])
    check(x, t, u, k=[700, 1, 600, V // 2, 1200, V - 1])
    check(x, t, u, k=[700, 2, 600, V // 2, 1200, V - 1], p=ps)
    check(x, t, u, k=[700, 2, 600, V // 2, 1200, V - 1], p=0.97, m=[0.95, 0.9, 0.714, 0.5, 0.2, 0.02])


@pytest.mark.parametrize("t", [0.9, 1.0, 0.37])
def test_min_p_next_to_a_weight(t):
    """min-p within some roundings of the weight of thousands of ids, which are a good part
    of the whole: they are drawn from if the distribution has them."""
    rng = np.random.default_rng(3)
    n, V = 400, 8000
    x = np.full((n, V), -80.0, np.float32)
    t = np.float32(t)
    l0 = np.repeat(rng.uniform(-12, -4, n // 8) * t, 8).astype(np.float32)
    x[:, rng.permutation(V)[:4000]] = l0[:, None]
    x[:, 77] = 0
    m = (np.exp(l0.astype(np.float64) / float(t)) * (1 + (np.arange(n) % 8 - 3.5) * 2.0 ** -23)).astype(np.float32)
    for u in (uniform(rng, n, V), np.where(x > -80, 0.9, 0.5)):
        check(x, t, u, m=m)
        check(x, t, u, m=m, p=0.99999)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [900, 20011])
@pytest.mark.parametrize("t", [1e30, 1e36, 2e37, 1e38, 3.4e38, math.inf])
def test_differences_past_the_largest_number(t, V, dtype):
    """Logits next to the largest of both signs, whose differences fp32 does not hold, at
    temperatures that make ordinary weights of them."""
    rng = np.random.default_rng(V)
    n = 4
    x = 3.3e38 * rng.uniform(-1, 1, (n, V))
    x[1] = np.where(rng.random(V) < 0.5, 3.3e38, -3.3e38)
    x[2] = -3.3e38
    x[2, 11] = 3.3e38
    u = uniform(rng, n, V)
    for arg in ({}, dict(p=0.9), dict(p=0.3), dict(k=20), dict(k=700), dict(k=700, p=0.8), dict(m=0.4), dict(m=0.02, p=0.95)):
        check(x, t, u, dtype=dtype, **arg)


def flat(rng, n, V):
    return 0.02 * peaked(rng, n, V)


def tails(rng, n, V):
    x = 0.01 * rng.standard_normal((n, V))
    x[:, 77] = 12.0
    x[-1] = -np.arange(V) * 0.001
    return x


def two_values(rng, n, V):
    return rng.integers(0, 2, (n, V)) * 0.5


def wide(rng, n, V):
    return 4.0 * rng.standard_normal((n, V))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [3001, 50257])
@pytest.mark.parametrize("rows", [peaked, flat, tails, two_values, wide])
def test_every_row_between_its_borders(rows, V, dtype):
    """Rows whose cuts lie among few ids and among thousands, with neighbours next to the
    border or not.  With 8 of the settings 6 rows each, the first of them uncut or by count,
    a third at least leaves one set only."""
    rng = np.random.default_rng(V)
    n = 6
    x, u = rows(rng, n, V), uniform(rng, n, V)
    one = 0
    for arg in (dict(), dict(k=[1, 50, 700, 3000, V - 1, V]), dict(k=V // 3), dict(p=[0.0, 0.3, 0.5, 0.9, 0.999, 0.99999]),
                dict(m=[1.0, 0.9, 0.5, 0.1, 1e-3, 1e-6]), dict(p=0.9, m=0.05), dict(k=900, p=[0.2, 0.5, 0.8, 0.95, 0.99, 1.0]),
                dict(k=2000, p=0.97, m=[1.0, 0.9, 0.5, 0.1, 1e-3, 1e-6])):
        one += check(x, 0.8, u, dtype=dtype, **arg)[1]
    assert one >= 16
