"""GPU parity of the sampling operation against a plain implementation in 64
bits: temperature, top-k, top-p, min-p, from given random numbers."""
import math

import numpy as np
import pytest

from transformer_decode_token_gb300 import binding

from test_gpu_spec import dt, i32, uniform

pytestmark = pytest.mark.gpu

# a weight is off by 2^-22 (the exponential) and 2^-25 (its argument), the sum of
# the weights by as much, the division by 2^-24
OFF = 2 * (2.0 ** -22 + 2.0 ** -25) + 2.0 ** -24
NEAR = 1e-6      # a cut or a draw within this of its border may go either way (gpt2.h)


def sample64(row, u, t, k, p, m):
    """By the definition in gpt2.h: the tokens that may come out (one, unless a
    border is near), the probability of each, the distribution, and whether a
    cut's border is near."""
    V = len(row)
    none = {-1: 0.0}, np.zeros(V), False
    if not t > 0:
        ok = np.where(np.isnan(row), -np.inf, row)
        if ok.max() == -np.inf:
            return none
        w = int(ok.argmax())
        return {w: 1.0}, np.eye(1, V, w)[0], False
    if np.isnan(row).any() or (row == np.inf).any() or (row == -np.inf).all():
        return none
    with np.errstate(all="ignore"):
        d = (row - row.max()) / t if np.isfinite(t) else np.where(np.isfinite(row), 0.0, -np.inf)
        w = np.where(row == row.max(), 1.0, np.exp(d))
    ids = np.argsort(-row, kind="stable")
    if 0 < k < V:
        ids = ids[:k]
    near = False
    r = w[ids]
    if p < 1:
        before = np.cumsum(r) - r
        border = max(p, 0) * r.sum()
        near |= bool((np.abs(before[1:] - border) < NEAR * r.sum()).any())
        n = max(1, int((before < border).sum()))
        ids, r = ids[:n], r[:n]
    if m > 0:
        m = min(m, 1.0)
        near |= bool((np.abs(r[1:] - m) < NEAR).any() and m < 1)
        n = max(1, int((r >= m).sum()))
        ids, r = ids[:n], r[:n]
    dist = np.zeros(V)
    dist[ids] = r / r.sum()
    with np.errstate(all="ignore"):
        score = np.where(dist > 0, dist / -np.log(u.astype(np.float64)), 0)
    best = score.max()
    may = np.flatnonzero(score >= best * (1 - NEAR))
    return {int(v): dist[v] for v in may}, dist, near


def check(logits, t, u, k=None, p=None, m=None, dtype="f32", pad=0, dist=False):
    import torch
    n, V = logits.shape
    x = torch.zeros((n, V + pad), dtype=dt(dtype), device="cuda")
    x[:, :V] = torch.from_numpy(logits.astype(np.float32)).to(dt(dtype)).cuda()
    held = x[:, :V].float().cpu().numpy().astype(np.float64)
    f32 = lambda a: None if a is None else torch.tensor(np.asarray(a, np.float32), device="cuda")
    ud = torch.from_numpy(u.astype(np.float32)).cuda()
    whole = torch.full((n, V), 7.0, device="cuda") if dist else None
    token, prob = binding.op_sample(x[:, :V], f32(t), ud, None if k is None else i32(k), f32(p), f32(m), dist=whole)
    again, _ = binding.op_sample(x[:, :V], f32(t), ud, None if k is None else i32(k), f32(p), f32(m))
    assert torch.equal(token, again)
    token, prob = token.tolist(), prob.cpu().numpy().astype(np.float64)
    for i in range(n):
        s = lambda a, off: off if a is None else float(np.asarray(a, np.float32)[i])
        may, want, near = sample64(held[i], u[i].astype(np.float32), s(t, 0.0), 0 if k is None else int(k[i]), s(p, 1.0),
                                   s(m, 0.0))
        if near:
            continue                     # (the cut may keep one id more or less)
        assert token[i] in may, (i, token[i], may)
        assert abs(prob[i] - may[token[i]]) <= OFF * may[token[i]] + 1e-30, (i, prob[i], may)
        if dist:
            got = whole[i].cpu().numpy().astype(np.float64)
            assert np.all(np.abs(got - want) <= OFF * want + 1e-34)
    return token


def peaked(rng, n, V):
    x = rng.standard_normal((n, V))
    return (2 * x + 6 * np.maximum(x - 2, 0)) * np.exp(0.3 * rng.standard_normal((n, 1)))


SETTINGS = [dict(), dict(k=1), dict(k=5), dict(k=50), dict(k=3000), dict(p=0.9), dict(p=0.3), dict(p=0.999), dict(m=0.1),
            dict(m=0.001), dict(k=40, p=0.9), dict(k=40, p=0.9, m=0.05), dict(k=2000, p=0.95), dict(p=0.0), dict(m=1.0),
            dict(k=700, m=0.0001)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [1, 2, 33, 1000, 5003, 50257])
@pytest.mark.parametrize("setting", SETTINGS, ids=str)
def test_settings(setting, V, dtype):
    """Each cut and their combinations, in peaked rows and flat ones."""
    rng = np.random.default_rng(V)
    n = 6
    logits = peaked(rng, n, V)
    logits[4:] *= 0.02                   # flat: a cut keeps thousands of ids
    arg = {a: np.full(n, v) for a, v in setting.items()}
    check(logits, np.full(n, 0.8), uniform(rng, n, V), dtype=dtype, pad=5 if V > 2 else 0, dist=V <= 5003, **arg)


@pytest.mark.parametrize("n,V", [(1, 50257), (64, 50257), (200, 9000), (3, 200000), (40, 131072), (2, 524288)])
def test_shapes(n, V):
    """Every split of a row, rows with settings of their own."""
    rng = np.random.default_rng(n)
    i = np.arange(n)
    check(peaked(rng, n, V), np.where(i % 5 == 0, 0.0, 0.5 + 0.1 * (i % 7)), uniform(rng, n, V),
          k=np.select([i % 3 == 0, i % 3 == 1], [0, 50], 400), p=np.where(i % 4 == 1, 1.0, 0.9),
          m=np.where(i % 2 == 0, 0.0, 0.02))


@pytest.mark.parametrize("V", [300, 5003, 50257])
def test_equal_logits(V):
    """Rows of equal logits, and of a few values: ties go to the lowest ids, so
    top-k keeps the first ids of the border's value, top-p the first so many."""
    rng = np.random.default_rng(V)
    n = 8
    logits = np.zeros((n, V))
    logits[1:] = rng.integers(0, 2, (n - 1, V)) * 0.5
    logits[3] = np.where(np.arange(V) % 7 == 0, -0.0, 0.0)
    logits[4] = rng.integers(0, 3, V) * 1e-6          # logits whose weights are the same
    ks = np.array([270, 270, V // 2, 270, 270, 1, V - 1, V // 3])
    u = uniform(rng, n, V)
    check(logits, np.ones(n), u, k=ks, dist=True)
    check(logits, np.ones(n), u, p=np.full(n, 0.3712345), dist=V <= 5003)
    check(logits, np.ones(n), u, k=ks, p=np.full(n, 0.8765432))
    assert check(logits, np.zeros(n), u)[0] == 0
    for k in (257, 300 - 1):                          # the kept ids are the first ones
        got = check(np.zeros((1, V)), np.ones(1), u[:1], k=[k])
        assert got[0] < k


def test_edges():
    """-infinity, NaN and +infinity among the logits, rows without a choice,
    extreme temperatures and logits, settings outside their range."""
    rng = np.random.default_rng(9)
    V = 2000
    base = 3 * rng.standard_normal(V)
    rows = [base, base.copy(), base.copy(), base.copy(), np.full(V, -np.inf), base.copy(), base * 1e37, base * 1e-37]
    rows[1][rng.permutation(V)[:1900]] = -np.inf
    rows[2][17] = np.nan
    rows[3][18] = np.inf
    rows[5][:] = -np.inf
    rows[5][1234] = -3e38
    x = np.stack(rows)
    n = len(rows)
    u = uniform(rng, n, V)
    for t in (0.0, 1.0, 1e-30, 1e-38, 1e30, 3e38, math.inf, -1.0, math.nan):
        for arg in ({}, dict(k=np.full(n, 30)), dict(p=np.full(n, 0.9)), dict(m=np.full(n, 0.2)),
                    dict(k=np.full(n, 500), p=np.full(n, 0.7))):
            token = check(x, np.full(n, t), u, dist=True, **arg)
            assert token[4] == -1 and token[5] == 1234
            if t > 0:
                assert token[2] == token[3] == -1
    for k in (0, -5, V, V + 1, 2 ** 31 - 1, -2 ** 31):
        check(x[:2], np.ones(2), u[:2], k=np.full(2, k))
    for p in (1.0, 1.5, math.inf, math.nan, -1.0, -math.inf):
        check(x[:2], np.ones(2), u[:2], p=np.full(2, p))
    for m in (0.0, -1.0, math.nan, 1.0, 3.0, math.inf):
        check(x[:2], np.ones(2), u[:2], m=np.full(2, m))


def test_long_tails():
    """A cut far down: most of the mass in very many small weights, and a k that
    reaches weights too small to be drawn."""
    rng = np.random.default_rng(10)
    V, n = 50257, 4
    x = 0.01 * rng.standard_normal((n, V))
    x[:, 77] = 12.0
    x[3] = -np.arange(V) * 0.001
    u = uniform(rng, n, V)
    for p in (0.5, 0.9, 0.99999):
        check(x, np.ones(n), u, p=np.full(n, p))
    for k in (2, 1000, 30000):
        check(x, np.ones(n), u, k=np.full(n, k), dist=True)
        check(x, np.full(n, 0.05), u, k=np.full(n, k))
        check(x, np.ones(n), u, k=np.full(n, k), p=np.full(n, 0.97))


def test_distribution():
    """Over many draws the tokens have the distribution that is returned: with N
    draws a frequency is off by 6 sqrt(q (1 - q) / N) at most."""
    import torch
    rng = np.random.default_rng(12)
    V, N = 60, 40000
    row = 1.5 * rng.standard_normal(V)
    logits = torch.from_numpy(np.tile(row, (N, 1)).astype(np.float32)).cuda()
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    u = (torch.randint(0, 1 << 23, (N, V), generator=g, device="cuda").float() + 0.5) * 2.0 ** -23
    ones = torch.ones(N, device="cuda")
    dist = torch.empty((N, V), device="cuda")
    for arg in ({}, dict(top_k=torch.full((N,), 20, dtype=torch.int32, device="cuda"), top_p=ones * 0.85)):
        token, _ = binding.op_sample(logits, ones * 0.9, u, dist=dist, **arg)
        q = dist[0].double().cpu().numpy()
        f = np.bincount(token.cpu().numpy(), minlength=V) / N
        assert abs(q.sum() - 1) < 1e-5
        assert np.all(np.abs(f - q) <= 6 * np.sqrt(q * (1 - q) / N) + 1e-9)


def test_streams_and_graphs():
    """Another stream; a captured call replayed with other logits, settings and
    random numbers; two calls in flight at once."""
    import torch
    rng = np.random.default_rng(13)
    n, V = 12, 5003
    x = torch.from_numpy(peaked(rng, n, V).astype(np.float32)).cuda()
    u = torch.from_numpy(uniform(rng, n, V).astype(np.float32)).cuda()
    t, p = torch.ones(n, device="cuda"), torch.full((n,), 0.9, device="cuda")
    k = torch.full((n,), 40, dtype=torch.int32, device="cuda")
    want = binding.op_sample(x, t, u, k, p)[0]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [binding.op_sample(x, t, u, k, p, stream=s)[0] for s in streams for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) for a in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token, prob = binding.op_sample(x, t, u, k, p)
    for turn in range(3):
        x.copy_(torch.from_numpy(peaked(rng, n, V).astype(np.float32)))
        u.copy_(torch.from_numpy(uniform(rng, n, V).astype(np.float32)))
        t.fill_(0.5 + turn * 0.4)
        k.fill_(10 + 300 * turn)
        graph.replay()
        torch.cuda.synchronize()
        a, b = binding.op_sample(x, t, u, k, p)
        assert torch.equal(token, a) and torch.equal(prob, b)


def test_binding_refuses():
    import torch
    x = torch.zeros((3, 50), device="cuda")
    t, u = torch.ones(3, device="cuda"), torch.full((3, 50), 0.5, device="cuda")
    k = torch.ones(3, dtype=torch.int32, device="cuda")
    binding.op_sample(x, t, u, k, t, t)
    for bad in (dict(logits=x.double()), dict(logits=x[0]), dict(logits=x.cpu()), dict(logits=x.t()),
                dict(logits=x.expand(3, 50)[:, ::2]), dict(temperature=t[:2]), dict(temperature=k), dict(u=u[:, :9]),
                dict(u=None), dict(top_k=t), dict(top_p=k), dict(min_p=t.cpu()), dict(token=t), dict(prob=k),
                dict(dist=u[:2]), dict(logits=x[:1].expand(3, 50))):
        with pytest.raises(ValueError):
            binding.op_sample(**{**dict(logits=x, temperature=t, u=u, top_k=k, top_p=t, min_p=t), **bad})
    token, prob = binding.op_sample(x)               # greedy, without random numbers
    assert token.tolist() == [0, 0, 0] and prob.tolist() == [1, 1, 1]
    out = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert binding.op_sample(x, token=out)[0] is out or torch.equal(out, token)
    assert binding.op_sample(x[:0])[0].shape == (0,)
