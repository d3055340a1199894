"""GPU parity of the paged-cache operations (block tables and slot maps,
attention over pages) against plain implementations in 64 bits."""
import math

import numpy as np
import pytest

from transformer_decode_token_gb300 import binding

from test_gpu_spec import COMBOS, DIMS, dt, i32, make_cache

pytestmark = pytest.mark.gpu


# ---- block tables and slot maps ------------------------------------------------------------

def page_map_plain(cached, grow, table, ring, state, bs, n_rows):
    """The definition in gpt2.h, a sequence at a time."""
    table, ring = table.copy(), ring.copy()
    n, width = len(ring), table.shape[1]
    count = min(max(int(state[1]), 0), n)
    head = int(state[0]) % n
    out, first, rows = [], [0], []
    start = asked = used = back = 0
    for b in range(len(cached)):
        c, g = min(max(int(cached[b]), 0), width * bs), int(grow[b])
        have, end = -(-c // bs), start + max(g, 0)
        served = False
        if g < 0:
            for k in range(have):
                if count + back < n:
                    ring[(head + count + back) % n] = table[b, k]
                    back += 1
            out.append(0)
        else:
            if end <= n_rows and c + g <= width * bs:
                need = -(-(c + g) // bs) - have
                asked += need
                served = need == 0 or asked <= count
                if served:
                    for k in range(need):
                        table[b, have + k] = ring[(head + used) % n]
                        used += 1
            out.append(c + g if served else c)
        for t in range(max(0, min(end, n_rows) - start)):
            p = c + t
            rows.append((b, table[b, p // bs], p % bs, p) if served else (b, -1, -1, -1))
        start = end
        first.append(min(end, n_rows))
    rows += [(-1, -1, -1, -1)] * (n_rows - len(rows))
    new = [(head + used) % n, count - used + back]
    return [np.array(x, np.int64) for x in (out, new, first)] + list(np.array(rows, np.int64).reshape(n_rows, 4).T) + \
        [table, ring]


def check_map(cached, grow, table, ring, state, bs, n_rows, in_place=False):
    import torch
    want = page_map_plain(cached, grow, table, ring, state, bs, n_rows)
    t = [i32(x) for x in (cached, grow, table, ring, state)]
    got = binding.op_page_map(*t, bs, n_rows, *((t[0], t[4]) if in_place else ()))
    torch.cuda.synchronize()
    if in_place:
        assert got[0] is t[0] and got[1] is t[4]
    for name, g, w in zip(("cached_out", "free_state_out", "first", "seq", "slot", "offset", "position", "table",
                           "free_blocks"), list(got) + [t[2], t[3]], want):
        assert np.array_equal(g.cpu().numpy(), w), name
    return want


def random_pages(rng, B, bs, width, free, longest):
    """Sequences of random lengths that hold distinct blocks, and a ring of the rest."""
    cached = rng.integers(0, longest + 1, B)
    have = -(-cached // bs)
    n = int(have.sum()) + free
    order = rng.permutation(max(n, 1))
    table = np.full((B, width), -7, np.int64)
    at = 0
    for b in range(B):
        table[b, :have[b]] = order[at:at + have[b]]
        at += have[b]
    ring = np.full(max(n, 1), -9, np.int64)
    head = int(rng.integers(0, max(n, 1)))
    ring[(head + np.arange(free)) % max(n, 1)] = order[at:at + free]
    return cached, table, ring, np.array([head, free])


@pytest.mark.parametrize("B,bs,width,free,longest,n_rows", [
    (1, 16, 4, 3, 40, 8), (7, 16, 8, 40, 100, 64), (64, 16, 64, 200, 1000, 64), (300, 7, 30, 100, 150, 2500),
    (1000, 1, 50, 900, 40, 700), (513, 64, 20, 2000, 1200, 9000), (8192, 8, 10, 5000, 60, 20000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_page_map_is_the_definition(B, bs, width, free, longest, n_rows, in_place):
    """Mixes of single tokens, prompts, sequences that rest and that leave, with
    too few rows, blocks or table entries for some of them."""
    rng = np.random.default_rng(B + bs)
    cached, table, ring, state = random_pages(rng, B, bs, width, free, longest)
    kind = rng.integers(0, 6, B)
    grow = np.select([kind < 3, kind == 3, kind == 4], [1, rng.integers(0, 3 * bs + 2, B), 0], -1)
    check_map(cached, grow, table, ring, state, bs, n_rows, in_place)


def test_page_map_edges():
    """No sequences; nothing to do; no rows; lengths outside their range; a ring
    that has run out and one that is full; growth past 32 bits in all."""
    rng = np.random.default_rng(3)
    ring = np.array([4, 2, 9, 1, 0])
    for state in ([0, 5], [3, 4], [4, 0], [-1, 9], [7, -3]):
        check_map(np.array([], np.int64), np.array([], np.int64), np.zeros((0, 3), np.int64), ring, state, 16, 4)
        check_map(np.array([5, 0, 31]), np.array([0, 0, 0]), np.arange(9).reshape(3, 3), ring, state, 16, 0)
        check_map(np.array([-4, 1000, 16, 48]), np.array([1, 1, 1, -1]), np.arange(12).reshape(4, 3), ring, state, 16, 9)
        check_map(np.array([16, 15, 16]), np.array([1, 1, 17]), np.arange(9).reshape(3, 3), ring, state, 16, 19)
        check_map(np.array([3, 2, 4]), np.array([2 ** 31 - 1, 2 ** 31 - 1, 1]), np.arange(9).reshape(3, 3), ring, state,
                  16, 5)
        check_map(np.array([40, 48]), np.array([-1, -(2 ** 31)]), np.arange(6).reshape(2, 3), ring, state, 16, 2)


def test_page_map_over_many_steps():
    """A server's life: requests begin, grow and leave, in place; no block is
    held twice or lost, and what a sequence holds stays where it is."""
    import torch
    rng = np.random.default_rng(11)
    B, bs, width, n = 40, 16, 12, 260
    cached, table = i32(np.zeros(B)), i32(np.full((B, width), -1))
    ring, state = i32(rng.permutation(n)), i32([0, n])
    left = rng.integers(-20, 150, B)
    lens = np.zeros(B, np.int64)
    for step in range(120):
        grow = np.where(left == 0, -1, np.where(left > 0, 1, 0))
        begin = (lens == 0) & (left > 0)
        grow[begin] = rng.integers(1, 60, begin.sum())
        binding.op_page_map(cached, i32(grow), table, ring, state, bs, 256, cached, state)
        now = cached.cpu().numpy()
        served = now == lens + np.maximum(grow, 0)
        assert (now[(~served) & (grow >= 0)] == lens[(~served) & (grow >= 0)]).all() and (now[grow < 0] == 0).all()
        left = np.where(grow < 0, rng.integers(-20, 150, B), np.where(served & (left > 0), left - 1, np.where(left < 0, left + 1, left)))
        left = np.where((now >= width * bs - 1) & (grow >= 0), 0, left)
        lens = now.astype(np.int64)
        t, r, (h, c) = table.cpu().numpy(), ring.cpu().numpy(), state.tolist()
        held = [t[b, k] for b in range(B) for k in range(-(-lens[b] // bs))]
        free = [r[(h + i) % n] for i in range(c)]
        assert sorted(held + free) == list(range(n))
    assert lens.max() > 100


# ---- attention over pages ------------------------------------------------------------------

def pages(rng, ct, lens, bs, K, D, spare=2):
    """A paged cache whose sequences' blocks lie in random order, and its table."""
    have = [-(-n // bs) for n in lens]
    n, width = sum(have) + spare, max(have + [1])
    kc, ks = make_cache(rng, ct, n, K, bs, D)
    vc, vs = make_cache(rng, ct, n, K, bs, D)
    order = rng.permutation(n)
    table = np.full((len(lens), width), -1, np.int64)
    at = 0
    for b, h in enumerate(have):
        table[b, :h] = order[at:at + h]
        at += h
    return kc, vc, ks, vs, table


def paged64(q, kc, vc, ks, vs, table, position, seq, scale):
    """Per (row, head) in float64, and the error allowed for each element."""
    import torch
    q = q.float().cpu().numpy().astype(np.float64)
    n, H, D = q.shape
    N, K, bs, _ = kc.shape

    def wide(c, s):
        c = c.cpu().float().numpy().astype(np.float64)
        return c if s is None else c * s.cpu().numpy().astype(np.float64)[..., None]

    k, v = wide(kc, ks), wide(vc, vs)
    out, tol = np.zeros((n, H, D)), np.zeros((n, H, D))
    for r in range(n):
        b = r if seq is None else int(seq[r])
        if not 0 <= b < table.shape[0]:
            continue
        j = np.arange(min(int(position[r]) + 1, table.shape[1] * bs))
        block = table[b][j // bs]
        yes = (block >= 0) & (block < N)
        block, off = block[yes], (j % bs)[yes]
        if not len(block):
            continue
        for h in range(H):
            kk, vv = k[block, h // (H // K), off], v[block, h // (H // K), off]
            with np.errstate(all="ignore"):
                a = kk @ q[r, h] * scale
                if a.max() == -np.inf:
                    continue
                w = np.exp(a - a.max())
                w /= w.sum()
                out[r, h] = w @ vv
            size = (np.abs(kk) @ np.abs(q[r, h])).max() * abs(scale)
            tol[r, h] = (2 * size * 2.0 ** -18 + 2.0 ** -16) * (w @ np.abs(vv))
            if kc.dtype == torch.float16:
                # two fp16 parts of the weights in units of 2^-13 of the largest: what
                # the second drops below fp16's smallest step is at most 2^-25 / 2^13
                tol[r, h] += len(block) * 2.0 ** -38 * np.abs(vv).max()
    return out, tol


def check_close(got, want, tol):
    """A score sums at most 128 / 2 products in fp32 one after another (each off by
    at most 2^-24 of the sum of |q k| scale, log2(e) times that in the exponent),
    so it is off by less than 2^-18 of it; a weight by that much relatively, twice (numerator and
    denominator), and 2^-16 for its two parts of bf16 and the sums over a share
    (at most some 200 terms one after another); then half a step of the result's type."""
    import torch
    g = got.double().cpu().numpy()
    lim = tol + np.abs(want) * torch.finfo(got.dtype).eps / 2 + 1e-30
    if got.dtype == torch.float16:
        lim = lim + 2.0 ** -25           # half a step below fp16's normal numbers
    err = np.abs(g - want)
    assert np.all(err <= lim), f"worst {np.nanmax(err / lim):.3g} of what is allowed, {err.max():.3g}"


def run_paged(rng, qt, ct, D, K, G, bs, position, seq=None, lens=None, scale=None):
    import torch
    lens = lens or [max(p + 1, 0) for p in position]
    kc, vc, ks, vs, table = pages(rng, ct, lens, bs, K, D)
    n = len(position)
    q = torch.from_numpy((1.5 * rng.standard_normal((n, K * G, D))).astype(np.float32)).to(dt(qt)).cuda()
    out = torch.full_like(q, 77.0)
    got = binding.op_paged_attention(q, kc, vc, i32(table), i32(position), None if seq is None else i32(seq), ks, vs,
                                     scale=scale, out=out)
    assert got is out
    want, tol = paged64(q, kc, vc, ks, vs, table, position, seq, 1 / math.sqrt(D) if scale is None else scale)
    check_close(got, want, tol)
    return q, kc, vc, ks, vs, table, got


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("qt,ct", COMBOS)
@pytest.mark.parametrize("G", [1, 2, 3, 8, 12])
def test_paged_attention_types(qt, ct, D, G):
    """Every type, head size and kernel: lengths around the tiles and pages, a
    row that sees nothing."""
    run_paged(np.random.default_rng(D + G), qt, ct, D, 2, G, 16, [0, 14, 15, 16, 31, 32, 33, 63, 64, 100, -1, 300])


@pytest.mark.parametrize("bs", [1, 3, 8, 24, 128, 1000])
@pytest.mark.parametrize("qt,ct,G", [("f32", "f32", 1), ("f32", "int8", 1), ("bf16", "bf16", 4), ("f16", "e4m3", 5)])
def test_page_sizes(qt, ct, G, bs):
    run_paged(np.random.default_rng(bs), qt, ct, 64, 3, G, bs, [200, 5, 63, 0, 127, 999, 24, 1])


@pytest.mark.parametrize("G", [1, 2, 4, 5, 8, 9, 12, 16, 17])
@pytest.mark.parametrize("qt,ct", [("f32", "f32"), ("f32", "bf16"), ("f32", "e4m3"), ("bf16", "int8"), ("f16", "f16")])
def test_groups_of_heads(qt, ct, G):
    run_paged(np.random.default_rng(G), qt, ct, 64, 2, G, 16, [90, 33, 4, 257])


@pytest.mark.parametrize("qt,ct,G", [("f32", "f32", 1), ("f32", "bf16", 1), ("f32", "int8", 2), ("bf16", "bf16", 8),
                                     ("f16", "int8", 4), ("bf16", "bf16", 16), ("f16", "e4m3", 11)])
@pytest.mark.parametrize("position", [[9000], [4500, -1, 3], [700] * 150, list(range(-1, 260, 3))])
def test_splits(qt, ct, G, position):
    """One long row cut into many parts, rows shorter than a share, equal rows,
    rows of every length; every call gives the same bits."""
    import torch
    rng = np.random.default_rng(len(position))
    q, kc, vc, ks, vs, table, got = run_paged(rng, qt, ct, 64 if len(position) > 3 else 128, 2, G, 16, position)
    again = binding.op_paged_attention(q, kc, vc, i32(table), i32(position), None, ks, vs)
    assert torch.equal(again, got)


@pytest.mark.parametrize("qt,ct,G", [("f32", "bf16", 1), ("bf16", "bf16", 4)])
def test_rows_of_one_sequence(qt, ct, G):
    """Several rows of a sequence, in any order (a prompt's positions, a drafted
    chain), rows of a sequence that is none, positions past the table."""
    rng = np.random.default_rng(8)
    seq = [2, 0, 0, 0, 1, 2, 2, -1, 3, 1, 0]
    position = [70, 3, 4, 5, 20, 0, 71, 5, 5, 1000, -3]
    run_paged(rng, qt, ct, 64, 2, G, 16, position, seq=seq, lens=[10, 40, 72])


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
@pytest.mark.parametrize("G", [1, 4])
def test_scales(scale, G):
    run_paged(np.random.default_rng(1), "bf16", "bf16", 64, 2, G, 16, [100, 7], scale=scale)


@pytest.mark.parametrize("ct,e", [(ct, e) for ct in ("int8", "e4m3", "bf16", "f32") for e in (-100, -60, 60, 110)] +
                         [("int8", -113), ("e4m3", -113)])
@pytest.mark.parametrize("G", [1, 4, 12])
def test_sizes_of_queries(ct, G, e):
    """bf16 queries far outside fp16's range, their elements 2^0 to 2^-24 apart, a
    head of zeros: the scores are ordinary again by the call's scale."""
    import torch
    rng = np.random.default_rng(G)
    D, K, position = 64, 2, [300, 40, 5]
    kc, vc, ks, vs, table = pages(rng, ct, [p + 1 for p in position], 16, K, D)
    q = 1.5 * rng.standard_normal((3, K * G, D)) * 2.0 ** (e - rng.integers(0, 25, (3, K * G, D)))
    q[:, 1] = 0
    q = torch.from_numpy(q).to(torch.bfloat16 if ct != "f32" else torch.float32).cuda()
    got = binding.op_paged_attention(q, kc, vc, i32(table), i32(position), None, ks, vs, scale=2.0 ** -e / 4)
    want, tol = paged64(q, kc, vc, ks, vs, table, position, None, 2.0 ** -e / 4)
    check_close(got, want, tol)


def test_nothing_to_do():
    """No rows, no sequences: results of these shapes on the device."""
    import torch
    c = torch.zeros(2, 2, 4, 64, device="cuda")
    got = binding.op_paged_attention(torch.zeros(0, 2, 64, device="cuda"), c, c, i32(np.zeros((3, 2))), i32([]))
    assert got.shape == (0, 2, 64) and got.is_cuda and got.dtype == torch.float32 and got.clone().numel() == 0
    token, prob = binding.op_sample(torch.zeros(0, 7, device="cuda"))
    assert token.shape == prob.shape == (0,) and token.is_cuda and token.dtype == torch.int32 and prob.dtype == torch.float32
    check_map(np.array([], np.int64), np.array([], np.int64), np.zeros((0, 1), np.int64), np.array([3]), [0, 1], 1, 0)
    x = binding.op_page_map(i32([3]), i32([1]), i32([[0]]), i32([1]), i32([0, 1]), 4, 1)
    assert all(t.is_contiguous() and t.device == c.device for t in x) and [len(t) for t in x] == [1, 2, 2, 1, 1, 1, 1]
    assert (x[0] + 1).tolist() == [5] and torch.cat(x).tolist() == [4, 0, 1, 0, 1, 0, 0, 3, 3]


@pytest.mark.parametrize("qt,ct", COMBOS)
@pytest.mark.parametrize("G", [1, 4, 12])
def test_what_is_not_seen_does_not_enter(qt, ct, G):
    """NaN everywhere but in the rows that are seen (behind the last position in its
    page, in other pages): codes of 8-bit caches by their scales.  Blocks outside
    the cache are not seen, and a row all of whose blocks are outside gets zeros."""
    import torch
    rng = np.random.default_rng(5)
    D, K, bs, position = 64, 2, 16, [37, 0, 100, 64, 20]
    kc, vc, ks, vs, table = pages(rng, ct, [p + 1 for p in position], bs, K, D)
    table[2, 1], table[2, 4], table[3, :] = -5, kc.shape[0], 1 << 30
    seen = torch.zeros(kc.shape[:3], dtype=torch.bool)
    for b, p in enumerate(position):
        for j in range(p + 1):
            if 0 <= table[b, j // bs] < kc.shape[0]:
                seen[table[b, j // bs], :, j % bs] = True
    clean = [None if t is None else t.clone() for t in (kc, vc, ks, vs)]
    for c, s in ((kc, ks), (vc, vs)):
        if s is not None:
            s[~seen] = math.nan
        else:
            c[~seen] = math.nan
    q = torch.from_numpy((1.5 * rng.standard_normal((len(position), K * G, D))).astype(np.float32)).to(dt(qt)).cuda()
    got = binding.op_paged_attention(q, kc, vc, i32(table), i32(position), None, ks, vs)
    want, tol = paged64(q, *clean, table, position, None, 1 / 8)
    check_close(got, want, tol)
    assert (got[3] == 0).all()


@pytest.mark.parametrize("qt,ct", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "int8"),
                                   ("f16", "e4m3")])
@pytest.mark.parametrize("G", [1, 4, 12])
@pytest.mark.parametrize("n", [20, 3000])
def test_infinities_that_are_seen(qt, ct, G, n):
    """An infinite value gives an infinity in its dimension (in both: a NaN) and
    leaves the others; a key of score -infinity has the weight zero; a NaN key
    makes a NaN of its head's row alone; whole units and cut ones (n keys)."""
    import torch
    rng = np.random.default_rng(n)
    D, K, bs = 64, 3, 16
    kc, vc, ks, vs, table = pages(rng, ct, [n, n], bs, K, D)
    q = torch.from_numpy(np.abs(rng.standard_normal((2, K * G, D))).astype(np.float32) + 0.25).to(dt(qt)).cuda()
    scaled = ks is not None
    at = lambda b, j: (int(table[b, j // bs]), j % bs)
    b0, o0 = at(0, n // 2)
    b1, o1 = at(0, n // 3)
    b2, o2 = at(1, n - 1)
    if scaled:
        # (codes are finite: an infinite scale of the row; its sign is the code's)
        vc[b0, 0, o0] = vc[b0, 0, o0].float().abs().clamp(min=1).to(vc.dtype)
        vs[b0, 0, o0] = math.inf
        kc[b1, 1, o1] = (-kc[b1, 1, o1].float().abs().clamp(min=1)).to(kc.dtype)
        ks[b1, 1, o1] = math.inf
        ks[b2, 2, o2] = math.nan
    else:
        vc[b0, 0, o0, 5], vc[b0, 0, o0, 6] = math.inf, -math.inf
        b3, o3 = at(0, n // 2 + 1)
        vc[b0, 0, o0, 7], vc[b3, 0, o3, 7] = math.inf, -math.inf
        kc[b1, 1, o1, 9] = -math.inf
        kc[b2, 2, o2, 3] = math.nan
    got = binding.op_paged_attention(q, kc, vc, i32(table), i32([n - 1, n - 1]), None, ks, vs).double().cpu().numpy()
    r0, r1, r2 = (got[:, h * G:(h + 1) * G] for h in range(3))
    assert np.isnan(r2[1]).all() and np.isfinite(r2[0]).all() and np.isfinite(r0[1]).all()
    assert np.isfinite(r1).all()
    if scaled:
        assert (r0[0] == math.inf).all()
    else:
        assert (r0[0, :, 5] == math.inf).all() and (r0[0, :, 6] == -math.inf).all() and np.isnan(r0[0, :, 7]).all()
        assert np.isfinite(np.delete(r0[0], [5, 6, 7], 1)).all()
        # the key of score -infinity: as if it were not there
        keep = kc.clone()
        keep[b1, 1, o1, 9] = 0
        vals = vc.clone()
        vals[~torch.isfinite(vals)] = 0
        k2 = torch.nan_to_num(keep)
        want, tol = paged64(q, k2, vals, None, None, table, [n - 1, n - 1], None, 1 / 8)
        kk = np.stack([k2[table[0, j // bs], 1, j % bs].double().cpu().numpy() for j in range(n)])
        vv = np.stack([vals[table[0, j // bs], 1, j % bs].double().cpu().numpy() for j in range(n)])
        for h in range(G):
            a = kk @ q[0, G + h].double().cpu().numpy() / 8
            a[n // 3] = -math.inf
            w = np.exp(a - a.max())
            check_close(torch.from_numpy(got[0, G + h]).to(dt(qt)), w @ vv / w.sum(), 2 * tol[0, G + h])


def test_strided_rows_streams_and_graphs():
    """q inside fused rows, out inside wider ones; another stream; a captured and
    replayed call with positions and tables that changed, two workspaces apart."""
    import torch
    rng = np.random.default_rng(2)
    D, K, G, bs, B = 64, 3, 1, 16, 20
    lens = [int(x) for x in rng.integers(1, 200, B)]
    kc, vc, ks, vs, table = pages(rng, "bf16", [200] * B, bs, K, D)
    wide = torch.from_numpy(rng.standard_normal((B, 3 * K * D)).astype(np.float32)).cuda()
    q = wide[:, :K * D].unflatten(1, (K, D))
    out = torch.full((B, K * D + 8), 5.0, device="cuda")
    o = out[:, :K * D].unflatten(1, (K, D))
    pos = i32([n - 1 for n in lens])
    t = i32(table)
    want, tol = paged64(q, kc, vc, ks, vs, table, [n - 1 for n in lens], None, 1 / 8)
    binding.op_paged_attention(q, kc, vc, t, pos, out=o)
    check_close(o, want, tol)
    assert (out[:, K * D:] == 5).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = binding.op_paged_attention(q, kc, vc, t, pos, stream=side)
    side.synchronize()
    assert torch.equal(got, o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = binding.op_paged_attention(q, kc, vc, t, pos)
        b = binding.op_paged_attention(q, kc, vc, t, pos)
    for turn in range(3):
        now = [int(x) for x in rng.integers(-1, 200, B)]
        pos.copy_(i32(now))
        line = table[rng.permutation(B)]
        t.copy_(i32(line))
        graph.replay()
        torch.cuda.synchronize()
        want, tol = paged64(q, kc, vc, ks, vs, line, now, None, 1 / 8)
        check_close(a, want, tol)
        assert torch.equal(a, b)


def test_many_rows():
    """More rows than a CTA has threads, most of them short."""
    rng = np.random.default_rng(4)
    seq = rng.integers(0, 6, 1500)
    position = np.minimum(rng.integers(-1, 90, 1500), 60 + seq)
    run_paged(rng, "f32", "f16", 32, 2, 1, 16, position.tolist(), seq=seq.tolist(), lens=[100] * 6)


def test_offsets_past_32_bits():
    """Blocks whose bytes lie past 2^32 in the cache."""
    import torch
    rng = np.random.default_rng(6)
    D, K, bs, N = 128, 2, 16, 270000                       # 4.4 GB each of keys and values
    kc, vc = (torch.empty((N, K, bs, D), dtype=torch.float32, device="cuda") for _ in range(2))
    blocks = [N - 1, 3, N - 7, 262144, N - 2]
    small, where = [], i32(blocks).long()
    for c in (kc, vc):
        x = torch.from_numpy(rng.standard_normal((len(blocks), K, bs, D)).astype(np.float32)).cuda()
        c[where] = x
        small.append(x)
    q = torch.from_numpy(rng.standard_normal((1, K, D)).astype(np.float32)).cuda()
    got = binding.op_paged_attention(q, kc, vc, i32([blocks]), i32([70]))
    want, tol = paged64(q, *small, None, None, np.arange(5)[None], [70], None, 1 / math.sqrt(D))
    check_close(got, want, tol)


def test_blocks_of_very_many_rows():
    """A table whose few blocks hold 2^28 rows each: what 32 of them would hold passes
    32 bits, and the entries behind the table's end are not read."""
    import torch
    rng = np.random.default_rng(7)
    bs, D = 1 << 28, 32
    kc, vc = (torch.empty((1, 1, bs, D), dtype=torch.int8, device="cuda") for _ in "kv")
    ks, vs = (torch.empty((1, 1, bs), device="cuda") for _ in "kv")
    small = []
    for c in (kc, vc):
        c[0, 0, :200] = torch.from_numpy(rng.integers(-127, 128, (200, D)).astype(np.int8)).cuda()
        small.append(c[:, :, :200].clone())
    for s in (ks, vs):
        s[0, 0, :200] = 0.02
        small.append(s[:, :, :200].clone())
    q = torch.from_numpy(rng.standard_normal((2, 1, D)).astype(np.float32)).cuda()
    got = binding.op_paged_attention(q, kc, vc, i32([[0], [0]]), i32([150, 31]), None, ks, vs)
    want, tol = paged64(q, *small, np.zeros((2, 1), np.int64), [150, 31], None, 1 / math.sqrt(D))
    check_close(got, want, tol)


def test_binding_refuses():
    import torch
    rng = np.random.default_rng(1)
    kc, vc, ks, vs, table = pages(rng, "int8", [20, 30], 16, 2, 64)
    t, p = i32(table), i32([19, 29])
    q = torch.zeros((2, 2, 64), device="cuda")
    ok = dict(q=q, k_cache=kc, v_cache=vc, table=t, position=p, k_scale=ks, v_scale=vs)
    binding.op_paged_attention(**ok)
    for bad in (dict(q=q.double()), dict(q=q.cpu()), dict(q=q[0]), dict(q=q[:, :, :32]), dict(q=q.transpose(0, 1)),
                dict(k_scale=None), dict(k_scale=ks[:1]), dict(table=t.long()), dict(table=t[0]), dict(table=t[:1]),
                dict(table=t.cpu()), dict(table=t.t()), dict(position=p[:1]), dict(position=p.float()),
                dict(seq=p[:1]), dict(seq=p.long()), dict(out=q.half()), dict(out=q[:1]), dict(scale="x"),
                dict(workspace=torch.zeros(8))):
        with pytest.raises(ValueError):
            binding.op_paged_attention(**{**ok, **bad})
    with pytest.raises(binding.GPT2Error):
        binding.op_paged_attention(**ok, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(binding.GPT2Error):
        binding.op_paged_attention(**ok, scale=math.inf)
    c, g, f, s = i32([3, 4]), i32([1, 1]), i32(np.arange(9)), i32([0, 9])
    binding.op_page_map(c, g, t, f, s, 16, 2)
    for bad in (lambda: binding.op_page_map(c.long(), g, t, f, s, 16, 2), lambda: binding.op_page_map(c, g[:1], t, f, s, 16, 2),
                lambda: binding.op_page_map(c, g, t[:1], f, s, 16, 2), lambda: binding.op_page_map(c, g, t, f, s[:1], 16, 2),
                lambda: binding.op_page_map(c, g, t, f[:0], s, 16, 2), lambda: binding.op_page_map(c, g, t, f, s, 16, -1),
                lambda: binding.op_page_map(c, g, t, f, s, "16", 2), lambda: binding.op_page_map(c, g, t, f, s, 16, 2, g[:1]),
                lambda: binding.op_page_map(c.cpu(), g, t, f, s, 16, 2)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(binding.GPT2Error):
        binding.op_page_map(c, g, t, f, s, 0, 2)
    # nothing to do
    assert binding.op_paged_attention(q[:0], kc, vc, t, p[:0], None, ks, vs).shape == (0, 2, 64)
